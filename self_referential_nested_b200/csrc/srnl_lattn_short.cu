// Linear attention over at most 16 tokens (sm_100a): a decayed pass (srnl_lattn.cu) written out for
// a sequence that is no longer than a corner of the tensor cores' tiles,
//   out_i = sum_{j <= i} g^(i - j) (a_i . b_j) c_j + g^(i + lead) Z0^T a_i,   Zn = g^n Z0 + sum_j w_j b_j c_j^T
// all in fp32.  A block of 128 threads (256 for 128-wide heads) takes one (pass, sequence, head); a thread owns a channel of c
// and a share of the tokens.  a and b lie transposed in shared memory, so that a row of the state
// meets the tokens in 16-byte broadcasts; c stays in registers; the state comes 32 rows at a time,
// a piece ahead.
//
// What bounds it: the states' bytes where they come or go (64 sequences of 16 tokens, 16 heads of 128,
// both: 71 us, 2.1 TB/s; 113 on the tensor cores), else latency: the blocks are small and many of them
// share an SM (backward of 36 sequences of one token, 31 heads of 64: 11 us; 63 on the tensor cores,
// whose CTAs take 5 us each however few tokens they hold).  At 32 tokens the products' time counts:
// 64 sequences, 16 heads of 64, with states: 79 us, 46 on the tensor cores.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "srnl_lattn.h"

namespace srnl {
namespace {

using bf16 = __nv_bfloat16;
__host__ __device__ constexpr int short_threads(int d) { return d == 128 ? 256 : 128; }

template <int D, int TT>
constexpr size_t short_smem() { return (size_t)(2 * D * TT + TT * (TT + 4) + 32 * (D + 4)) * sizeof(float); }

template <int D, int TT>
__global__ void __launch_bounds__(short_threads(D), D == 128 ? (TT == 8 ? 4 : 3) : TT == 8 ? 6 : 4)
    decay_short_kernel(const __grid_constant__ LaArgs args) {
  constexpr int kThreads = short_threads(D), G = kThreads / D, TG = TT / G;   // threads of a channel, tokens of a thread
  constexpr int kP = TT + 4;
  extern __shared__ __align__(16) float sm[];
  float *aT = sm, *bT = aT + D * TT, *p = bT + D * TT, *zt = p + TT * kP;
  const int tid = threadIdx.x, c = tid % D, tg = tid / D;
  const int head = blockIdx.x % args.heads, batch = blockIdx.x / args.heads;
  const LaPass& P = args.pass[blockIdx.z];
  const float lg = args.log2g[head];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int n = args.lengths != nullptr ? min(max(args.lengths[batch], 0), args.T) : args.T;
  const int lead = P.reverse ? 0 : 1;   // a reversed pass's state meets its first token undecayed
  const int64_t row0 = (int64_t)batch * args.T + (P.reverse ? n - 1 : 0), step = P.reverse ? -1 : 1;   // tokens in the pass's order

  // tokens behind the last one are zeros: they may hold anything
  for (int u = tid; u < TT * (D / 8); u += kThreads) {
    const int i = u % TT, ch = u / TT * 8;
    uint4 av = make_uint4(0u, 0u, 0u, 0u), bv = av;
    if (i < n) {
      av = *reinterpret_cast<const uint4*>(P.a + (row0 + step * i) * P.lda + head * D + ch);
      bv = *reinterpret_cast<const uint4*>(P.b + (row0 + step * i) * P.ldb + head * D + ch);
    }
    const uint32_t aw[4] = {av.x, av.y, av.z, av.w}, bw[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      aT[(ch + e) * TT + i] = __uint_as_float(e & 1 ? aw[e / 2] & 0xFFFF0000u : aw[e / 2] << 16);
      bT[(ch + e) * TT + i] = __uint_as_float(e & 1 ? bw[e / 2] & 0xFFFF0000u : bw[e / 2] << 16);
    }
  }
  float cv[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) cv[j] = j < n ? __bfloat162float(P.c[(row0 + step * j) * P.ldc + head * D + c]) : 0.f;
  __syncthreads();
  // the masked products of a and b, a column j and some rows a thread
  constexpr int kRows = TT * TT / kThreads > 0 ? TT * TT / kThreads : 1;
  if (tid < TT * (TT / kRows)) {
    const int j = tid % TT, i0 = tid / TT * kRows;
    float s[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) s[k] = 0.f;
#pragma unroll 4
    for (int r = 0; r < D; ++r) {
      const float b = bT[r * TT + j];
#pragma unroll
      for (int k = 0; k < kRows; ++k) s[k] = fmaf(aT[r * TT + i0 + k], b, s[k]);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) p[(i0 + k) * kP + j] = j <= i0 + k ? s[k] * exp2f(lg * (float)(i0 + k - j)) : 0.f;
  }
  __syncthreads();
  if (P.zn != nullptr) {   // w b: what each token still weighs behind the last one
    for (int u = tid; u < D * TT; u += kThreads) {
      const int i = u % TT;
      bT[u] *= i < n ? exp2f(lg * (float)(n - 1 - i + (1 - lead))) : 0.f;
    }
    __syncthreads();
  }
  float acc[TG];
#pragma unroll
  for (int k = 0; k < TG; ++k) acc[k] = 0.f;
  const int64_t at = ((int64_t)batch * args.heads + head) * D * D;
  if (P.z0 != nullptr || P.zn != nullptr) {
    constexpr int kZ = D + 4, kMine = 32 * D / kThreads;   // a piece's pitch; a thread's values of it
    const float gn = exp2f(lg * (float)n);
    float next[kMine];
    auto fetch = [&](int r0) {   // rows r0 .. + 31 of Z0; of its transpose's rows, 32 values by a warp
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int u = tid + k * kThreads;
        next[k] = P.z0_t ? P.z0[at + (int64_t)(u / 32) * D + r0 + u % 32] : P.z0[at + (int64_t)r0 * D + u];
      }
    };
    if (P.z0 != nullptr) fetch(0);
#pragma unroll 1
    for (int r0 = 0; r0 < D; r0 += 32) {
      if (P.z0 != nullptr) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const int u = tid + k * kThreads;
          zt[P.z0_t ? u % 32 * kZ + u / 32 : u / D * kZ + u % D] = next[k];
        }
        __syncthreads();
        if (r0 + 32 < D) fetch(r0 + 32);
      }
      if (P.z0 != nullptr)
#pragma unroll 4
        for (int r = 0; r < 32; ++r) {
          const float z = zt[r * kZ + c];
#pragma unroll
          for (int k = 0; k < TG; ++k) acc[k] = fmaf(aT[(r0 + r) * TT + tg * TG + k], z, acc[k]);
        }
      if (P.zn != nullptr)
#pragma unroll 2
        for (int r = tg; r < 32; r += G) {
          float s[4] = {P.z0 != nullptr ? gn * zt[r * kZ + c] : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < TT; ++j) s[j % 4] = fmaf(bT[(r0 + r) * TT + j], cv[j], s[j % 4]);
          P.zn[at + (int64_t)(r0 + r) * D + c] = (s[0] + s[1]) + (s[2] + s[3]);
        }
    }
  }
#pragma unroll
  for (int k = 0; k < TG; ++k) {
    const int i = tg * TG + k;
    if (i < n) {
      float o = acc[k] * exp2f(lg * (float)(i + lead));
#pragma unroll
      for (int j = 0; j < TT; ++j) o = fmaf(p[i * kP + j], j <= i ? cv[j] : 0.f, o);   // a later token may hold anything
      P.out[(row0 + step * i) * P.ldo + head * D + c] = __float2bfloat16_rn(o);
    }
  }
}

template <int D, int TT>
cudaError_t launch_short(const LaArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(a.B * a.heads), 1, (unsigned)a.passes);
  lc.blockDim = dim3(short_threads(D));
  lc.dynamicSmemBytes = short_smem<D, TT>();
  lc.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, decay_short_kernel<D, TT>, a);
}

template <int D>
cudaError_t launch_short(const LaArgs& a, cudaStream_t s) {
  return a.T <= 8 ? launch_short<D, 8>(a, s) : launch_short<D, kShortTokens>(a, s);
}

}  // namespace

cudaError_t launch_la_short(const LaArgs& a, cudaStream_t s) {
  return a.d == 128 ? launch_short<128>(a, s) : a.d == 64 ? launch_short<64>(a, s) : launch_short<32>(a, s);
}

}  // namespace srnl
