// Linear attention with a decay for each head (sm_100a): the plain decayed memory beside the
// SRNL sequence layer, with its backward pass and its form for single tokens.
//
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t     per (batch, head), g in (0, 1] per head
//
// Every pass over a sequence here is one form, a decayed pass over three rows a, b, c per token:
//   out_t = sum_{j <= t} g^(t - j) (a_t . b_j) c_j + g^(t + 1) Z0^T a_t,   Z = sum g^.. b c^T
// The forward is (q, k, v).  The gradients are three more, from the recurrence's derivative
// with R_t = g R_{t+1} + q_t do_t^T carried back:
//   dq_t = S_t do_t     (do, v, k), Z = S^T
//   dv_t = R_t^T k_t    (k, q, do) over the tokens in reverse, Z = R;  dS_0 = g R_1
//   dk_t = R_t v_t      (v, do, q) over the tokens in reverse, Z = R^T
//
// Chunked: within C tokens, with i, j the places in the chunk and Z the state at its start,
//   out = ((a b^T) * g^(i - j) [j <= i]) c + g^(i + 1) (a Z),   Z <- g^C Z + (g^(C - 1 - j) b_j)^T c
// so all powers are of g <= 1 with exponents >= 0 and nothing overflows.
//
// Roundings: the state is fp32 throughout.  As an operand of a Z it is split into two bf16
// parts (16 bits), and so are the decayed rows of the state's update, into three where the state
// itself is asked for; the masked a b^T is rounded to bf16 once; out is rounded once.
//
// Heads of 64 and 128 channels run on tcgen05 (srnl_lattn_tc.cu), 32-wide ones here: their
// products are too narrow for its 128 rows and go by mma.sync.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <new>
#include <vector>

#include "srnl_common.cuh"
#include "srnl_internal.h"
#include "srnl_lattn.h"
#include "srnl_scan.h"

namespace srnl {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint32_t s_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

constexpr int kD32 = 32, kWarps32 = 4;
constexpr int kC32 = 16 * kWarps32;        // tokens per chunk: a warp takes 16 of its rows
constexpr int kPitch32 = kD32 * 2 + 16;    // bytes of a shared row: ldmatrix rows in distinct banks
constexpr int kCols32 = 16;                // the state over 2 x 2 warps: 16 rows x 16 columns each
constexpr size_t kSmem32 = (size_t)(3 * kC32 + 2 * kD32) * kPitch32 + kC32 * 4;

// z <- g^m z.  A factor near one is applied as z + (g^m - 1) z: rounded to fp32 it would be off
// by the same half step in every chunk, which thousands of chunks add up.
template <int NB>
__device__ __forceinline__ void decay_state(float (&z)[NB][4], float lg, int m) {
  const float e = lg * (float)m;
  const bool near = e > -1.f;
  const float f = near ? expm1f(e * 0.69314718055994531f) : exp2f(e);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) z[i][k] = fmaf(z[i][k], f, near ? z[i][k] : 0.f);
}

// One CTA per (segment, sequence and head, pass).  kStateOnly: the state that the segment adds,
// from zero, to seg_state; otherwise the outputs, from the state at the segment's start.
template <bool kStateOnly>
__global__ void __launch_bounds__(kWarps32 * 32) decay_pass_kernel(const __grid_constant__ LaArgs args) {
  constexpr int D = kD32, C = kC32, NB = kCols32 / 8;
  extern __shared__ __align__(16) unsigned char sm[];
  unsigned char *sa = sm, *sb = sa + C * kPitch32, *sc = sb + C * kPitch32, *zh = sc + C * kPitch32,
                *zl = zh + D * kPitch32;
  float* w = reinterpret_cast<float*>(zl + D * kPitch32);   // g^(count - 1 - j)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const LaPass& P = args.pass[blockIdx.z];
  const int seg = blockIdx.x, head = blockIdx.y % args.heads, batch = blockIdx.y / args.heads;
  const float lg = args.log2g[head];
  int n = args.T;
  if (args.lengths != nullptr) n = min(max(args.lengths[batch], 0), args.T);
  const int begin = seg * args.seg_len, end = min(begin + args.seg_len, n);
  const int64_t zbase = ((int64_t)batch * args.heads + head) * D * D;
  const int64_t sbase = (((int64_t)blockIdx.z * args.B + batch) * args.heads + head) * args.segs * D * D;

  // the warp's part of the state: rows zr .. zr + 15, columns zc .. zc + 15
  const int zr = (warp >> 1) * 16, zc = (warp & 1) * kCols32;
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  float z[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) z[i][e] = 0.f;
  if constexpr (!kStateOnly) {
    // state at the segment's start: z0, and what each earlier segment added, decayed from its end
    const int from = min(begin, n);
    auto add = [&](const float* src, float f, int t) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = zr + r0 + (e >> 1) * 8, c = zc + i * 8 + c0 + (e & 1);
          z[i][e] = fmaf(f, t ? src[c * D + r] : src[r * D + c], z[i][e]);
        }
    };
    if (P.z0 != nullptr) add(P.z0 + zbase, exp2f(lg * (float)max(from - P.reverse, 0)), P.z0_t);
    for (int s = 0; s < seg; ++s) {
      const int se = min((s + 1) * args.seg_len, n);
      if (s * args.seg_len < n) add(args.seg_state + sbase + (int64_t)s * D * D, exp2f(lg * (float)(from - se)), 0);
    }
  }

  for (int t0 = begin; t0 < end; t0 += C) {
    const int cnt = min(C, end - t0);
    // z0 of a reversed pass meets its first token undecayed
    const int lead = (P.reverse && t0 == 0) ? 0 : 1;
    __syncthreads();   // the previous chunk's readers are done
    constexpr int V = D / 8;
    for (int idx = tid; idx < C * V; idx += kWarps32 * 32) {
      const int i = idx / V, v = idx - i * V;
      const bool on = i < cnt;
      const int t = P.reverse ? n - 1 - (t0 + i) : t0 + i;
      const int64_t row = (int64_t)batch * args.T + (on ? t : 0);
      const int col = head * D + v * 8;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (!kStateOnly)
        *reinterpret_cast<uint4*>(sa + i * kPitch32 + v * 16) = on ? *reinterpret_cast<const uint4*>(P.a + row * P.lda + col) : zero;
      *reinterpret_cast<uint4*>(sb + i * kPitch32 + v * 16) = on ? *reinterpret_cast<const uint4*>(P.b + row * P.ldb + col) : zero;
      *reinterpret_cast<uint4*>(sc + i * kPitch32 + v * 16) = on ? *reinterpret_cast<const uint4*>(P.c + row * P.ldc + col) : zero;
    }
    for (int j = tid; j < C; j += kWarps32 * 32) w[j] = j < cnt ? exp2f(lg * (float)(cnt - 1 - j)) : 0.f;
    if constexpr (!kStateOnly) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x = z[i][2 * h], y = z[i][2 * h + 1];
          const uint32_t hw = pack2(x, y);
          const uint32_t off = (uint32_t)(zr + r0 + 8 * h) * kPitch32 + (zc + i * 8 + c0) * 2;
          *reinterpret_cast<uint32_t*>(zh + off) = hw;
          *reinterpret_cast<uint32_t*>(zl + off) = pack2(x - lo_f(hw), y - hi_f(hw));
        }
    }
    __syncthreads();

    if constexpr (!kStateOnly) {
      const int row = warp * 16;
      // a's rows as the left operand: lanes 0-15 rows, the upper half 8 columns on
      const uint32_t a_at = s_u32(sa) + (row + (lane & 15)) * kPitch32 + (lane >> 4) * 16;
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      const uint32_t t_row = (lane & 7) + ((lane >> 3) & 1) * 8, t_col = (lane >> 4) * 8;   // transposed operand blocks
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t af[4];
        ldm4(af, a_at + k * 32);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t bh[4], bl[4];
          const uint32_t off = (k * 16 + t_row) * kPitch32 + (i * 16 + t_col) * 2;
          ldm4t(bh, s_u32(zh) + off);
          ldm4t(bl, s_u32(zl) + off);
          mma16816(o[2 * i], af, bh[0], bh[1]);
          mma16816(o[2 * i + 1], af, bh[2], bh[3]);
          mma16816(o[2 * i], af, bl[0], bl[1]);
          mma16816(o[2 * i + 1], af, bl[2], bl[3]);
        }
      }
      const int i0 = row + r0, i1 = i0 + 8;
      const float f0 = exp2f(lg * (float)(i0 + lead)), f1 = exp2f(lg * (float)(i1 + lead));
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= f0; o[i][1] *= f0;
        o[i][2] *= f1; o[i][3] *= f1;
      }
      // 16 columns of the masked a b^T at a time, up to the diagonal
#pragma unroll 1
      for (int jb = 0; jb <= warp; ++jb) {
        float p[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const uint32_t b_at = s_u32(sb) + (jb * 16 + (lane & 7) + (lane >> 4) * 8) * kPitch32 + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t af[4], bf[4];
          ldm4(af, a_at + k * 32);
          ldm4(bf, b_at + k * 32);
          mma16816(p[0], af, bf[0], bf[1]);
          mma16816(p[1], af, bf[2], bf[3]);
        }
        uint32_t pf[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = jb * 16 + h * 8 + c0;
          auto m = [&](float v, int i, int jj) { return jj <= i ? v * exp2f(lg * (float)(i - jj)) : 0.f; };
          pf[2 * h] = pack2(m(p[h][0], i0, j), m(p[h][1], i0, j + 1));
          pf[2 * h + 1] = pack2(m(p[h][2], i1, j), m(p[h][3], i1, j + 1));
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t cf[4];
          ldm4t(cf, s_u32(sc) + (jb * 16 + t_row) * kPitch32 + (i * 16 + t_col) * 2);
          mma16816(o[2 * i], pf, cf[0], cf[1]);
          mma16816(o[2 * i + 1], pf, cf[2], cf[3]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = row + r0 + 8 * h;
        if (i >= cnt) continue;
        const int t = P.reverse ? n - 1 - (t0 + i) : t0 + i;
        bf16* dst = P.out + ((int64_t)batch * args.T + t) * P.ldo + head * D;
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
          *reinterpret_cast<uint32_t*>(dst + k * 8 + c0) = pack2(o[k][2 * h], o[k][2 * h + 1]);
      }
    }
    // the state's update: rows of b, decayed to the chunk's end, in two bf16 parts
    decay_state<NB>(z, lg, cnt - 1 + lead);
    const uint32_t t_row = (lane & 7) + ((lane >> 3) & 1) * 8, t_col = (lane >> 4) * 8;
#pragma unroll 2
    for (int k = 0; k < C / 16; ++k) {
      // b^T as the left operand: blocks (rows of Z, tokens) in the order of the fragment
      uint32_t bt[4], ah[4], al[4], ar[4];
      ldm4t(bt, s_u32(sb) + (k * 16 + (lane & 7) + (lane >> 4) * 8) * kPitch32 + (zr + ((lane >> 3) & 1) * 8) * 2);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int j = k * 16 + (h >> 1) * 8 + c0;
        const float x = lo_f(bt[h]) * w[j], y = hi_f(bt[h]) * w[j + 1];
        ah[h] = pack2(x, y);
        const float xr = x - lo_f(ah[h]), yr = y - hi_f(ah[h]);
        al[h] = pack2(xr, yr);
        ar[h] = pack2(xr - lo_f(al[h]), yr - hi_f(al[h]));
      }
#pragma unroll
      for (int i = 0; i < kCols32 / 16; ++i) {
        uint32_t cf[4];
        ldm4t(cf, s_u32(sc) + (k * 16 + t_row) * kPitch32 + (zc + i * 16 + t_col) * 2);
        mma16816(z[2 * i], ah, cf[0], cf[1]);
        mma16816(z[2 * i + 1], ah, cf[2], cf[3]);
        mma16816(z[2 * i], al, cf[0], cf[1]);
        mma16816(z[2 * i + 1], al, cf[2], cf[3]);
        if (P.zn != nullptr) {
          mma16816(z[2 * i], ar, cf[0], cf[1]);
          mma16816(z[2 * i + 1], ar, cf[2], cf[3]);
        }
      }
    }
  }
  float* dst = nullptr;
  float f = 1.f;
  if constexpr (kStateOnly) {
    dst = args.seg_state + sbase + (int64_t)seg * D * D;
  } else {
    // the segment that holds the last token (the first one of an empty sequence)
    const int last = n > 0 ? (n - 1) / args.seg_len : 0;
    if (P.zn != nullptr && seg == last) dst = P.zn + zbase;
    if (P.reverse && n > 0) f = exp2f(lg);
  }
  if (dst != nullptr)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(dst + (zr + r0 + 8 * h) * D + zc + i * 8 + c0) =
            make_float2(f * z[i][2 * h], f * z[i][2 * h + 1]);
}

// One token per sequence: state <- g state + k v^T, o = state^T q, the state read and written
// once.  A CTA per (sequence, head); a thread owns 4 columns of every kRows-th row.
template <int D>
__global__ void __launch_bounds__(256) decay_step_kernel(const bf16* __restrict__ q, const bf16* __restrict__ k,
                                                         const bf16* __restrict__ v, bf16* __restrict__ o,
                                                         float* __restrict__ state, const float* __restrict__ g,
                                                         int heads, int64_t ld) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes, kPer = D / kRows;
  __shared__ float4 part[kRows][kLanes];
  const int head = blockIdx.x % heads, batch = blockIdx.x / heads;
  const int c = threadIdx.x % kLanes, r = threadIdx.x / kLanes;
  float4* s = reinterpret_cast<float4*>(state + (int64_t)blockIdx.x * D * D) + c;
  float4 x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = s[(i * kRows + r) * kLanes];
  const int64_t at = (int64_t)batch * ld + head * D;
  const uint2 vw = *reinterpret_cast<const uint2*>(v + at + 4 * c);
  const float4 vv = make_float4(lo_f(vw.x), hi_f(vw.x), lo_f(vw.y), hi_f(vw.y));
  const float gg = g[head];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float kk = __bfloat162float(k[at + i * kRows + r]), qq = __bfloat162float(q[at + i * kRows + r]);
    x[i].x = fmaf(gg, x[i].x, kk * vv.x);
    x[i].y = fmaf(gg, x[i].y, kk * vv.y);
    x[i].z = fmaf(gg, x[i].z, kk * vv.z);
    x[i].w = fmaf(gg, x[i].w, kk * vv.w);
    s[(i * kRows + r) * kLanes] = x[i];
    acc.x = fmaf(qq, x[i].x, acc.x);
    acc.y = fmaf(qq, x[i].y, acc.y);
    acc.z = fmaf(qq, x[i].z, acc.z);
    acc.w = fmaf(qq, x[i].w, acc.w);
  }
  part[r][c] = acc;
  __syncthreads();
  if (threadIdx.x < kLanes) {
    float4 t = part[0][c];
#pragma unroll
    for (int i = 1; i < kRows; ++i) {
      const float4 p = part[i][c];
      t.x += p.x; t.y += p.y; t.z += p.z; t.w += p.w;
    }
    *reinterpret_cast<uint2*>(o + (int64_t)batch * heads * D + head * D + 4 * c) = make_uint2(pack2(t.x, t.y), pack2(t.z, t.w));
  }
}

// Segments per sequence: one when the sequences fill the GPU by themselves (each input is then
// read once), else enough of them, of four chunks or more, to give every SM work.
int la_segments(int T, int chunk, int seqs, int sms) {
  const int chunks = (T + chunk - 1) / chunk, want = (sms + seqs - 1) / seqs;
  const int most = chunks / 4 > 1 ? chunks / 4 : 1;
  return want < most ? want : most;
}

cudaError_t launch_passes32(LaArgs& a, int sms, cudaStream_t s) {
  const int seqs = a.B * a.heads, chunks = (a.T + kC32 - 1) / kC32;
  const int segs = la_segments(a.T, kC32, seqs * a.passes, sms);
  a.seg_len = (chunks + segs - 1) / segs * kC32;
  a.segs = (a.T + a.seg_len - 1) / a.seg_len;
  if (a.segs > 1) {
    decay_pass_kernel<true><<<dim3(a.segs - 1, seqs, a.passes), kWarps32 * 32, kSmem32, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  decay_pass_kernel<false><<<dim3(a.segs, seqs, a.passes), kWarps32 * 32, kSmem32, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace srnl

// ------------------------------------------------------------------ C ABI
struct srnl_lattn {
  srnl_lattn_config cfg{};
  int device = 0, sms = 0;
  int64_t ld = 0;
  float *log2g = nullptr, *g = nullptr;   // [heads]
  float* seg_state = nullptr;             // what the segments of long sequences add
  int* dev_err = nullptr;
  char err[256] = "";
};

namespace {

thread_local char g_lattn_create_error[256] = "";

srnl_status la_fail(srnl_lattn* h, srnl_status st, const char* msg) {
  snprintf(h != nullptr ? h->err : g_lattn_create_error, 256, "%s", msg);
  return st;
}

srnl_status la_cuda_fail(srnl_lattn* h, cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return la_fail(h, e == cudaErrorMemoryAllocation ? SRNL_E_NOMEM : SRNL_E_CUDA, msg);
}

void la_free(srnl_lattn* h) {
  void* ptrs[] = {h->log2g, h->g, h->seg_state, h->dev_err};
  for (void* p : ptrs)
    if (p != nullptr) cudaFree(p);
}

// A buffer of `rows` rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, width, pitch;
  const char* name;
};

// Whether two buffers share a byte.  Slices of one interleaved buffer (equal pitches) share a
// span of addresses but no byte unless their columns meet.
bool la_meet(const Rows& a, const Rows& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0) return false;
  const int64_t x = (int64_t)reinterpret_cast<uintptr_t>(a.p), y = (int64_t)reinterpret_cast<uintptr_t>(b.p);
  const int64_t ea = x + (a.rows - 1) * a.pitch + a.width, eb = y + (b.rows - 1) * b.pitch + b.width;
  if (x >= eb || y >= ea) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t d = (((y - x) % a.pitch) + a.pitch) % a.pitch;   // b's columns after a's
  return d < a.width || d + b.width > a.pitch;
}

srnl_status la_check(srnl_lattn* h, const Rows* in, int ni, const Rows* out, int no, const void* lengths) {
  char msg[256];
  for (int i = 0; i < ni + no; ++i) {
    const Rows& r = i < ni ? in[i] : out[i - ni];
    if (reinterpret_cast<uintptr_t>(r.p) & 15u) {
      snprintf(msg, sizeof msg, "%s must be 16-byte aligned", r.name);
      return la_fail(h, SRNL_E_INVAL, msg);
    }
  }
  if (reinterpret_cast<uintptr_t>(lengths) & 3u) return la_fail(h, SRNL_E_INVAL, "lengths must be 4-byte aligned");
  for (int i = 0; i < no; ++i)
    for (int j = 0; j < ni + i; ++j) {
      const Rows& r = j < ni ? in[j] : out[j - ni];
      if (la_meet(out[i], r)) {
        snprintf(msg, sizeof msg, "%s overlaps %s", out[i].name, r.name);
        return la_fail(h, SRNL_E_INVAL, msg);
      }
    }
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return la_cuda_fail(h, e, "cudaGetDevice");
  if (cur != h->device) return la_fail(h, SRNL_E_INVAL, "the current device is not the handle's device");
  return SRNL_OK;
}

cudaError_t la_run(srnl_lattn* h, srnl::LaArgs& a, cudaStream_t s) {
  a.B = h->cfg.B; a.T = h->cfg.T; a.heads = h->cfg.heads;
  a.log2g = h->log2g; a.seg_state = h->seg_state; a.err = h->dev_err;
  return h->cfg.d == 32 ? srnl::launch_passes32(a, h->sms, s) : srnl::launch_la_tc(a, h->cfg.d, h->sms, s);
}

}  // namespace

extern "C" {

srnl_status srnl_lattn_create(srnl_lattn** out, const srnl_lattn_config* cfg, const float* decay) {
  using namespace srnl;
  if (out == nullptr) return la_fail(nullptr, SRNL_E_INVAL, "out is NULL");
  *out = nullptr;
  if (cfg == nullptr || decay == nullptr) return la_fail(nullptr, SRNL_E_INVAL, "cfg or decay is NULL");
  if (cfg->B <= 0 || cfg->T <= 0 || cfg->heads <= 0 || cfg->d <= 0)
    return la_fail(nullptr, SRNL_E_INVAL, "B, T, heads and d must be positive");
  if (cfg->act_dtype != SRNL_BF16) return la_fail(nullptr, SRNL_E_UNSUPPORTED, "linear attention takes bf16 activations");
  if (cfg->d != 32 && cfg->d != 64 && cfg->d != 128) return la_fail(nullptr, SRNL_E_UNSUPPORTED, "d must be 32, 64 or 128");
  if ((int64_t)cfg->heads * cfg->d > (1 << 20)) return la_fail(nullptr, SRNL_E_UNSUPPORTED, "heads x d must be at most 2^20");
  if ((int64_t)cfg->B * cfg->heads > 65535) return la_fail(nullptr, SRNL_E_UNSUPPORTED, "B x heads must be at most 65535");
  if (cfg->T > (1 << 24)) return la_fail(nullptr, SRNL_E_UNSUPPORTED, "T must be at most 2^24");
  const int D = cfg->heads * cfg->d;
  if (cfg->ld != 0 && (cfg->ld < D || cfg->ld % 8 != 0))
    return la_fail(nullptr, SRNL_E_INVAL, "ld must be 0 or a multiple of 8, at least heads x d");
  for (int i = 0; i < cfg->heads; ++i)
    if (!(decay[i] > 0.f && decay[i] <= 1.f)) return la_fail(nullptr, SRNL_E_INVAL, "every decay must be in (0, 1]");
  srnl_lattn* h = new (std::nothrow) srnl_lattn;
  float* host = new (std::nothrow) float[cfg->heads];
  if (h == nullptr || host == nullptr) {
    delete h;
    delete[] host;
    return la_fail(nullptr, SRNL_E_NOMEM, "host allocation failed");
  }
  h->cfg = *cfg;
  h->ld = cfg->ld != 0 ? cfg->ld : D;
  for (int i = 0; i < cfg->heads; ++i) host[i] = (float)std::log2((double)decay[i]);
  const size_t nb = (size_t)cfg->heads * sizeof(float);
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) e = cudaMalloc(&h->log2g, nb);
  if (e == cudaSuccess) e = cudaMalloc(&h->g, nb);
  if (e == cudaSuccess) e = cudaMemcpy(h->log2g, host, nb, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(h->g, decay, nb, cudaMemcpyHostToDevice);
  delete[] host;
  if (e == cudaSuccess) {
    // the most any call splits: one pass (the forward) or three (the backward)
    size_t most = 0;
    for (int passes = 1; passes <= 3; passes += 2) {
      const int groups = (D + 127) / 128;
      const int segs = cfg->d == 32 ? la_segments(cfg->T, kC32, cfg->B * cfg->heads * passes, h->sms)
                                    : la_tc_segments(cfg->T, cfg->B * groups * passes, h->sms);
      const size_t n = segs > 1 ? (size_t)passes * cfg->B * cfg->heads * segs * cfg->d * cfg->d * sizeof(float) : 0;
      if (n > most) most = n;
    }
    if (most > 0) e = cudaMalloc(&h->seg_state, most);
  }
  if (e == cudaSuccess) e = cudaMalloc(&h->dev_err, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(h->dev_err, 0, sizeof(int));
  if (e == cudaSuccess && cfg->d != 32) e = prepare_la_tc(cfg->d);
  if (e != cudaSuccess) {
    const srnl_status st = la_cuda_fail(nullptr, e, "linear attention create");
    la_free(h);
    delete h;
    return st;
  }
  *out = h;
  return SRNL_OK;
}

srnl_status srnl_lattn_forward(srnl_lattn* h, const void* q, const void* k, const void* v, void* o, const int* lengths,
                               const float* state_in, float* state_out, void* stream) {
  using namespace srnl;
  if (h == nullptr) return la_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr) return la_fail(h, SRNL_E_INVAL, "q, k, v or o is NULL");
  const srnl_lattn_config& c = h->cfg;
  const int64_t n = (int64_t)c.B * c.T, D = (int64_t)c.heads * c.d, s = (int64_t)c.B * c.heads * c.d * c.d * 4;
  const Rows in[] = {{q, n, 2 * D, 2 * h->ld, "q"}, {k, n, 2 * D, 2 * h->ld, "k"}, {v, n, 2 * D, 2 * h->ld, "v"},
                     {state_in, 1, s, s, "state_in"}};
  const Rows out[] = {{o, n, 2 * D, 2 * D, "o"}, {state_out, 1, s, s, "state_out"}};
  const srnl_status st = la_check(h, in, 4, out, 2, lengths);
  if (st != SRNL_OK) return st;
  LaArgs a{};
  a.passes = 1;
  a.lengths = lengths;
  a.pass[0] = {static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<const bf16*>(v), static_cast<bf16*>(o),
               h->ld, h->ld, h->ld, D, state_in, state_out, 0, 0};
  const cudaError_t e = la_run(h, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SRNL_OK : la_cuda_fail(h, e, "linear attention launch");
}

srnl_status srnl_lattn_backward(srnl_lattn* h, const void* q, const void* k, const void* v, const void* d_o, void* dq,
                                void* dk, void* dv, const int* lengths, const float* state_in, const float* dstate_out,
                                float* dstate_in, void* stream) {
  using namespace srnl;
  if (h == nullptr) return la_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  if (q == nullptr || k == nullptr || v == nullptr || d_o == nullptr || dq == nullptr || dk == nullptr || dv == nullptr)
    return la_fail(h, SRNL_E_INVAL, "q, k, v, do, dq, dk or dv is NULL");
  const srnl_lattn_config& c = h->cfg;
  const int64_t n = (int64_t)c.B * c.T, D = (int64_t)c.heads * c.d, s = (int64_t)c.B * c.heads * c.d * c.d * 4, ld = h->ld;
  const Rows in[] = {{q, n, 2 * D, 2 * ld, "q"}, {k, n, 2 * D, 2 * ld, "k"}, {v, n, 2 * D, 2 * ld, "v"},
                     {d_o, n, 2 * D, 2 * D, "do"}, {state_in, 1, s, s, "state_in"}, {dstate_out, 1, s, s, "dstate_out"}};
  const Rows out[] = {{dq, n, 2 * D, 2 * ld, "dq"}, {dk, n, 2 * D, 2 * ld, "dk"}, {dv, n, 2 * D, 2 * ld, "dv"},
                      {dstate_in, 1, s, s, "dstate_in"}};
  const srnl_status st = la_check(h, in, 6, out, 4, lengths);
  if (st != SRNL_OK) return st;
  const bf16 *Q = static_cast<const bf16*>(q), *K = static_cast<const bf16*>(k), *V = static_cast<const bf16*>(v),
             *G = static_cast<const bf16*>(d_o);
  LaArgs a{};
  a.passes = 3;
  a.lengths = lengths;
  a.pass[0] = {G, V, K, static_cast<bf16*>(dq), D, ld, ld, ld, state_in, nullptr, 1, 0};
  a.pass[1] = {V, G, Q, static_cast<bf16*>(dk), ld, D, ld, ld, dstate_out, nullptr, 1, 1};
  a.pass[2] = {K, Q, G, static_cast<bf16*>(dv), ld, ld, D, ld, dstate_out, dstate_in, 0, 1};
  const cudaError_t e = la_run(h, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SRNL_OK : la_cuda_fail(h, e, "linear attention backward launch");
}

srnl_status srnl_lattn_step(srnl_lattn* h, const void* q, const void* k, const void* v, void* o, float* state, void* stream) {
  using namespace srnl;
  if (h == nullptr) return la_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || state == nullptr)
    return la_fail(h, SRNL_E_INVAL, "q, k, v, o or state is NULL");
  const srnl_lattn_config& c = h->cfg;
  const int64_t n = c.B, D = (int64_t)c.heads * c.d, s = (int64_t)c.B * c.heads * c.d * c.d * 4, ld = h->ld;
  const Rows in[] = {{q, n, 2 * D, 2 * ld, "q"}, {k, n, 2 * D, 2 * ld, "k"}, {v, n, 2 * D, 2 * ld, "v"}};
  const Rows out[] = {{o, n, 2 * D, 2 * D, "o"}, {state, 1, s, s, "state"}};
  const srnl_status st = la_check(h, in, 3, out, 2, nullptr);
  if (st != SRNL_OK) return st;
  const bf16 *Q = static_cast<const bf16*>(q), *K = static_cast<const bf16*>(k), *V = static_cast<const bf16*>(v);
  bf16* O = static_cast<bf16*>(o);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(c.B * c.heads);
  if (c.d == 32) decay_step_kernel<32><<<grid, 256, 0, cs>>>(Q, K, V, O, state, h->g, c.heads, ld);
  else if (c.d == 64) decay_step_kernel<64><<<grid, 256, 0, cs>>>(Q, K, V, O, state, h->g, c.heads, ld);
  else decay_step_kernel<128><<<grid, 256, 0, cs>>>(Q, K, V, O, state, h->g, c.heads, ld);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SRNL_OK : la_cuda_fail(h, e, "linear attention step launch");
}

srnl_status srnl_lattn_device_status(srnl_lattn* h) {
  if (h == nullptr) return la_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  int v = 0;
  const cudaError_t e = cudaMemcpy(&v, h->dev_err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return la_cuda_fail(h, e, "status read");
  return v == 0 ? SRNL_OK : la_fail(h, static_cast<srnl_status>(v), "a bounded in-kernel wait gave up");
}

const char* srnl_lattn_last_error(const srnl_lattn* h) { return h != nullptr ? h->err : g_lattn_create_error; }

void srnl_lattn_destroy(srnl_lattn* h) {
  if (h == nullptr) return;
  int prev = -1;
  if (cudaGetDevice(&prev) == cudaSuccess && prev != h->device) cudaSetDevice(h->device);
  cudaDeviceSynchronize();
  la_free(h);
  if (prev >= 0 && prev != h->device) cudaSetDevice(prev);
  delete h;
}

}  // extern "C"
