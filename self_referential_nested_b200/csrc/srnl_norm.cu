// Layer normalisation with its backward pass (sm_100a), for training the layers around the
// SRNL operator: the residual block's norm (srnl_block.cu) is forward-only.
//
//   forward   mean = sum(x) / D, rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),
//             y = (x - mean) rstd gamma + beta
//   backward  xhat = (x - mean) rstd, w = dy gamma,
//             dx = rstd (w - sum(w) / D - xhat sum(w xhat) / D) [+ dres],
//             dgamma = sum_rows dy xhat, dbeta = sum_rows dy
//
// Both passes are bound by memory: each input is read once and each output written once (backward of
// 8209 x 2560 fp32: 52 us, 4.9 TB/s; of 25088 x 384 bf16 with dres: 21 us, 3.6 TB/s; forward of 100352 x
// 64 bf16: 5.4 us, 4.9 TB/s, in L2), short calls by their launches.  All statistics, sums and
// gradients of gamma and beta are fp32; only y and dx are rounded, once, to the activations' type.
//
// Layout of the work: a row belongs to a group of lanes that hold it in registers between the
// sums and the output: 8 to 32 lanes of a warp for rows of up to 128 16-byte vectors, a block for
// longer ones (two blocks of a cluster for the longest fp32 rows backward).  A lane owns the same columns in every row it meets, so the weights' gradients
// stay in its registers until the end.  Several rows are taken at once where they are short, so
// that enough loads are in flight.  The arithmetic goes in pairs (two fp32 operations an
// instruction): at full bandwidth the issue slots, not the loads, come next.
//
// Rows that are not whole 16-byte vectors: a block's groups stride over the rows by a multiple of the
// vector's length, so all its rows start at the same offset within a vector.  Its lanes stay on
// aligned vectors, and the weights are copied to shared memory at that offset; the two vectors at a
// row's ends are shared with its neighbours.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <new>

#include "srnl_common.cuh"
#include "srnl_internal.h"
#include "srnl_norm.h"
#include "srnl_scan.h"

namespace srnl {
namespace {

constexpr int kNormMaxDim = 8192;
constexpr int kNormBlocks = 8;     // most blocks per SM, and partial sums of the weights' gradients

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 16 bytes of a row as fp32 pairs, and back.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& raw, float2* v) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
    v[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  }
}
template <typename T>
__device__ __forceinline__ uint4 repack(const float2* v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  }
}

// The 16-byte unit at column c of a row.  An odd row's units at its ends hold values of its
// neighbours too.  They are read whole and the neighbours' values taken out once they have arrived
// (clip): value by value a lane packs bf16 ones, and so waits for each unit in turn (8000 x 1533
// backward: 81 us, 41 whole).  fp32 ones need no packing, and blocks of long rows take them value by
// value (41 us whole, 38 so).  Nothing is read behind the buffer's end (room: values up to there).
template <typename T, int LPR, bool ODD>
__host__ __device__ constexpr bool whole_units() { return ODD && (sizeof(T) == 2 || LPR != 0); }

template <typename T, int LPR, bool ODD>
__device__ __forceinline__ uint4 load_cols(const T* row, int c, int dim, int room) {
  constexpr int V = 16 / sizeof(T);
  if (!ODD || unit_in_one_piece(c, V, dim, room, whole_units<T, LPR, ODD>())) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (c + e >= 0 && c + e < dim) {
      if constexpr (sizeof(T) == 2) w[e >> 1] |= (uint32_t)__bfloat16_as_ushort(row[c + e]) << (16 * (e & 1));
      else w[e] = __float_as_uint(row[c + e]);
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T, int LPR, bool ODD>
__device__ __forceinline__ uint4 clip(const uint4& raw, int c, int dim) {
  constexpr int V = 16 / sizeof(T);
  if (!whole_units<T, LPR, ODD>() || (c >= 0 && c + V <= dim)) return raw;
  uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (c + e < 0 || c + e >= dim) {
      if constexpr (sizeof(T) == 2) w[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
      else w[e] = 0u;
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// A bf16 unit at one of an odd row's ends goes in pieces of 8, 4 and 2 bytes, each where it is aligned:
// at the row's end from the unit's first value on, at its start up to the unit's last.
template <typename T, bool ODD>
__device__ __forceinline__ void store_cols(T* row, int c, int dim, const float2* v) {
  constexpr int V = 16 / sizeof(T);
  const uint4 raw = repack<T>(v);
  if (!ODD || (c >= 0 && c + V <= dim)) {
    *reinterpret_cast<uint4*>(row + c) = raw;
    return;
  }
  if (sizeof(T) == 2 && c >= 0) {
    const int n = dim - c;   // the first n
    if (n & 4) *reinterpret_cast<uint2*>(row + c) = make_uint2(raw.x, raw.y);
    if (n & 2) *reinterpret_cast<uint32_t*>(row + c + (n & 4)) = n & 4 ? raw.z : raw.x;
    if (n & 1) *reinterpret_cast<unsigned short*>(row + dim - 1) = (unsigned short)(n & 4 ? (n & 2 ? raw.w : raw.z) : n & 2 ? raw.y : raw.x);
  } else if (sizeof(T) == 2 && c + V <= dim) {
    const int n = c + V;     // the last n
    if (n & 4) *reinterpret_cast<uint2*>(row + n - 4) = make_uint2(raw.z, raw.w);
    if (n & 2) *reinterpret_cast<uint32_t*>(row + n - (n & 4) - 2) = n & 4 ? raw.y : raw.w;
    if (n & 1) *reinterpret_cast<unsigned short*>(row) = (unsigned short)((n & 4 ? (n & 2 ? raw.x : raw.y) : n & 2 ? raw.z : raw.w) >> 16);
  } else {                   // fp32, or a row within one unit
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e >= 0 && c + e < dim) {
        if constexpr (sizeof(T) == 2) row[c + e] = __ushort_as_bfloat16((unsigned short)(w[e >> 1] >> (16 * (e & 1))));
        else row[c + e] = __uint_as_float(w[e]);
      }
  }
}
// V weights, 16-byte aligned, as pairs.
template <int V>
__device__ __forceinline__ void load_weights(const float* p, float2* v) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float4 f = *reinterpret_cast<const float4*>(p + 4 * i);
    v[2 * i] = make_float2(f.x, f.y);
    v[2 * i + 1] = make_float2(f.z, f.w);
  }
}
// An odd row's weights come from a copy in shared memory that is shifted as the block's rows are:
// column c is at c + sh; zeros around them (2000 x 8191 bf16 forward: 46 us with the weights value by
// value, 27 so).
__host__ __device__ constexpr int shifted(int dim) { return (dim + 16) / 4 * 4 + 4; }
__device__ __forceinline__ void shift_weights(float* to, const float* p, int sh, int dim) {
#pragma unroll 4
  for (int i = 4 * threadIdx.x; i < dim; i += 4 * blockDim.x) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i + 4 <= dim) {
      v = *reinterpret_cast<const float4*>(p + i);
    } else {
      v.x = p[i];
      if (i + 1 < dim) v.y = p[i + 1];
      if (i + 2 < dim) v.z = p[i + 2];
    }
    to[sh + i] = v.x; to[sh + i + 1] = v.y; to[sh + i + 2] = v.z; to[sh + i + 3] = v.w;
  }
  const int end = sh + (dim + 3) / 4 * 4;
  if ((int)threadIdx.x < sh) to[threadIdx.x] = 0.f;
  if (end + (int)threadIdx.x < shifted(dim)) to[end + threadIdx.x] = 0.f;
}

__device__ __forceinline__ uint32_t cluster_block() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of N values over a row's lanes: LPR of a warp, or (LPR == 0) CL blocks, by way of red ([CL]
// [kMostWarps][N] in each; calls alternate between two of them, so that one barrier a call is enough).
constexpr int kLongWarps = 17, kMostWarps = 32;
template <int LPR, int CL, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float* red) {
#pragma unroll
  for (int o = (LPR == 0 ? 32 : LPR) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if constexpr (LPR == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if constexpr (CL == 1) {
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[warp * N + i] = s[i];
      __syncthreads();
    } else {
      // a warp's sums go to every block of the cluster
      if (lane < CL) {
        const uint32_t own = (uint32_t)__cvta_generic_to_shared(red + (cluster_block() * kMostWarps + warp) * N);
        uint32_t to;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(own), "r"(lane));
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * i), "f"(s[i]) : "memory");
      }
      cluster_barrier();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int k = 0; k < CL; ++k) s[i] += lane < warps ? red[(k * kMostWarps + lane) * N + i] : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  }
}

constexpr int kLongThreads = 32 * kLongWarps;   // 8192 columns and an odd start: 1025 bf16 vectors by two, 2049 fp32 ones by four
// Most threads of a block, and the blocks whose registers an SM has to hold: one fewer where a row's
// values and weights would not fit (20000 x 256 bf16: 7.0 us with three, 5.1 with two).
__host__ __device__ constexpr int norm_threads(int lpr, int per, int r, bool bwd) {
  return lpr == 0 ? (per > 1 ? kLongThreads : r > 1 ? 256 : 1024) : bwd ? 128 : 256;
}
__host__ __device__ constexpr int norm_resident(int lpr, int per, int r, int esize, bool odd, bool bwd) {
  return lpr == 0 ? (per > 1 ? (bwd ? 1 : 2) : r > 1 ? (bwd ? 2 : 4) : 1) 
         : bwd    ? (esize == 2 && per == 4 ? 3 : 4)
                  : (esize == 2 && per == 2 && r == 2) || (odd && r == 4) ? 2 : 3;
}

// LPR: lanes per row (0: CL blocks, a cluster); PER: vectors per lane; R: rows at once.
template <typename T, int LPR, int PER, int R, bool ODD, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(norm_threads(LPR, PER, R, false), norm_resident(LPR, PER, R, sizeof(T), ODD, false))
    norm_forward_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                        T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t rows,
                        int dim, float eps) {
  constexpr int V = 16 / sizeof(T), H = V / 2;
  if constexpr (CL > 1) cluster_barrier();   // its blocks are all there
  // gamma and beta in registers, else from L1 or shared memory for each R rows
  constexpr bool kKeep = LPR != 0 && PER * V <= 16;
  constexpr int kRed = CL * kMostWarps * R;
  __shared__ float red[LPR == 0 ? 2 * kRed : 1];
  const int lanes = LPR == 0 ? CL * blockDim.x : LPR;
  const int lane = LPR != 0 ? threadIdx.x % LPR : CL == 1 ? threadIdx.x : cluster_block() * blockDim.x + threadIdx.x;
  // the groups of a block are spread over the rows where those are odd: the grid is a multiple of a
  // vector's length then, and all of its rows start at the same offset
  const int64_t group = LPR == 0 ? blockIdx.x / CL
                        : ODD ? (int64_t)(threadIdx.x / (LPR ? LPR : 1)) * gridDim.x + blockIdx.x
                              : ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / (LPR ? LPR : 1);
  const int64_t groups = LPR == 0 ? gridDim.x / CL : (int64_t)gridDim.x * blockDim.x / LPR;
  // of the warp's first group: all lanes of a warp make the same passes
  const int64_t lead = LPR == 0 || LPR == 32 ? group : group - (int64_t)((threadIdx.x % 32) / (LPR ? LPR : 1)) * (ODD ? gridDim.x : 1);
  const int sh = ODD ? (int)(group * dim % V) : 0, c0 = lane * V - sh, cs = lanes * V;
  extern __shared__ __align__(16) float copies[];   // odd rows: gamma, beta
  const float *gp = gamma, *bp = beta;
  if constexpr (ODD) {
    shift_weights(copies, gamma, sh, dim);
    shift_weights(copies + shifted(dim), beta, sh, dim);
    __syncthreads();
    gp = copies + sh;
    bp = copies + shifted(dim) + sh;
  }
  const float inv_d = 1.f / (float)dim;
  bool on[PER];
  float2 g[kKeep ? PER * H : 1], b[kKeep ? PER * H : 1];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    on[i] = c0 + i * cs < dim && (!ODD || c0 + i * cs + V > 0);
    if constexpr (kKeep)
      if (on[i]) {
        load_weights<V>(gp + c0 + i * cs, g + i * H);
        load_weights<V>(bp + c0 + i * cs, b + i * H);
      }
  }
  uint4 raw[R][PER];
  auto load = [&](int64_t from) {
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        raw[q][i] = make_uint4(0u, 0u, 0u, 0u);
        const int64_t r = from + q * groups;
        if (on[i] && r < rows) raw[q][i] = load_cols<T, LPR, ODD>(x + r * dim, c0 + i * cs, dim, row_room(r, rows, dim));
      }
  };
  if (LPR == 0) load(group);
  for (int64_t r0 = group, base = lead; base < rows; r0 += groups * R, base += groups * R) {
    float2 v[R][PER * H];
    float s[R];
    if (LPR != 0) load(r0);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        unpack<T>(clip<T, LPR, ODD>(raw[q][i], c0 + i * cs, dim), v[q] + i * H);
#pragma unroll
        for (int e = 0; e < H; ++e) t = __fadd2_rn(t, v[q][i * H + e]);
      }
      s[q] = t.x + t.y;
    }
    if (LPR == 0) load(r0 + groups * R);   // a block waits on its barriers: the next rows are on their way meanwhile
    row_sum<LPR, CL, R>(s, red);
    float mean[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mean[q] = s[q] * inv_d;
      float2 t = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = c0 + i * cs;
        if (!on[i]) continue;
#pragma unroll
        for (int e = 0; e < H; ++e) {
          float2 d = __fadd2_rn(v[q][i * H + e], both(-mean[q]));
          if (ODD && (c < 0 || c + V > dim)) {
            if (c + 2 * e < 0 || c + 2 * e >= dim) d.x = 0.f;
            if (c + 2 * e + 1 < 0 || c + 2 * e + 1 >= dim) d.y = 0.f;
          }
          v[q][i * H + e] = d;
          t = __ffma2_rn(d, d, t);
        }
      }
      s[q] = t.x + t.y;
    }
    row_sum<LPR, CL, R>(s, red + (LPR == 0 ? kRed : 0));
#pragma unroll
    for (int q = 0; q < R; ++q) s[q] = rsqrtf(s[q] * inv_d + eps);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (!on[i]) continue;
      const int c = c0 + i * cs;
      float2 gw[H], bw[H];
      if constexpr (kKeep) {
#pragma unroll
        for (int e = 0; e < H; ++e) { gw[e] = g[i * H + e]; bw[e] = b[i * H + e]; }
      } else {
        load_weights<V>(gp + c, gw);
        load_weights<V>(bp + c, bw);
      }
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int64_t r = r0 + q * groups;
        if (r >= rows) continue;
        float2 o[H];
#pragma unroll
        for (int e = 0; e < H; ++e) o[e] = __ffma2_rn(__fmul2_rn(v[q][i * H + e], both(s[q])), gw[e], bw[e]);
        store_cols<T, ODD>(y + r * dim, c, dim, o);
      }
    }
    if (lane == 0) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int64_t r = r0 + q * groups;
        if (r < rows && mean_out != nullptr) mean_out[r] = mean[q];
        if (r < rows && rstd_out != nullptr) rstd_out[r] = s[q];
      }
    }
  }
  if constexpr (CL > 1) cluster_barrier();   // no block leaves while another may still write to it
}

// dx per row, and per block the partial sums of dgamma and dbeta: part[block][2][dim].
template <typename T, int LPR, int PER, int R, bool ODD, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(norm_threads(LPR, PER, R, true), norm_resident(LPR, PER, R, sizeof(T), ODD, true))
    norm_backward_kernel(const T* __restrict__ x, const T* __restrict__ dy, const T* __restrict__ dres,
                         const float* __restrict__ gamma, const float* __restrict__ mean_in,
                         const float* __restrict__ rstd_in, T* __restrict__ dx, float* __restrict__ part,
                         int64_t rows, int dim) {
  constexpr int V = 16 / sizeof(T), H = V / 2;
  if constexpr (CL > 1) cluster_barrier();   // its blocks are all there
  extern __shared__ __align__(16) float copies[];   // odd rows: gamma; then [warps][2][dim]: groups of different warps share columns
  float* fold = copies + (ODD ? shifted(dim) : 0);
  constexpr int kRed = CL * kMostWarps * 2 * R;
  __shared__ float red[LPR == 0 ? 2 * kRed : 1];
  const int lanes = LPR == 0 ? CL * blockDim.x : LPR;
  const int lane = LPR != 0 ? threadIdx.x % LPR : CL == 1 ? threadIdx.x : cluster_block() * blockDim.x + threadIdx.x;
  // the groups of a block are spread over the rows where those are odd: the grid is a multiple of a
  // vector's length then, and all of its rows start at the same offset
  const int64_t group = LPR == 0 ? blockIdx.x / CL
                        : ODD ? (int64_t)(threadIdx.x / (LPR ? LPR : 1)) * gridDim.x + blockIdx.x
                              : ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / (LPR ? LPR : 1);
  const int64_t groups = LPR == 0 ? gridDim.x / CL : (int64_t)gridDim.x * blockDim.x / LPR;
  const int64_t lead = LPR == 0 || LPR == 32 ? group : group - (int64_t)((threadIdx.x % 32) / (LPR ? LPR : 1)) * (ODD ? gridDim.x : 1);
  const int sh = ODD ? (int)(group * dim % V) : 0, c0 = lane * V - sh, cs = lanes * V;
  const float* gp = gamma;
  if constexpr (ODD) {
    shift_weights(copies, gamma, sh, dim);
    __syncthreads();
    gp = copies + sh;
  }
  const float inv_d = 1.f / (float)dim;
  bool on[PER];
  constexpr bool kKeep = LPR != 0 && PER * V <= 16;
  float2 dg[PER * H], db[PER * H], g[kKeep ? PER * H : 1];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    on[i] = c0 + i * cs < dim && (!ODD || c0 + i * cs + V > 0);
    if constexpr (kKeep)
      if (on[i]) load_weights<V>(gp + c0 + i * cs, g + i * H);
#pragma unroll
    for (int e = 0; e < H; ++e) dg[i * H + e] = db[i * H + e] = make_float2(0.f, 0.f);
  }
  int flip = 0;
  uint4 xr[R][PER], yr[R][PER], er[R][PER];
  float mean[R], rstd[R];
  auto load = [&](int64_t from) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t r = from + q * groups;
      mean[q] = r < rows ? mean_in[r] : 0.f;
      rstd[q] = r < rows ? rstd_in[r] : 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        xr[q][i] = yr[q][i] = er[q][i] = make_uint4(0u, 0u, 0u, 0u);
        if (on[i] && r < rows) {
          xr[q][i] = load_cols<T, LPR, ODD>(x + r * dim, c0 + i * cs, dim, row_room(r, rows, dim));
          yr[q][i] = load_cols<T, LPR, ODD>(dy + r * dim, c0 + i * cs, dim, row_room(r, rows, dim));
          if (dres != nullptr) er[q][i] = load_cols<T, LPR, ODD>(dres + r * dim, c0 + i * cs, dim, row_room(r, rows, dim));
        }
      }
    }
  };
  // Between a block's barriers its next rows are on their way; not with two bf16 vectors a lane,
  // whose sums leave no registers for it.
  constexpr bool kAhead = LPR == 0 && PER * V < 16;
  if (kAhead) load(group);
  for (int64_t r0 = group, base = lead; base < rows; r0 += groups * R, base += groups * R, flip ^= 1) {
    float s[2 * R], f[R];
    uint4 res[R][PER];
    if (!kAhead) load(r0);
    // w carries rstd from the start.  Values past a row's ends are zeros in x and dy and add nothing to any sum:
    // w (x - mean) is zero there even where the row lies so far from zero that mean rstd, and xhat, are infinite.
    float2 xh[R][PER * H], w[R][PER * H];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 t = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float2 xv[H], yv[H], gw[H];
        unpack<T>(clip<T, LPR, ODD>(xr[q][i], c0 + i * cs, dim), xv);
        unpack<T>(clip<T, LPR, ODD>(yr[q][i], c0 + i * cs, dim), yv);
        if (!on[i]) {
#pragma unroll
          for (int e = 0; e < H; ++e) gw[e] = make_float2(0.f, 0.f);
        } else if constexpr (kKeep) {
#pragma unroll
          for (int e = 0; e < H; ++e) gw[e] = g[i * H + e];
        } else {
          load_weights<V>(gp + c0 + i * cs, gw);
        }
#pragma unroll
        for (int e = 0; e < H; ++e) {
          const int k = i * H + e;
          const float2 d = __fadd2_rn(xv[e], both(-mean[q]));
          xh[q][k] = __fmul2_rn(d, both(rstd[q]));
          dg[k] = __ffma2_rn(yv[e], xh[q][k], dg[k]);
          db[k] = __fadd2_rn(db[k], yv[e]);
          w[q][k] = __fmul2_rn(__fmul2_rn(yv[e], gw[e]), both(rstd[q]));
          t = __fadd2_rn(t, w[q][k]);
          u = __ffma2_rn(w[q][k], d, u);
        }
      }
      s[2 * q] = t.x + t.y;
      s[2 * q + 1] = u.x + u.y;
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      f[q] = rstd[q];
#pragma unroll
      for (int i = 0; i < PER; ++i) res[q][i] = er[q][i];
    }
    if (kAhead) load(r0 + groups * R);
    row_sum<LPR, CL, 2 * R>(s, red + (LPR == 0 ? kRed * flip : 0));
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t r = r0 + q * groups;
      if (r >= rows) continue;
      const float2 a = both(-s[2 * q] * inv_d), m = both(-s[2 * q + 1] * inv_d * f[q]);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!on[i]) continue;
        float2 o[H];
        unpack<T>(res[q][i], o);
#pragma unroll
        for (int e = 0; e < H; ++e) o[e] = __fadd2_rn(__ffma2_rn(xh[q][i * H + e], m, __fadd2_rn(w[q][i * H + e], a)), o[e]);
        store_cols<T, ODD>(dx + r * dim, c0 + i * cs, dim, o);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;");
  if constexpr (CL > 1) cluster_barrier();   // no block leaves while another may still write to it
  // groups in one order: those of a warp, then the warps
  float* mine = part + (int64_t)(blockIdx.x / CL) * 2 * dim;
  auto put = [&](float* to) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = c0 + i * cs + e, k = i * H + e / 2;
        if (!on[i] || c >= dim || (ODD && c < 0)) continue;
        const float p = e & 1 ? dg[k].y : dg[k].x, q = e & 1 ? db[k].y : db[k].x;
        to[c] = p;
        to[dim + c] = q;
      }
  };
  if constexpr (LPR == 0) {
    put(mine);
  } else {
    const int warp = threadIdx.x >> 5;
    float* to = fold + warp * 2 * dim;
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < PER * H; ++k) {
        dg[k].x += __shfl_xor_sync(0xffffffffu, dg[k].x, o);
        dg[k].y += __shfl_xor_sync(0xffffffffu, dg[k].y, o);
        db[k].x += __shfl_xor_sync(0xffffffffu, db[k].x, o);
        db[k].y += __shfl_xor_sync(0xffffffffu, db[k].y, o);
      }
    if ((threadIdx.x & 31) < LPR) put(to);
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * dim; c += blockDim.x) {
      float t = 0.f;
      for (int k = 0; k < (int)(blockDim.x >> 5); ++k) t += fold[k * 2 * dim + c];
      mine[c] = t;
    }
  }
}

// dgamma[c] = sum_b part[b][0][c], dbeta[c] = sum_b part[b][1][c]: 32 columns per block, the
// blocks' partials split over 32 warps and folded in a fixed order.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* __restrict__ part, int blocks, int dim,
                                                                float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;   // column of [2][dim]
  float s = 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the rows' kernel still runs
  if (c < 2 * dim) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) s += part[(int64_t)b * 2 * dim + c];
  }
  sm[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += sm[k][lane];
    if (c < dim) {
      if (dgamma != nullptr) dgamma[c] = t;
    } else if (c < 2 * dim) {
      if (dbeta != nullptr) dbeta[c - dim] = t;
    }
  }
}

// The lanes a row length takes.
struct NormPlan {
  int lpr, per, threads;   // threads of a block (lpr == 0)
  int blocks;              // blocks a row (lpr == 0)
  bool odd;                // rows that are not whole 16-byte vectors
};

NormPlan norm_plan(int dim, int esize, bool bwd) {
  NormPlan p{};
  const int V = 16 / esize;
  p.odd = dim % V != 0;
  const int n = (dim + (p.odd ? V - 1 : 0) + V - 1) / V;   // vectors a row may touch
  if (n <= 8) { p.lpr = 8; p.per = 1; }
  else if (n <= 16) { p.lpr = 16; p.per = 1; }
  else if (n <= 32) { p.lpr = 16; p.per = 2; }
  else if (n <= 48) { p.lpr = 16; p.per = 3; }
  else if (n <= 64) { p.lpr = 32; p.per = 2; }
  else if (n <= 96) { p.lpr = 32; p.per = 3; }
  else if (n <= 128) { p.lpr = 32; p.per = 4; }
  else {
    p.lpr = 0;
    // The backward pass keeps its sums in registers.  fp32: a second block for the longest rows,
    // where four vectors a lane would not fit (2000 x 8192: 90 us in one block, 71 in two; forward
    // it would cost: 25 and 46).  bf16: a vector a lane, so that the next row's loads fit (2000 x
    // 8192: 49 us with two, 41 with one), but for odd rows, which may touch 1025 of them.
    p.blocks = bwd && esize == 4 && n > 2 * kLongThreads ? 2 : 1;
    p.per = n <= 256 || (bwd && esize == 2 && !p.odd) ? 1 : n <= 2 * kLongThreads * p.blocks ? 2 : 4;
    p.threads = ((n + p.per * p.blocks - 1) / (p.per * p.blocks) + 31) / 32 * 32;
  }
  return p;
}

// Blocks of a call: what the SMs hold at once, or fewer for few rows; a multiple of 8 (a vector's
// values) for odd rows, whose groups rely on it.
int norm_blocks(const NormPlan& p, int threads, int64_t rows, int sms, int per_sm) {
  const int per_block = p.lpr == 0 ? 1 : threads / p.lpr, each = p.lpr == 0 ? p.blocks : 1;
  const int64_t need = (rows + per_block - 1) / per_block, most = (int64_t)sms * per_sm / each;
  int n = (int)(need < most ? need : most);
  if (p.odd) n = n < 8 || (n + 7) / 8 * 8 <= most ? (n + 7) / 8 * 8 : n / 8 * 8;   // never a few more than fit at once
  return n * each;
}

// Shared memory of a block: an odd row's weights; backward, the warps' sums.
size_t norm_smem(const NormPlan& p, int dim, int threads, bool bwd) {
  return ((p.odd ? (size_t)shifted(dim) * (bwd ? 1 : 2) : 0) + (bwd && p.lpr != 0 ? (size_t)(threads / 32) * 2 * dim : 0)) * sizeof(float);
}

// Short rows go several at a time, so that a lane has two to four vectors in flight.
#define SRNL_NORM_PLAN(T, ODD, FWD, CALL)                                  \
  do {                                                                     \
    if (p.lpr == 8) { CALL(T, 8, 1, (FWD ? 4 : 2), ODD, 1); }                 \
    else if (p.lpr == 16 && p.per == 1) { CALL(T, 16, 1, (FWD ? 4 : 2), ODD, 1); } \
    else if (p.lpr == 16 && p.per == 2) { CALL(T, 16, 2, (FWD ? 2 : 1), ODD, 1); } \
    else if (p.lpr == 16) { CALL(T, 16, 3, 1, ODD, 1); }                      \
    else if (p.lpr == 32 && p.per == 2) { CALL(T, 32, 2, (FWD ? 2 : 1), ODD, 1); } \
    else if (p.lpr == 32 && p.per == 3) { CALL(T, 32, 3, 1, ODD, 1); }        \
    else if (p.lpr == 32) { CALL(T, 32, 4, 1, ODD, 1); }                      \
    else if (p.per == 1 && p.threads <= 256) { CALL(T, 0, 1, 2, ODD, 1); }  \
    else if (p.per == 1) { CALL(T, 0, 1, (FWD || sizeof(T) == 4 ? 2 : 1), ODD, 1); } \
    else if (p.per == 2 && p.blocks == 1) { CALL(T, 0, 2, 1, ODD, 1); }    \
    else if (sizeof(T) == 4) { CALL(T, 0, (sizeof(T) == 4 && FWD ? 4 : 2), 1, ODD, (sizeof(T) == 4 && !FWD ? 2 : 1)); } \
  } while (0)
#define SRNL_NORM_DISPATCH(FWD, CALL)                                      \
  do {                                                                     \
    if (bf16 && p.odd) SRNL_NORM_PLAN(__nv_bfloat16, true, FWD, CALL);     \
    else if (bf16) SRNL_NORM_PLAN(__nv_bfloat16, false, FWD, CALL);        \
    else if (p.odd) SRNL_NORM_PLAN(float, true, FWD, CALL);                \
    else SRNL_NORM_PLAN(float, false, FWD, CALL);                          \
  } while (0)

}  // namespace
}  // namespace srnl

// ------------------------------------------------------------------ C ABI
struct srnl_ln {
  srnl_ln_config cfg{};
  int device = 0, sms = 0;
  srnl::NormPlan fwd{}, bwd{};
  int fwd_per_sm = 1, bwd_per_sm = 1;   // blocks an SM holds
  float* part = nullptr;                // [bwd_per_sm * sms + 8][2][dim]
  char err[256] = "";
};

namespace {

thread_local char g_ln_create_error[256] = "";

srnl_status ln_fail(srnl_ln* h, srnl_status st, const char* msg) {
  snprintf(h != nullptr ? h->err : g_ln_create_error, 256, "%s", msg);
  return st;
}

srnl_status ln_cuda_fail(srnl_ln* h, cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return ln_fail(h, e == cudaErrorMemoryAllocation ? SRNL_E_NOMEM : SRNL_E_CUDA, msg);
}

bool ln_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool ln_overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

srnl_status ln_device(srnl_ln* h) {
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return ln_cuda_fail(h, e, "cudaGetDevice");
  if (cur != h->device) return ln_fail(h, SRNL_E_INVAL, "the current device is not the handle's device");
  return SRNL_OK;
}

}  // namespace

extern "C" {

srnl_status srnl_ln_create(srnl_ln** out, const srnl_ln_config* cfg) {
  if (out == nullptr) return ln_fail(nullptr, SRNL_E_INVAL, "out is NULL");
  *out = nullptr;
  if (cfg == nullptr) return ln_fail(nullptr, SRNL_E_INVAL, "cfg is NULL");
  if (cfg->dim <= 0) return ln_fail(nullptr, SRNL_E_INVAL, "dim must be positive");
  if (!(cfg->eps > 0.f) || std::isinf(cfg->eps)) return ln_fail(nullptr, SRNL_E_INVAL, "eps must be positive and finite");
  if (cfg->act_dtype != SRNL_F32 && cfg->act_dtype != SRNL_BF16)
    return ln_fail(nullptr, SRNL_E_INVAL, "act_dtype must be SRNL_F32 or SRNL_BF16");
  if (cfg->dim > srnl::kNormMaxDim) return ln_fail(nullptr, SRNL_E_UNSUPPORTED, "dim must be at most 8192");
  srnl_ln* h = new (std::nothrow) srnl_ln;
  if (h == nullptr) return ln_fail(nullptr, SRNL_E_NOMEM, "host allocation failed");
  h->cfg = *cfg;
  h->fwd = srnl::norm_plan(cfg->dim, cfg->act_dtype == SRNL_BF16 ? 2 : 4, false);
  h->bwd = srnl::norm_plan(cfg->dim, cfg->act_dtype == SRNL_BF16 ? 2 : 4, true);
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) {
    const bool bf16 = cfg->act_dtype == SRNL_BF16;
    {
      const srnl::NormPlan& p = h->fwd;
      const int threads = p.lpr == 0 ? p.threads : 256;
      const size_t smem = srnl::norm_smem(p, cfg->dim, threads, false);
// the limit is the kernel's, not the handle's, and counts its static shared memory too: raised to the
// longest row's for every odd row of a block's own
#define SRNL_NORM_OCC(T, LPR, PER, R, ODD, CL)                                                                              \
  if (p.odd && p.lpr == 0)                                                                                                  \
    e = cudaFuncSetAttribute(srnl::norm_forward_kernel<T, LPR, PER, R, ODD, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                             (int)(2 * srnl::shifted(srnl::kNormMaxDim) * sizeof(float)));                                  \
  if (e == cudaSuccess)                                                                                                     \
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&h->fwd_per_sm, srnl::norm_forward_kernel<T, LPR, PER, R, ODD, CL>,     \
                                                    threads, smem)
      SRNL_NORM_DISPATCH(true, SRNL_NORM_OCC);
#undef SRNL_NORM_OCC
    }
    if (e == cudaSuccess) {
      const srnl::NormPlan& p = h->bwd;
      const int threads = p.lpr == 0 ? p.threads : 128;
      const size_t smem = srnl::norm_smem(p, cfg->dim, threads, true);
#define SRNL_NORM_OCC(T, LPR, PER, R, ODD, CL)                                                                              \
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&h->bwd_per_sm, srnl::norm_backward_kernel<T, LPR, PER, R, ODD, CL>,    \
                                                    threads, smem)   /* at most 37 KB */
      SRNL_NORM_DISPATCH(false, SRNL_NORM_OCC);
#undef SRNL_NORM_OCC
    }
    if (e == cudaSuccess && (h->fwd_per_sm < 1 || h->bwd_per_sm < 1)) e = cudaErrorLaunchOutOfResources;
    if (h->bwd_per_sm > srnl::kNormBlocks) h->bwd_per_sm = srnl::kNormBlocks;
  }
  if (e == cudaSuccess)
    e = cudaMalloc(&h->part, ((size_t)h->sms * h->bwd_per_sm + 8) * 2 * cfg->dim * sizeof(float));
  if (e != cudaSuccess) {
    const srnl_status st = ln_cuda_fail(nullptr, e, "layer norm create");
    delete h;
    return st;
  }
  *out = h;
  return SRNL_OK;
}

srnl_status srnl_ln_forward(srnl_ln* h, const void* x, const float* gamma, const float* beta, void* y, float* mean,
                            float* rstd, int64_t rows, void* stream) {
  if (h == nullptr) return ln_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  if (rows < 0) return ln_fail(h, SRNL_E_INVAL, "rows must be >= 0");
  if (rows == 0) return SRNL_OK;
  if (x == nullptr || y == nullptr || gamma == nullptr || beta == nullptr)
    return ln_fail(h, SRNL_E_INVAL, "x, y, gamma or beta is NULL");
  if (!ln_aligned(x, 16) || !ln_aligned(y, 16) || !ln_aligned(gamma, 16) || !ln_aligned(beta, 16))
    return ln_fail(h, SRNL_E_INVAL, "x, y, gamma and beta must be 16-byte aligned");
  if (!ln_aligned(mean, 4) || !ln_aligned(rstd, 4)) return ln_fail(h, SRNL_E_INVAL, "mean and rstd must be 4-byte aligned");
  const bool bf16 = h->cfg.act_dtype == SRNL_BF16;
  const int dim = h->cfg.dim;
  const size_t n = (size_t)rows * dim * (bf16 ? 2 : 4), nr = (size_t)rows * 4, nd = (size_t)dim * 4;
  const struct { const void* p; size_t n; } ins[] = {{x, n}, {gamma, nd}, {beta, nd}}, outs[] = {{y, n}, {mean, nr}, {rstd, nr}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& in : ins)
      if (ln_overlap(in.p, in.n, outs[i].p, outs[i].n)) return ln_fail(h, SRNL_E_INVAL, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (ln_overlap(outs[j].p, outs[j].n, outs[i].p, outs[i].n)) return ln_fail(h, SRNL_E_INVAL, "two outputs overlap");
  }
  const srnl_status st = ln_device(h);
  if (st != SRNL_OK) return st;
  const srnl::NormPlan& p = h->fwd;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int threads = p.lpr == 0 ? p.threads : 256, blocks = srnl::norm_blocks(p, threads, rows, h->sms, h->fwd_per_sm);
#define SRNL_NORM_RUN(T, LPR, PER, R, ODD, CL)                                                      \
  srnl::norm_forward_kernel<T, LPR, PER, R, ODD, CL><<<blocks, threads, srnl::norm_smem(p, dim, threads, false), s>>>( \
      static_cast<const T*>(x), gamma, beta, static_cast<T*>(y), mean, rstd, rows, dim, h->cfg.eps)
  SRNL_NORM_DISPATCH(true, SRNL_NORM_RUN);
#undef SRNL_NORM_RUN
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SRNL_OK : ln_cuda_fail(h, e, "layer norm launch");
}

srnl_status srnl_ln_backward(srnl_ln* h, const void* x, const void* dy, const void* dres, const float* gamma,
                             const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta,
                             int64_t rows, void* stream) {
  if (h == nullptr) return ln_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  if (rows < 0) return ln_fail(h, SRNL_E_INVAL, "rows must be >= 0");
  if (rows > 0 && (x == nullptr || dy == nullptr || dx == nullptr || gamma == nullptr || mean == nullptr || rstd == nullptr))
    return ln_fail(h, SRNL_E_INVAL, "x, dy, dx, gamma, mean or rstd is NULL");
  if (!ln_aligned(x, 16) || !ln_aligned(dy, 16) || !ln_aligned(dres, 16) || !ln_aligned(dx, 16) || !ln_aligned(gamma, 16))
    return ln_fail(h, SRNL_E_INVAL, "x, dy, dres, dx and gamma must be 16-byte aligned");
  if (!ln_aligned(mean, 4) || !ln_aligned(rstd, 4) || !ln_aligned(dgamma, 4) || !ln_aligned(dbeta, 4))
    return ln_fail(h, SRNL_E_INVAL, "mean, rstd, dgamma and dbeta must be 4-byte aligned");
  const bool bf16 = h->cfg.act_dtype == SRNL_BF16;
  const int dim = h->cfg.dim;
  const size_t n = (size_t)rows * dim * (bf16 ? 2 : 4), nr = (size_t)rows * 4, nd = (size_t)dim * 4;
  const struct { const void* p; size_t n; } ins[] = {{x, n}, {dy, n}, {dres, n}, {gamma, nd}, {mean, nr}, {rstd, nr}},
                                             outs[] = {{dx, n}, {dgamma, nd}, {dbeta, nd}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& in : ins)
      if (ln_overlap(in.p, in.n, outs[i].p, outs[i].n)) return ln_fail(h, SRNL_E_INVAL, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (ln_overlap(outs[j].p, outs[j].n, outs[i].p, outs[i].n)) return ln_fail(h, SRNL_E_INVAL, "two outputs overlap");
  }
  const srnl_status st = ln_device(h);
  if (st != SRNL_OK) return st;
  const srnl::NormPlan& p = h->bwd;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int threads = p.lpr == 0 ? p.threads : 128, blocks = srnl::norm_blocks(p, threads, rows, h->sms, h->bwd_per_sm);
  if (rows > 0) {
    const size_t smem = srnl::norm_smem(p, dim, threads, true);
#define SRNL_NORM_RUN(T, LPR, PER, R, ODD, CL)                                                                     \
  srnl::norm_backward_kernel<T, LPR, PER, R, ODD, CL><<<blocks, threads, smem, s>>>(                               \
      static_cast<const T*>(x), static_cast<const T*>(dy), static_cast<const T*>(dres), gamma, mean, rstd,     \
      static_cast<T*>(dx), h->part, rows, dim)
    SRNL_NORM_DISPATCH(false, SRNL_NORM_RUN);
#undef SRNL_NORM_RUN
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return ln_cuda_fail(h, e, "layer norm backward launch");
  }
  if (dgamma != nullptr || dbeta != nullptr) {
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)((2 * dim + 31) / 32));
    lc.blockDim = dim3(1024);
    lc.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = &at;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, srnl::norm_weight_grad_kernel, static_cast<const float*>(h->part),
                                             p.lpr == 0 ? blocks / p.blocks : blocks,
                                             dim, dgamma, dbeta);
    if (e != cudaSuccess) return ln_cuda_fail(h, e, "layer norm weight gradient launch");
  }
  return SRNL_OK;
}

const char* srnl_ln_last_error(const srnl_ln* h) { return h != nullptr ? h->err : g_ln_create_error; }

void srnl_ln_destroy(srnl_ln* h) {
  if (h == nullptr) return;
  int prev = -1;
  if (cudaGetDevice(&prev) == cudaSuccess && prev != h->device) cudaSetDevice(h->device);
  cudaDeviceSynchronize();
  if (h->part != nullptr) cudaFree(h->part);
  if (prev >= 0 && prev != h->device) cudaSetDevice(prev);
  delete h;
}

}  // extern "C"
