// Layer normalisation with its backward pass (sm_100a), for training the layers around the
// SRNL operator: the residual block's norm (srnl_block.cu) is forward-only.
//
//   forward   mean = sum(x) / D, rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),
//             y = (x - mean) rstd gamma + beta
//   backward  xhat = (x - mean) rstd, w = dy gamma,
//             dx = rstd (w - sum(w) / D - xhat sum(w xhat) / D) [+ dres],
//             dgamma = sum_rows dy xhat, dbeta = sum_rows dy
//
// Both passes are bound by memory: each input row is read once into registers and each output
// row written once.  All statistics, sums and gradients of gamma and beta are fp32; only y and
// dx are rounded, once, to the activations' type.
//
// Layout of the work: a row belongs to a group of lanes.  Rows of up to 128 16-byte vectors
// take 8, 16 or 32 lanes of a warp (a 64-channel bf16 row is 8 vectors: a whole warp on it
// would leave 24 lanes idle), longer rows a block.  Groups walk the rows with the stride of
// the grid and load their next row before they reduce the present one, so gamma and beta stay
// in registers and a load is always in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <new>

#include "srnl_common.cuh"
#include "srnl_internal.h"
#include "srnl_scan.h"

namespace srnl {
namespace {

constexpr int kNormMaxDim = 8192;
constexpr int kNormWaves = 4;      // partial sums of the weights' gradients: at most this many blocks per SM

// V consecutive values of a row, as fp32.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float* v) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(*p);
    else v[0] = *p;
  } else if constexpr (sizeof(T) == 2) {
    const uint4 raw = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(v[0]);
    else *p = v[0];
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// Sums over a row's group: LPR lanes of a warp, or (LPR == 0) the whole block.
template <int LPR, int N>
__device__ __forceinline__ void group_sum(float (&s)[N], float* red) {
  constexpr int W = LPR == 0 ? 32 : LPR;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if constexpr (LPR == 0) {   // red: two alternating halves of [warps][N], so one barrier per sum is enough
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[warp * N + i] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = lane < nw ? red[lane * N + i] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  }
}

// T: activations' type; V: values per load; LPR: lanes per row (0: a block per row); PER:
// loads per lane and row.
template <typename T, int V, int LPR, int PER>
__global__ void __launch_bounds__(LPR == 0 ? 512 : 256)
    norm_forward_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                        T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t rows,
                        int dim, float eps) {
  constexpr int N = PER * V;
  __shared__ float red[LPR == 0 ? 32 : 1];
  const int lanes = LPR == 0 ? blockDim.x : LPR;
  const int lane = LPR == 0 ? threadIdx.x : threadIdx.x % LPR;
  const int64_t first = LPR == 0 ? blockIdx.x : ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / LPR;
  const int64_t step = LPR == 0 ? gridDim.x : (int64_t)gridDim.x * blockDim.x / LPR;
  const float inv_d = 1.f / (float)dim;
  float g[N], b[N], v[N];
  bool on[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * lanes + lane) * V;
    on[i] = c < dim;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      g[i * V + e] = on[i] ? gamma[c + e] : 0.f;
      b[i * V + e] = on[i] ? beta[c + e] : 0.f;
      v[i * V + e] = 0.f;
    }
    if (on[i] && first < rows) load_vec<T, V>(x + first * dim + c, v + i * V);
  }
  // Every lane of a warp makes the same number of passes, so the warp's shuffles stay whole:
  // the bound is that of the warp's first row.
  const int64_t lead = LPR == 0 || LPR == 32 ? first : first - (threadIdx.x % 32) / LPR;
  int64_t r = first;
  for (int64_t base = lead; base < rows; base += step, r += step) {
    float nx[N];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) nx[i * V + e] = 0.f;
      if (on[i] && r + step < rows) load_vec<T, V>(x + (r + step) * dim + (i * lanes + lane) * V, nx + i * V);
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < N; ++i) s[0] += v[i];
    group_sum<LPR, 1>(s, red);
    const float mean = s[0] * inv_d;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = on[i] ? v[i * V + e] - mean : 0.f;
        q[0] = fmaf(c, c, q[0]);
      }
    group_sum<LPR, 1>(q, red + (LPR == 0 ? 16 : 0));
    const float rstd = rsqrtf(q[0] * inv_d + eps);
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!on[i]) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf((v[i * V + e] - mean) * rstd, g[i * V + e], b[i * V + e]);
        store_vec<T, V>(y + r * dim + (i * lanes + lane) * V, o);
      }
      if (lane == 0) {
        if (mean_out != nullptr) mean_out[r] = mean;
        if (rstd_out != nullptr) rstd_out[r] = rstd;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = nx[i];
  }
}

// dx per row, and per block the partial sums of dgamma and dbeta: part[block][2][dim].  A lane
// owns the same columns in every row it meets, so its sums stay in registers until the end.
template <typename T, int V, int LPR, int PER>
__global__ void __launch_bounds__(LPR == 0 ? 512 : 256)
    norm_backward_kernel(const T* __restrict__ x, const T* __restrict__ dy, const T* __restrict__ dres,
                         const float* __restrict__ gamma, const float* __restrict__ mean_in,
                         const float* __restrict__ rstd_in, T* __restrict__ dx, float* __restrict__ part,
                         int64_t rows, int dim) {
  constexpr int N = PER * V;
  extern __shared__ float fold[];   // warps sharing columns: [2][dim]
  __shared__ float red[LPR == 0 ? 64 : 1];
  const int lanes = LPR == 0 ? blockDim.x : LPR;
  const int lane = LPR == 0 ? threadIdx.x : threadIdx.x % LPR;
  const int64_t first = LPR == 0 ? blockIdx.x : ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / LPR;
  const int64_t step = LPR == 0 ? gridDim.x : (int64_t)gridDim.x * blockDim.x / LPR;
  const float inv_d = 1.f / (float)dim;
  float dg[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = db[i] = 0.f;
  const int64_t lead = LPR == 0 || LPR == 32 ? first : first - (threadIdx.x % 32) / LPR;
  int64_t r = first;
  int flip = 0;
  for (int64_t base = lead; base < rows; base += step, r += step) {
    float xh[N], w[N];
    const bool live = r < rows;
    const float mean = live ? mean_in[r] : 0.f, rstd = live ? rstd_in[r] : 0.f;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * lanes + lane) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) xh[i * V + e] = w[i * V + e] = 0.f;
      if (live && c < dim) {
        load_vec<T, V>(x + r * dim + c, xh + i * V);
        load_vec<T, V>(dy + r * dim + c, w + i * V);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int k = i * V + e;
          xh[k] = (xh[k] - mean) * rstd;
          dg[k] = fmaf(w[k], xh[k], dg[k]);
          db[k] += w[k];
          w[k] *= gamma[c + e];
          s[0] += w[k];
          s[1] = fmaf(w[k], xh[k], s[1]);
        }
      }
    }
    group_sum<LPR, 2>(s, red + (LPR == 0 ? 32 * flip : 0));
    flip ^= 1;
    if (live) {
      const float a = s[0] * inv_d, bq = s[1] * inv_d;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = (i * lanes + lane) * V;
        if (c >= dim) continue;
        float o[V];
        if (dres != nullptr) load_vec<T, V>(dres + r * dim + c, o);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = rstd * (w[i * V + e] - a - xh[i * V + e] * bq);
          o[e] = dres != nullptr ? d + o[e] : d;
        }
        store_vec<T, V>(dx + r * dim + c, o);
      }
    }
  }
  float* mine = part + (int64_t)blockIdx.x * 2 * dim;
  if constexpr (LPR == 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * lanes + lane) * V;
      if (c < dim)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          mine[c + e] = dg[i * V + e];
          mine[dim + c + e] = db[i * V + e];
        }
    }
  } else {
    // groups of one warp first, then the warps one after the other: a fixed order
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dg[i] += __shfl_xor_sync(0xffffffffu, dg[i], o);
        db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
      }
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k) {
      if ((int)(threadIdx.x >> 5) == k && (threadIdx.x & 31) < LPR) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int c = (i * lanes + lane) * V;
          if (c < dim)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              fold[c + e] = (k == 0 ? 0.f : fold[c + e]) + dg[i * V + e];
              fold[dim + c + e] = (k == 0 ? 0.f : fold[dim + c + e]) + db[i * V + e];
            }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * dim; c += blockDim.x) mine[c] = fold[c];
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
  if (c < 2 * dim) {
#pragma unroll 4
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

struct NormPlan {
  int V, lpr, per, threads;
};

// The lanes a row takes.  16-byte loads need rows that are whole vectors (dim a multiple of 8
// in bf16, 4 in fp32); other widths go value by value.
NormPlan norm_plan(int dim, int esize) {
  NormPlan p{};
  p.V = (dim * esize) % 16 == 0 ? 16 / esize : 1;
  const int n = dim / p.V;
  p.threads = 256;
  if (p.V > 1) {
    if (n <= 8) { p.lpr = 8; p.per = 1; }
    else if (n <= 16) { p.lpr = 16; p.per = 1; }
    else if (n <= 32) { p.lpr = 32; p.per = 1; }
    else if (n <= 64) { p.lpr = 32; p.per = 2; }
    else if (n <= 128) { p.lpr = 32; p.per = 4; }
    else {
      p.lpr = 0;
      p.per = n <= 256 ? 1 : n <= 512 ? 2 : 4;
      p.threads = ((n + p.per - 1) / p.per + 31) / 32 * 32;
    }
  } else {
    if (n <= 32) { p.lpr = 32; p.per = 1; }
    else if (n <= 128) { p.lpr = 32; p.per = 4; }
    else if (n <= 512) { p.lpr = 32; p.per = 16; }
    else { p.lpr = 0; p.per = 16; p.threads = ((n + 15) / 16 + 31) / 32 * 32; }
  }
  return p;
}

int norm_blocks(const NormPlan& p, int64_t rows, int sms, int per_sm) {
  const int64_t per_block = p.lpr == 0 ? 1 : p.threads / p.lpr;
  const int64_t need = (rows + per_block - 1) / per_block;
  const int64_t most = (int64_t)sms * per_sm;
  return (int)(need < most ? need : most);
}

// Calls F with the template parameters of a plan; false for a plan that does not exist.
#define SRNL_NORM_DISPATCH(T, CALL)                                                                       \
  do {                                                                                                    \
    constexpr int W = 16 / sizeof(T);                                                                     \
    if (p.V == 1) {                                                                                       \
      if (p.lpr == 32 && p.per == 1) { CALL(T, 1, 32, 1); }                                               \
      else if (p.lpr == 32 && p.per == 4) { CALL(T, 1, 32, 4); }                                          \
      else if (p.lpr == 32) { CALL(T, 1, 32, 16); }                                                       \
      else { CALL(T, 1, 0, 16); }                                                                         \
    } else if (p.lpr == 8) { CALL(T, W, 8, 1); }                                                          \
    else if (p.lpr == 16) { CALL(T, W, 16, 1); }                                                          \
    else if (p.lpr == 32 && p.per == 1) { CALL(T, W, 32, 1); }                                            \
    else if (p.lpr == 32 && p.per == 2) { CALL(T, W, 32, 2); }                                            \
    else if (p.lpr == 32) { CALL(T, W, 32, 4); }                                                          \
    else if (p.per == 1) { CALL(T, W, 0, 1); }                                                            \
    else if (p.per == 2) { CALL(T, W, 0, 2); }                                                            \
    else { CALL(T, W, 0, 4); }                                                                            \
  } while (0)

}  // namespace
}  // namespace srnl

// ------------------------------------------------------------------ C ABI
struct srnl_ln {
  srnl_ln_config cfg{};
  int device = 0, sms = 0;
  srnl::NormPlan plan{};
  float* part = nullptr;   // [kNormWaves * sms][2][dim]
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
  h->plan = srnl::norm_plan(cfg->dim, cfg->act_dtype == SRNL_BF16 ? 2 : 4);
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess)
    e = cudaMalloc(&h->part, (size_t)h->sms * srnl::kNormWaves * 2 * cfg->dim * sizeof(float));
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
  if (!ln_aligned(x, 16) || !ln_aligned(y, 16)) return ln_fail(h, SRNL_E_INVAL, "x and y must be 16-byte aligned");
  if (!ln_aligned(gamma, 4) || !ln_aligned(beta, 4) || !ln_aligned(mean, 4) || !ln_aligned(rstd, 4))
    return ln_fail(h, SRNL_E_INVAL, "gamma, beta, mean and rstd must be 4-byte aligned");
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
  const srnl::NormPlan& p = h->plan;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = srnl::norm_blocks(p, rows, h->sms, 16);
#define SRNL_NORM_FWD(T, V, LPR, PER)                                                                              \
  srnl::norm_forward_kernel<T, V, LPR, PER><<<blocks, p.threads, 0, s>>>(                                          \
      static_cast<const T*>(x), gamma, beta, static_cast<T*>(y), mean, rstd, rows, dim, h->cfg.eps)
  if (bf16) SRNL_NORM_DISPATCH(__nv_bfloat16, SRNL_NORM_FWD);
  else SRNL_NORM_DISPATCH(float, SRNL_NORM_FWD);
#undef SRNL_NORM_FWD
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
  if (!ln_aligned(x, 16) || !ln_aligned(dy, 16) || !ln_aligned(dres, 16) || !ln_aligned(dx, 16))
    return ln_fail(h, SRNL_E_INVAL, "x, dy, dres and dx must be 16-byte aligned");
  if (!ln_aligned(gamma, 4) || !ln_aligned(mean, 4) || !ln_aligned(rstd, 4) || !ln_aligned(dgamma, 4) || !ln_aligned(dbeta, 4))
    return ln_fail(h, SRNL_E_INVAL, "gamma, mean, rstd, dgamma and dbeta must be 4-byte aligned");
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
  const srnl::NormPlan& p = h->plan;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = srnl::norm_blocks(p, rows, h->sms, srnl::kNormWaves);
  if (rows > 0) {
    const size_t smem = p.lpr == 0 ? 0 : (size_t)2 * dim * sizeof(float);
#define SRNL_NORM_BWD(T, V, LPR, PER)                                                                              \
  srnl::norm_backward_kernel<T, V, LPR, PER><<<blocks, p.threads, smem, s>>>(                                      \
      static_cast<const T*>(x), static_cast<const T*>(dy), static_cast<const T*>(dres), gamma, mean, rstd,         \
      static_cast<T*>(dx), h->part, rows, dim)
    if (bf16) SRNL_NORM_DISPATCH(__nv_bfloat16, SRNL_NORM_BWD);
    else SRNL_NORM_DISPATCH(float, SRNL_NORM_BWD);
#undef SRNL_NORM_BWD
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return ln_cuda_fail(h, e, "layer norm backward launch");
  }
  if (dgamma != nullptr || dbeta != nullptr) {
    srnl::norm_weight_grad_kernel<<<(2 * dim + 31) / 32, 1024, 0, s>>>(h->part, blocks, dim, dgamma, dbeta);
    const cudaError_t e = cudaGetLastError();
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
