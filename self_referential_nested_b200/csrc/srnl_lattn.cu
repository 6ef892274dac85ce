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
// The passes are in srnl_lattn_tc.cu, and for at most 16 tokens, without those splits, in
// srnl_lattn_short.cu; here are the single-token form and the entry points.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <new>

#include "srnl_common.cuh"
#include "srnl_internal.h"
#include "srnl_lattn.h"
#include "srnl_scan.h"

namespace srnl {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// One token per sequence: state <- g state + k v^T, o = state^T q, the state read and written
// once.  A CTA per (sequence, head); a thread owns 4 columns of every kRows-th row, all of whose
// loads it issues first.  Memory is what bounds it: 64 sequences of 16 heads of 64 (33.8 MB, which L2
// keeps from call to call) take 4.8 us, 7.0 TB/s.
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

srnl_status la_check(srnl_lattn* h, const Rows* in, int ni, const Rows* out, int no, const int* lengths) {
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
  const Rows n{lengths, 1, (int64_t)h->cfg.B * 4, (int64_t)h->cfg.B * 4, "lengths"};
  for (int i = 0; i < no; ++i)
    if (la_meet(out[i], n)) {
      snprintf(msg, sizeof msg, "%s overlaps lengths", out[i].name);
      return la_fail(h, SRNL_E_INVAL, msg);
    }
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return la_cuda_fail(h, e, "cudaGetDevice");
  if (cur != h->device) return la_fail(h, SRNL_E_INVAL, "the current device is not the handle's device");
  return SRNL_OK;
}

cudaError_t la_run(srnl_lattn* h, srnl::LaArgs& a, cudaStream_t s) {
  a.B = h->cfg.B; a.T = h->cfg.T; a.heads = h->cfg.heads; a.d = h->cfg.d;
  a.log2g = h->log2g; a.seg_state = h->seg_state; a.err = h->dev_err;
  return a.T <= srnl::kShortTokens ? srnl::launch_la_short(a, s) : srnl::launch_la_tc(a, h->sms, s);
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
      const int segs = la_tc_segments(cfg->T, cfg->B * la_groups(cfg->heads, cfg->d) * passes, h->sms);
      const size_t n = segs > 1 ? (size_t)passes * cfg->B * cfg->heads * segs * cfg->d * cfg->d * sizeof(float) : 0;
      if (n > most) most = n;
    }
    if (most > 0) e = cudaMalloc(&h->seg_state, most);
  }
  if (e == cudaSuccess) e = cudaMalloc(&h->dev_err, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(h->dev_err, 0, sizeof(int));
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);   // a call's stream need not wait for the one these and the copies ran on
  if (e == cudaSuccess) e = prepare_la_tc(cfg->d);
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
