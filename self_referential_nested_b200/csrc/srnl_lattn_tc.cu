// Tensor-core passes of linear attention (sm_100a).
//
// One CTA takes a 128-channel group (a 128-wide head, or two narrower ones) of a segment of a
// sequence, in chunks of 128 tokens, with the formulas of srnl_lattn.cu:
//   G  = a b^T                          tokens x tokens, per head          (1)
//   O  = a Z                            tokens x channels                  (4)
//   dZ = (w b)^T c                      channels of b x channels of c      (5)
//   O <- g^(i + 1) O + (mask(G) g^(i - j)) c                               (3)
//   Z <- g^C Z + dZ
// All five are tcgen05 products with accumulators in TMEM.  a, b and c arrive by TMA as 64-channel
// boxes, 128-byte rows, and serve as they lie, K-major where channels are summed over and
// MN-major where tokens are.  The masked G goes back to TMEM over G's own columns as the left
// operand of (3), and so does w b for (5) where TMEM has room (128-wide heads; narrower ones keep it
// in a ring in shared memory).  O leaves through a's tile.  Roles: two threads load, two issue
// products (those of the rows, and (5), whose chain of decayed b, dZ and Z goes on beside them), four
// warps a head own a token's row per thread (masking, O), eight half a row of the state per thread,
// in fp32 registers (the decayed b, Z).  Z and w b are split into two bf16 parts (a third of w b where
// the state itself is asked for).
//
// Two heads of up to 64 channels share a CTA so that every product has 128 rows; (5) computes
// the two heads' cross terms with it and nobody reads them.  A 32-wide head runs as a 64-wide one
// whose upper half the loads fill with zeros and the stores leave out.
//
// What bounds it: a chunk's operands, parts and results pass through shared memory about 4400 times
// 128 bytes (5400 for narrow heads), two thirds of the 7000 cycles that a chunk takes; the rest is the
// chain of products, masking and the state's update, which wait for one another.  One sequence of
// 16384 tokens, 16 heads of 128, states in and out: 128 us with cold operands (2.2 TB/s), 51 of them
// the segments' states, 115 us with operands in L2; backward of 8 x 2048 tokens, 16 heads of 64, lengths
// at random (a little over half of the tokens, 132 MB): 68 us (1.9 TB/s), the longest sequence's chunks.
//
// Sequences that leave SMs idle are cut into segments.  One kernel sums what each segment adds to
// the state, a second turns the sums into the states they start from, and the pass itself follows.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "srnl_lattn.h"
#include "srnl_scan.h"
#include "srnl_tma.cuh"
#include "srnl_umma.cuh"

namespace srnl {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kC = 128;                  // tokens per chunk, and channels per CTA
constexpr uint32_t kBoxBytes = kC * 128; // 128 tokens x 64 channels
constexpr uint32_t kTile = 2 * kBoxBytes;
__host__ __device__ constexpr int la_threads(int nh) { return 128 * (3 + nh); }   // loads and products, 4 row warps a head, 8 state warps
constexpr int kMaxSorted = 512;          // sequences that a CTA ranks by length
constexpr int kSegFormers = 8, kSegThreads = 128 + 32 * kSegFormers;   // of the segments' kernel
constexpr int kStateThreads = 256;

struct LaMaps {
  CUtensorMap m[3][4];   // [pass][a, b, c, out]: (channel of 64 or fewer, 64-channel piece, token, batch)
};

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int piece, int token, int batch) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(piece), "r"(token), "r"(batch), "r"(src)
               : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int piece, int token, int batch, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(piece), "r"(token), "r"(batch), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int piece, int token, int batch) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(0),
               "r"(piece), "r"(token), "r"(batch)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// D (+)= A B^T over K = 16 with A in TMEM (bf16 pairs, 8 columns).
__device__ __forceinline__ void mma_k16_tmem_a(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc, bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(bd), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A warp's arrival: every lane's writes are done, one lane signals.
__device__ __forceinline__ void warp_arrive(unsigned long long* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

enum { kTwo, kThree, kThirdOnly };   // parts of w b to write; the third alone takes the first's place

// Parts of w b for 32 tokens from row `row0` of tile b into a slot of the ring: x = w b, part 0 =
// bf16(x), part 1 = bf16(x - part 0), or the rest alone.  256 threads (t), a 16-byte unit of two
// rows.  A row without weight (no token of this sequence: it may hold anything) becomes zero.  All
// loads come first: the products' operands take most of the shared memory's time, and a load waits
// long for its turn.
constexpr uint32_t kSlot = 16384, kSlotPart = 8192, kSlotBox = 4096;   // two parts of 32 tokens, two boxes of 64 channels each
__device__ __forceinline__ void form_parts(const unsigned char* b, int row0, unsigned char* to, const float* w, int t, bool rest) {
  const int u = t & 15, box = u >> 3;
  const uint32_t sw = (uint32_t)(((u & 7) ^ ((t >> 4) & 7)) << 4);
  const float* wr = w + box * kC + row0 + (t >> 4);
  const unsigned char* src = b + box * kBoxBytes + (row0 + (t >> 4)) * 128 + sw;
  unsigned char* dst = to + (uint32_t)box * kSlotBox + (uint32_t)(t >> 4) * 128 + sw;
  uint4 raw[2];
  float f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    raw[i] = *reinterpret_cast<const uint4*>(src + i * 2048);
    f[i] = wr[16 * i];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool on = f[i] != 0.f;
    const float2 g = make_float2(f[i], f[i]);
    const uint32_t in[4] = {on ? raw[i].x : 0u, on ? raw[i].y : 0u, on ? raw[i].z : 0u, on ? raw[i].w : 0u};
    uint32_t o0[4], o1[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 x = __fmul2_rn(make_float2(bf16_lo(in[k]), bf16_hi(in[k])), g);
      o0[k] = pack_bf16(x.x, x.y);
      x = __fadd2_rn(x, make_float2(-bf16_lo(o0[k]), -bf16_hi(o0[k])));
      o1[k] = pack_bf16(x.x, x.y);
      if (rest) o0[k] = pack_bf16(x.x - bf16_lo(o1[k]), x.y - bf16_hi(o1[k]));
    }
    *reinterpret_cast<uint4*>(dst + i * 2048) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
    if (!rest) *reinterpret_cast<uint4*>(dst + kSlotPart + i * 2048) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  }
}
// The parts of w b as the left operand in TMEM: for 32 channels (lanes 32 q on) and 32 N tokens from
// `token` of tile b, part p to columns ta + 64 p + token / 2 on.  ldmatrix transposes as it reads: a
// register holds two tokens of a channel, in the places tcgen05.st's 16-lane shape wants them.
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_16lanes(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
template <int N>
__device__ __forceinline__ void form_tmem(uint32_t b, uint32_t ta, int q, int token, const float* w, float scale, int parts, int lane) {
#pragma unroll 1
  for (int k = 0; k < N; ++k) {
    const int t0 = token + 32 * k;
    uint32_t raw[2][2][4];
    float2 f[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // 16 channels
      const int unit = 2 * h + 4 * (q & 1) + ((lane >> 3) & 1);
      const uint32_t at = b + (q >> 1) * kBoxBytes + (uint32_t)(t0 + (lane >> 4) * 8 + (lane & 7)) * 128 + ((unit ^ (lane & 7)) << 4);
      ldmatrix_t(raw[h][0], at);
      ldmatrix_t(raw[h][1], at + 16 * 128);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const float2*>(w + t0 + 8 * i + 2 * (lane & 3));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t o[3][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 g = f[i >> 1];
        const uint32_t in = raw[h][i >> 2][i & 3];
        float2 x = make_float2(g.x != 0.f ? bf16_lo(in) : 0.f, g.y != 0.f ? bf16_hi(in) : 0.f);
        x = __fmul2_rn(x, make_float2(g.x * scale, g.y * scale));
        o[0][i] = pack_bf16(x.x, x.y);
        x = __fadd2_rn(x, make_float2(-bf16_lo(o[0][i]), -bf16_hi(o[0][i])));
        o[1][i] = pack_bf16(x.x, x.y);
        if (parts != kTwo) o[2][i] = pack_bf16(x.x - bf16_lo(o[1][i]), x.y - bf16_hi(o[1][i]));
      }
      const uint32_t at = ta + ((uint32_t)(32 * q + 16 * h) << 16) + (uint32_t)(t0 >> 1);
      if (parts != kThirdOnly) {
        tmem_st_16lanes(at, o[0]);
        tmem_st_16lanes(at + 64, o[1]);
      }
      if (parts != kTwo) tmem_st_16lanes(parts == kThree ? at + 128 : at, o[2]);
    }
  }
}
// Rows of tile c from token `from` on become zero (tokens behind a sequence's last one hold
// anything, and zero times NaN is NaN).
__device__ __forceinline__ void clear_rows(unsigned char* c, int from, int t, int threads) {
  for (int i = t; i < (kC - from) * 16; i += threads) {
    const int r = from + (i >> 4), u = i & 15;
    *reinterpret_cast<uint4*>(c + (u >> 3) * kBoxBytes + r * 128 + (u & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Causality of what is not finite.  P c (3) multiplies a masked pair's zero with the later token's c, and zero
// times NaN is NaN.  An infinity or NaN anywhere in a chunk's c thus shows in its first token's row, which
// is watched; once there is one, the CTA makes its pass again with an eye on c: the rows' warps look
// through their head's c, 32 tokens each, note the first token that has what is not finite, channel by
// channel, and replace it by zero once the state's product, where it belongs, has taken it; after (3)
// they put NaN from that token on.  Looking in the first pass cost 6 % and more (8 x 2048, 16 heads of
// 128: 67 -> 75 us), the watch costs 0 to 2 % (backward of 64: 114 -> 116.5).  The second pass is not
// made fast: 1 x 16384, 16 heads of 128, all NaN: 684 us.
constexpr int kNone = 255;
// Sums of products of pairs: not finite where a value is not (or where values beyond 2^63 meet, which costs time only).
__device__ __forceinline__ void add_pairs(uint32_t (&sum)[2], const uint4& x) {
  asm volatile("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[0]) : "r"(x.x), "r"(x.y));
  asm volatile("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[1]) : "r"(x.z), "r"(x.w));
}
__device__ __forceinline__ bool not_finite(const uint32_t (&sum)[2]) {
  return ((((sum[0] & 0x7F807F80u) + 0x00800080u) | ((sum[1] & 0x7F807F80u) + 0x00800080u)) & 0x80008000u) != 0u;
}
__device__ __forceinline__ bool look_through(const unsigned char* rows32, int rows, int lane) {
  uint4 v[8];
  const unsigned char* at = rows32 + lane * 16;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = 4 * i + (lane >> 3) < rows ? *reinterpret_cast<const uint4*>(at + i * 512) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t sum[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) add_pairs(sum, v[i]);
  return __any_sync(0xFFFFFFFFu, not_finite(sum));
}
// The rows in the chunk's order (rev: upwards from the last); a lane has two channels.  first: [64].
__device__ __noinline__ void take_out(unsigned char* rows32, int rows, int rev, unsigned char* first, int lane) {
  int at[2] = {kNone, kNone};
  for (int i = 0; i < rows; ++i) {
    const int r = rev ? rows - 1 - i : i;
    unsigned short* v = reinterpret_cast<unsigned short*>(rows32 + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    for (int e = 0; e < 2; ++e)
      if ((v[e] & 0x7F80u) == 0x7F80u) {
        if (at[e] == kNone) at[e] = r;
        v[e] = 0;
      }
  }
  first[2 * lane] = (unsigned char)at[0];
  first[2 * lane + 1] = (unsigned char)at[1];
  fence_async();
}
// NaN in a row's channels of a box from the first bad token on.  first: [4 blocks of rows][2 boxes][64], seen: the
// blocks that have any.
__device__ __noinline__ void spoil_row(uint32_t acc, const unsigned char* first, uint32_t seen, int row, int rev) {
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    float v[32];
    tmem_ld32(v, acc + 32 * b);
    tmem_wait_ld();
#pragma unroll 1
    for (int q = 0; q < 4; ++q)
      if (seen >> (8 * q) & 1)
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int at = first[q * 128 + 32 * b + j];
          if (at != kNone && (rev ? row <= 32 * q + at : row >= 32 * q + at)) v[j] = __int_as_float(0x7FC00000);
        }
    tmem_st32(acc + 32 * b, v);
    tmem_wait_st();
  }
}

// A warp's rows of a head's G (block q of 32 tokens), masked and decayed, as bf16 pairs over G's own
// columns: block j's at 32 j .. + 15.  The distance falls along a row's columns (rises, in reverse).
// Away from the diagonal the powers of g are one product after another from the nearest token on,
// two columns an instruction.  Nothing is read from shared memory, where a load waits some hundred
// cycles for its turn while the products run: a table of powers cost 2000 cycles a block.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool REV>
__device__ __forceinline__ void mask_rows(uint32_t tG, float log2g, int q, int lane) {
  const float g = exp2f(log2g);
  const float2 g2 = make_float2(g * g, g * g);
  float v[32];
  uint32_t w[16];
  tmem_ld32(v, tG + q * 32);
  tmem_wait_ld();
  // the diagonal block: no product of powers from one end reaches every row's own token without
  // leaving the range, so each power is an exponential.  Masked by selection: such a token may
  // hold anything, and its power may be infinite.
  float2 e = REV ? make_float2(log2g * -(float)lane, log2g * (float)(1 - lane)) : make_float2(log2g * (float)lane, log2g * (float)(lane - 1));
  const float2 de = make_float2(REV ? 2.f * log2g : -2.f * log2g, REV ? 2.f * log2g : -2.f * log2g);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(exp2_approx(e.x), exp2_approx(e.y)));
    w[i] = pack_bf16((REV ? 2 * i >= lane : 2 * i <= lane) ? x.x : 0.f, (REV ? 2 * i + 1 >= lane : 2 * i + 1 <= lane) ? x.y : 0.f);
    e = __fadd2_rn(e, de);
  }
  tmem_st16(tG + q * 32, w);
  const float g32 = exp2f(log2g * 32.f);
  float near = exp2f(log2g * (float)(REV ? 32 - lane : lane + 1));   // of the next block's nearest token
#pragma unroll 1
  for (int j = REV ? q + 1 : q - 1; REV ? j < 4 : j >= 0; j += REV ? 1 : -1) {
    tmem_ld32(v, tG + j * 32);
    tmem_wait_ld();
    float2 f = REV ? make_float2(near, near * g) : make_float2(near * g, near);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int i = REV ? k : 15 - k;
      const float2 x = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), f);
      w[i] = pack_bf16(x.x, x.y);
      f = __fmul2_rn(f, g2);
    }
    tmem_st16(tG + j * 32, w);
    near *= g32;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 0u;
#pragma unroll 1
  for (int j = REV ? 0 : q + 1; j < (REV ? q : 4); ++j) tmem_st16(tG + j * 32, w);
}

struct Chunk {
  int cnt, lead, token0;   // tokens, the exponent z0 adds, token of the tile's row 0 (may be negative)
};
__device__ __forceinline__ Chunk chunk_of(int t0, int end, int n, int reverse) {
  Chunk k;
  k.cnt = min(kC, end - t0);
  k.lead = reverse && t0 == 0 ? 0 : 1;
  k.token0 = reverse ? n - t0 - kC : t0;
  return k;
}

// A tile: pieces 2 group and 2 group + 1 of 128 tokens.  A piece past the last head, a token
// outside the sequence and the upper half of a 32-wide head's piece read as zeros.
__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* map, int group, int token, int batch, unsigned long long* bar) {
  mbar_expect(bar, kTile);
  for (int h = 0; h < 2; ++h) tma_load_4d(smem_u32(dst) + h * kBoxBytes, map, 2 * group + h, token, batch, bar);
}
// A tile into L2: c has one buffer and is loaded late.
__device__ __forceinline__ void prefetch_chunk(const CUtensorMap* map, int group, int token, int batch) {
  for (int h = 0; h < 2; ++h) tma_prefetch_4d(map, 2 * group + h, token, batch);
}

enum {   // barriers; two each of those that the next name leaves room for
  kFullA, kFullB = kFullA + 2, kFullC = kFullB + 2, kFreeA, kFreeB = kFreeA + 2, kFreeC = kFreeB + 2,
  kG, kRows, kO2, kO, kOFree, kParts, kPDone = kParts + 2, kZ = kPDone + 2, kDZ, kClear, kBars
};

// A CTA's shared memory behind its seven tiles.
template <int NH>
struct LaShared {
  float* wt;                    // [NH][kC]: weights of the chunk's rows of b
  unsigned long long* bar;      // two sets: one for the second pass
  uint32_t* tmem_slot;
  int *failed, *again;
  unsigned char* unsound;       // of c, two chunks in turn: the blocks of 32 rows that hold what is not finite [box][block]
  unsigned char* first_bad;     // and the first such row [block][box][64]
  __device__ __forceinline__ explicit LaShared(unsigned char* sm) {
    wt = reinterpret_cast<float*>(sm + 7 * kTile);
    bar = reinterpret_cast<unsigned long long*>(wt + NH * kC);
    tmem_slot = reinterpret_cast<uint32_t*>(bar + 2 * kBars);
    failed = reinterpret_cast<int*>(tmem_slot + 1);
    again = failed + 1;
    unsound = reinterpret_cast<unsigned char*>(again + 2);
    first_bad = unsound + 16;
  }
};
// What is a CTA's of a sequence of n tokens.
struct LaShare {
  int n, begin, end, chunks;
  int chunks_z;   // chunks whose update of the state is of use
  bool exact;     // the state leaves: a third part of w b
  bool fresh;     // the first chunk meets a zero state
};
__device__ __forceinline__ LaShare share_of(const LaArgs& args, const LaPass& P, int batch, int seg) {
  LaShare s;
  s.n = args.T;
  if (args.lengths != nullptr) s.n = min(max(args.lengths[batch], 0), args.T);
  s.begin = seg * args.seg_len;
  s.end = min(s.begin + args.seg_len, s.n);
  s.chunks = s.end > s.begin ? (s.end - s.begin + kC - 1) / kC : 0;
  // the segment that holds the last token (the first one of an empty sequence) writes the state
  s.exact = P.zn != nullptr && seg == (s.n > 0 ? (s.n - 1) / args.seg_len : 0);
  s.chunks_z = s.exact ? s.chunks : s.chunks - 1;
  s.fresh = P.z0 == nullptr && seg == 0;
  return s;
}

// The roles' work on a segment.  WATCH: with an eye on c, after a pass that met what is not finite; a
// copy of its own, since in one loop both were 10 % slower than the first alone.
template <int D, bool WATCH>
__device__ __forceinline__ void decay_pass(const LaMaps& maps, const LaArgs& args, unsigned char* sm, uint32_t tmem, int which, int group, int batch) {
  constexpr int NH = kC / D;
  // two tiles of a (O leaves through a's, when its products are done), two of b, c, the state's two
  // parts and, for narrow heads, the ring of w b
  constexpr uint32_t kZPart = NH == 2 ? kTile / 2 : kTile;
  unsigned char *sa = sm, *sb = sa + 2 * kTile, *sc = sb + 2 * kTile, *zh = sc + kTile, *zl = zh + kZPart, *ps = zl + kZPart;
  const LaShared<NH> sh(sm);
  float* wt = sh.wt;
  unsigned long long* bar = sh.bar + (WATCH ? kBars : 0);
  int *failed = sh.failed, *again = sh.again;
  unsigned char *unsound = sh.unsound, *first_bad = sh.first_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, seg = blockIdx.x;
  const LaPass& P = args.pass[which];
  const int rev = P.reverse, dr = args.d;   // dr: a head's channels, D or 32 of a 64-wide piece
  const uint32_t tG = tmem, tP = tmem + 128, tO = tmem + 256, tZ = tmem + 384;   // tP: wide heads' w b
  const LaShare share = share_of(args, P, batch, seg);
  const int n = share.n, begin = share.begin, end = share.end, chunks = share.chunks, chunks_z = share.chunks_z;
  const bool exact = share.exact, fresh = share.fresh;

  if (warp == 0) {
    if (lane == 0) {
      for (int k = 0; k < chunks; ++k) {
        if (!mbar_pass(&bar[kFreeB + (k & 1)], (k >> 1 & 1) ^ 1, failed)) break;
        load_tile(sb + (k & 1) * kTile, &maps.m[which][1], group, chunk_of(begin + k * kC, end, n, rev).token0, batch, &bar[kFullB + (k & 1)]);
      }
    }
  } else if (warp == 3) {
    if (lane == 0) {
      for (int k = 0; k < chunks; ++k) {
        const int token0 = chunk_of(begin + k * kC, end, n, rev).token0;
        if (k + 1 < chunks) prefetch_chunk(&maps.m[which][2], group, chunk_of(begin + (k + 1) * kC, end, n, rev).token0, batch);
        if (!mbar_pass(&bar[kFreeA + (k & 1)], (k >> 1 & 1) ^ 1, failed)) break;
        load_tile(sa + (k & 1) * kTile, &maps.m[which][0], group, token0, batch, &bar[kFullA + (k & 1)]);
        if (!mbar_pass(&bar[kFreeC], (k & 1) ^ 1, failed)) break;
        load_tile(sc, &maps.m[which][2], group, token0, batch, &bar[kFullC]);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t iG = idesc_mn(128, 128, false, false);                 // a b^T
      constexpr uint32_t iO = idesc_mn(128, NH == 2 ? 64 : 128, false, true);   // a Z, P c
      const uint64_t da0 = desc_k_major(smem_u32(sa)), db0 = desc_k_major(smem_u32(sb)), dc = desc_mn_major(smem_u32(sc), kBoxBytes);
      const uint64_t dzh = desc_mn_major(smem_u32(zh), kBoxBytes), dzl = desc_mn_major(smem_u32(zl), kBoxBytes);
      constexpr uint64_t kBox16 = kBoxBytes >> 4;
#pragma unroll 1
      for (int k = 0; k < chunks; ++k) {
        const uint32_t ph = k & 1, ph2 = k >> 1 & 1;
        const uint64_t da = da0 + (uint64_t)ph * (kTile >> 4), db = db0 + (uint64_t)ph * (kTile >> 4);
        // (1) G; its columns hold the previous chunk's left operand until (3) is done
        if (k > 0) mbar_pass(&bar[kO], ph ^ 1, failed);
        mbar_pass(&bar[kFullB + ph], ph2, failed);
        mbar_pass(&bar[kFullA + ph], ph2, failed);
        tmem_fence_after();
#pragma unroll
        for (int s = 0; s < 8; ++s) {   // 16 channels a step, four to a box
          const uint64_t at = (uint64_t)(s >> 2) * kBox16 + (uint64_t)(s & 3) * 2;
          mma_k16_desc(tG + (NH == 2 ? (s >> 2) * 128 : 0), da + at, db + at, iG, NH == 2 ? (s & 3) > 0 : s > 0);
        }
        mma_commit(&bar[kG]);
        mma_commit(&bar[kFreeB + ph]);
        // (4) O = a Z, once Z is written and the last O read
        mbar_pass(&bar[kZ], ph, failed);
        mbar_pass(&bar[kOFree], ph ^ 1, failed);
        tmem_fence_after();
        if (k > 0 || !fresh)
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const int h = NH == 2 ? s >> 2 : 0;
            const uint64_t az = (part == 0 ? dzh : dzl) +   // 16 rows of Z
                                (NH == 2 ? (uint64_t)h * (kTile >> 6) + (uint64_t)(s & 3) * 128 : (uint64_t)s * 128);
            mma_k16_desc(tO + h * 64, da + (uint64_t)(s >> 2) * kBox16 + (uint64_t)(s & 3) * 2, az, iO,
                         part > 0 || (NH == 2 ? (s & 3) > 0 : s > 0));
          }
        mma_commit(&bar[kO2]);
        // (3) O += P c
        mbar_pass(&bar[kRows], ph, failed);
        mbar_pass(&bar[kFullC], ph, failed);
        if (!rev && k == chunks - 1 && (end - begin) % kC != 0) mbar_pass(&bar[kClear], 0, failed);   // c's spare rows are zeros
        tmem_fence_after();
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_k16_tmem_a(tO + h * 64, tG + h * 128 + (s >> 1) * 32 + (s & 1) * 8, dc + (uint64_t)s * 128 + (uint64_t)h * kBox16, iO,
                           s > 0 || k > 0 || !fresh);
        mma_commit(&bar[kO]);
        mma_commit(&bar[kFreeC]);
      }
    }
  } else if (warp == 2) {
    if (lane == 0) {
      // (5) dZ from the parts of w b, the smaller ones first where they are there: the accumulator's sums
      // are cut off, not rounded, and are less in error while they are small (the returned state of
      // narrow heads: 0.94e-6 -> 0.52e-6 of its norm)
      const uint64_t dc = desc_mn_major(smem_u32(sc), kBoxBytes);
      const int uses = NH == 1 ? (exact ? 2 : 1) : exact ? 3 : 2;   // of a place of the parts in a chunk
#pragma unroll 1
      for (int k = 0; k < chunks_z; ++k) {
        mbar_pass(&bar[kFullC], k & 1, failed);
        // c's spare rows are zeros: all state warps clear them, and a wide head's first parts come from half of those
        if (!rev && k == chunks - 1 && (end - begin) % kC != 0) mbar_pass(&bar[kClear], 0, failed);
        if constexpr (NH == 1) {   // in TMEM, half the tokens a step; then the rest in the first part's place
          constexpr uint32_t iZ = idesc_mn(128, 128, false, true);
#pragma unroll 1
          for (int st = 0; st < 2 * uses; ++st) {
            const int half = st & 1;
            mbar_pass(&bar[kParts + half], (k * uses + (st >> 1)) & 1, failed);
            tmem_fence_after();
            const uint32_t pa = tP + half * 32;
            const uint64_t pc = dc + (uint64_t)half * 512;
            if (st < 2) {   // the second part, and the first behind it
#pragma unroll
              for (int i = 0; i < 4; ++i) mma_k16_tmem_a(tZ, pa + 64 + i * 8, pc + (uint64_t)i * 128, iZ, st > 0 || i > 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_k16_tmem_a(tZ, pa + i * 8, pc + (uint64_t)i * 128, iZ, true);
            mma_commit(&bar[kPDone + half]);
          }
        } else {   // in the ring, a quarter of the tokens a step, before them the rest, two quarters a step; the slots in turn
          constexpr uint32_t iZ = idesc_mn(128, 128, true, true);
          const uint64_t dp = desc_mn_major(smem_u32(ps), kSlotBox);
#pragma unroll 1
          for (int st = 0; st < 2 * uses; ++st) {
            const int slot = st & 1;
            mbar_pass(&bar[kParts + slot], (k * uses + (st >> 1)) & 1, failed);
            tmem_fence_after();
            const uint64_t pa = dp + (uint64_t)slot * (kSlot >> 4);
            const bool rest = exact && st < 2;
            const int quarter = exact ? st - 2 : st;
#pragma unroll
            for (int i = 0; i < 4; ++i)   // part 1 - (i >> 1), 16 tokens i & 1; of the rest: quarter i >> 1 of two
              mma_k16_desc(tZ, pa + (uint64_t)(rest ? i >> 1 : 1 - (i >> 1)) * (kSlotPart >> 4) + (uint64_t)(i & 1) * 128,
                           dc + (uint64_t)(rest ? st * 4 + i : quarter * 2 + (i & 1)) * 128, iZ, st > 0 || i > 0);
            mma_commit(&bar[kPDone + slot]);
          }
        }
        mma_commit(&bar[kDZ]);
        mma_commit(&bar[kFreeC]);
      }
    }
  } else if (warp >= 4 && warp < 4 + 4 * NH) {
    // ---- token rows: a warp has 32 of them, of one head
    const int q = warp & 3, head = NH == 2 ? (warp - 4) >> 2 : 0, r = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const int ord = rev ? kC - 1 - r : r;   // the token's place in the chunk's order
    const bool live = group * NH + head < args.heads;
    const float lg = live ? args.log2g[group * NH + head] : 0.f;
    const uint32_t tH = tG + lanes + head * 128, tR = tO + lanes + head * 64;
#pragma unroll 1
    for (int k = 0; k < chunks; ++k) {
      const uint32_t ph = k & 1;
      const Chunk c = chunk_of(begin + k * kC, end, n, rev);
      mbar_pass(&bar[kG], ph, failed);
      tmem_fence_after();
      int own = lane;
      asm volatile("" : "+r"(own));   // nothing of a row's place is taken out of the loop: it would cost 40 registers
      if (rev) mask_rows<true>(tH, lg, q, own);
      else mask_rows<false>(tH, lg, q, own);
      if (k > 0 && lane == 0) {   // the last chunk's O has left a's tile
        bulk_wait_read<0>();
        mbar_arrive(&bar[kFreeA + (ph ^ 1)]);
      }
      if constexpr (WATCH) {
        mbar_pass(&bar[kFullC], ph, failed);
        __syncwarp();
#pragma unroll 1
        for (int h = 0; h < 3 - NH; ++h) {   // the head's boxes
          unsigned char* rows32 = sc + (head + h) * kBoxBytes + q * 4096;
          const int rows = rev ? 32 : min(max(c.cnt - 32 * q, 0), 32);   // those behind the last token are not c's
          const bool found = look_through(rows32, rows, lane);
          if (lane == 0) unsound[8 * ph + 4 * (head + h) + q] = found;
          if (found) {
            if (k < chunks_z) mbar_pass(&bar[kDZ], ph, failed);
            __syncwarp();
            take_out(rows32, rows, rev, first_bad + 512 * ph + 128 * q + 64 * (head + h), lane);
          }
        }
      }
      // the state's share of O, decayed to the row
      const float f = exp2f(lg * (float)((rev ? kC - 1 - own : own) - (rev ? 32 * q : -32 * q) + c.lead));
      mbar_pass(&bar[kO2], ph, failed);
      tmem_fence_after();
      if (k > 0 || !fresh)
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
        float v[32];
        tmem_ld32(v, tR + cb * 32);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 x = __fmul2_rn(make_float2(v[j], v[j + 1]), make_float2(f, f));
          v[j] = x.x;
          v[j + 1] = x.y;
        }
        tmem_st32(tR + cb * 32, v);
      }
      tmem_wait_st();
      warp_arrive(&bar[kRows], lane);
      unsigned char* so = sa + ph * kTile;
      // O: a whole chunk's leaves by TMA, the last, shorter one's goes straight to its rows
      mbar_pass(&bar[kO], ph, failed);
      __syncwarp();
      tmem_fence_after();
      if constexpr (WATCH) {
        mbar_pass(&bar[kRows], ph, failed);   // what the others found
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 3 - NH; ++h) {   // the head's boxes
          const uint32_t seen = *reinterpret_cast<const uint32_t*>(unsound + 8 * ph + 4 * (head + h));
          if (seen != 0) spoil_row(tR + h * 64, first_bad + 512 * ph + (head + h) * 64, seen, r, rev);
        }
      }
      uint32_t sum[2] = {0u, 0u};
      bf16* dst = P.out + ((int64_t)batch * args.T + c.token0 + r) * P.ldo + (int64_t)(group * NH + head) * dr;
#pragma unroll
      for (int cb = 0; cb < D / 32; ++cb) {
        float v[32];
        tmem_ld32(v, tR + cb * 32);
        tmem_wait_ld();
        if (cb == D / 32 - 1) warp_arrive(&bar[kOFree], lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w = make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                                     pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
          if (!WATCH) add_pairs(sum, w);
          const int box = NH == 2 ? head : cb >> 1, unit = (cb & 1) * 4 + j;
          if (c.cnt == kC) *reinterpret_cast<uint4*>(so + box * kBoxBytes + r * 128 + ((unit ^ (r & 7)) << 4)) = w;
          else if (ord < c.cnt && live && cb * 32 < dr) *reinterpret_cast<uint4*>(dst + cb * 32 + j * 8) = w;
        }
      }
      if (!WATCH && ord == 0 && not_finite(sum)) *again = 1;
      if (c.cnt == kC) {
        fence_async();
        __syncwarp();
        if (lane == 0) {
          for (int h = 0; h < 2; ++h)
            if (live && (NH == 1 || h == head))
              tma_store_4d(&maps.m[which][3], smem_u32(so) + h * kBoxBytes + q * 4096, 2 * group + h, c.token0 + 32 * q, batch);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else if (warp >= 4 + 4 * NH) {
    // ---- rows of the state: channel r of the group's b, half of its head's c channels, fp32.  The
    // sums are taken here, not in the products' accumulator: their rounding there is not to
    // nearest and would add up over a long memory.
    constexpr int Z = D / 2;
    const int q = warp & 3, t = tid - 128 * (1 + NH), r = 32 * q + lane, h = NH == 2 ? r / 64 : 0, br = r % D,
              hf = (warp - 4 - 4 * NH) >> 2;
    const int head = group * NH + h;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t tD = tZ + lanes + (NH == 2 ? h * 64 : 0) + hf * Z;   // dZ
    const bool live = head < args.heads && br < dr && hf * Z < dr;
    const float lg = head < args.heads ? args.log2g[head] : 0.f;
    float z[Z];
    // columns 8 u .. + 7 in two bf16 parts: row r of Z, its head's columns (a box for each half of
    // a 128-wide head)
    auto put_z = [&](int u) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = z[8 * u + 2 * i], y = z[8 * u + 2 * i + 1];
        hi[i] = pack_bf16(x, y);
        const float2 e = __fadd2_rn(make_float2(x, y), make_float2(-bf16_lo(hi[i]), -bf16_hi(hi[i])));
        lo[i] = pack_bf16(e.x, e.y);
      }
      const int unit = NH == 2 ? hf * 4 + u : u;
      const uint32_t off = (NH == 2 ? (uint32_t)r * 128 : (uint32_t)hf * kBoxBytes + (uint32_t)r * 128) + (uint32_t)((unit ^ (r & 7)) << 4);
      *reinterpret_cast<uint4*>(zh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(zl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
    {
      const int64_t sq = (int64_t)batch * args.heads + head;
      const float* src = args.segs > 1 ? args.seg_state + (((int64_t)which * args.B * args.heads + sq) * args.segs + seg) * dr * dr
                                       : P.z0 != nullptr ? P.z0 + sq * dr * dr : nullptr;
      const bool tr = args.segs == 1 && P.z0_t;
#pragma unroll
      for (int i = 0; i < Z; i += 4) {
        const int c = hf * Z + i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && src != nullptr) {
          if (tr) v = make_float4(src[c * dr + br], src[(c + 1) * dr + br], src[(c + 2) * dr + br], src[(c + 3) * dr + br]);
          else v = *reinterpret_cast<const float4*>(src + br * dr + c);
        }
        z[i] = v.x; z[i + 1] = v.y; z[i + 2] = v.z; z[i + 3] = v.w;
      }
      if (!fresh) {
#pragma unroll
        for (int u = 0; u < Z / 8; ++u) put_z(u);
        fence_async();
      }
      warp_arrive(&bar[kZ], lane);
    }
#pragma unroll 1
    for (int k = 0; k < chunks; ++k) {
      const uint32_t ph = k & 1;
      const Chunk c = chunk_of(begin + k * kC, end, n, rev);
      if (c.cnt < kC) {   // the last chunk: its own weights, g^(tokens behind the row's)
        asm volatile("bar.sync 2, 256;" ::: "memory");
        for (int i = t; i < NH * kC; i += kStateThreads) {
          const int row = i % kC, o = rev ? kC - 1 - row : row;
          const int hh = group * NH + i / kC;
          wt[i] = o < c.cnt && hh < args.heads ? exp2f(args.log2g[hh] * (float)(c.cnt - 1 - o)) : 0.f;
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (!rev) {
          mbar_pass(&bar[kFullC], ph, failed);
          clear_rows(sc, c.cnt, t, kStateThreads);
          fence_async();
          warp_arrive(&bar[kClear], lane);
        }
      }
      if (k == chunks_z) break;   // nobody asks for the state behind the last chunk
      mbar_pass(&bar[kFullB + ph], k >> 1 & 1, failed);
      if constexpr (NH == 1) {   // 64 tokens of 32 channels a warp
        const uint32_t tile = smem_u32(sb + ph * kTile);
        const int first = k * (exact ? 2 : 1);   // use of the parts' place
        if (first > 0) mbar_pass(&bar[kPDone + hf], (first - 1) & 1, failed);   // its last products are done
        tmem_fence_after();
        form_tmem<2>(tile, tP, q, 64 * hf, wt, 1.f, kTwo, lane);
        tmem_wait_st();
        warp_arrive(&bar[kParts + hf], lane);
        if (exact) {
          mbar_pass(&bar[kPDone + hf], first & 1, failed);
          tmem_fence_after();
          form_tmem<2>(tile, tP, q, 64 * hf, wt, 1.f, kThirdOnly, lane);
          tmem_wait_st();
          warp_arrive(&bar[kParts + hf], lane);
        }
        warp_arrive(&bar[kFreeB + ph], lane);
      } else {
        unsigned char* tile = sb + ph * kTile;
        const int uses = exact ? 3 : 2;
        if (exact) {   // the rest of two quarters a slot
#pragma unroll 1
          for (int st = 0; st < 2; ++st) {
            if (k > 0) mbar_pass(&bar[kPDone + st], (k * uses - 1) & 1, failed);   // the slot's last products are done
            form_parts(tile, 64 * st, ps + st * kSlot, wt, t, true);
            form_parts(tile, 64 * st + 32, ps + st * kSlot + kSlotPart, wt, t, true);
            fence_async();
            warp_arrive(&bar[kParts + st], lane);
          }
        }
#pragma unroll 1
        for (int st = 0; st < 4; ++st) {
          const int use = k * uses + (exact ? 1 : 0) + (st >> 1);
          if (use > 0) mbar_pass(&bar[kPDone + (st & 1)], (use - 1) & 1, failed);
          form_parts(tile, 32 * st, ps + (st & 1) * kSlot, wt, t, false);
          fence_async();
          warp_arrive(&bar[kParts + (st & 1)], lane);
        }
        warp_arrive(&bar[kFreeB + ph], lane);
      }
      // z <- g^m z + dZ; a factor near one is applied as z + (g^m - 1) z, whose error does not
      // add up over thousands of chunks
      const float e = lg * (float)(c.cnt - 1 + c.lead);
      const bool near = e > -1.f;
      const float fm = near ? expm1f(e * 0.69314718055994531f) : exp2f(e);
      const float2 f2 = make_float2(fm, fm);
      mbar_pass(&bar[kDZ], ph, failed);
      if (k + 1 < chunks) mbar_pass(&bar[kO2], ph, failed);   // (4) has read the old Z
      tmem_fence_after();
#pragma unroll
      for (int cb = 0; cb < Z / 16; ++cb) {
        float v[16];
        tmem_ld16(v, tD + cb * 16);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 x = make_float2(z[16 * cb + j], z[16 * cb + j + 1]);
          const float2 y = __fadd2_rn(__ffma2_rn(x, f2, near ? x : make_float2(0.f, 0.f)), make_float2(v[j], v[j + 1]));
          z[16 * cb + j] = y.x;
          z[16 * cb + j + 1] = y.y;
        }
        if (k + 1 < chunks) {
          put_z(2 * cb);
          put_z(2 * cb + 1);
        }
      }
      if (k + 1 < chunks) {
        fence_async();
        warp_arrive(&bar[kZ], lane);
      }
    }
    if (exact) {
      const float f = rev && n > 0 ? exp2f(lg) : 1.f;
      float* dst = P.zn + ((int64_t)batch * args.heads + head) * dr * dr + (int64_t)br * dr + hf * Z;
      if (live)
#pragma unroll
        for (int i = 0; i < Z; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(f * z[i], f * z[i + 1], f * z[i + 2], f * z[i + 3]);
    }
  }
}

template <int NH>
__device__ __forceinline__ void start_barriers(unsigned long long* bar) {
  for (int i = 0; i < kBars; ++i) {
    const bool rows = i == kRows || i == kOFree || i == kFreeA || i == kFreeA + 1, parts = i == kParts || i == kParts + 1;
    mbar_init(&bar[i], rows || parts ? 4 * NH : i == kZ || i == kClear ? 8 : i == kFreeB || i == kFreeB + 1 ? 9 : i == kFreeC ? 2 : 1);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Weights of a whole chunk's rows of b; m tokens behind the row's.
template <int NH>
__device__ __forceinline__ void whole_weights(float* wt, const LaArgs& args, int group, int rev) {
  for (int i = threadIdx.x; i < NH * kC; i += la_threads(NH)) {
    const int h = group * NH + i / kC, m = i % kC;
    wt[i - m + (rev ? m : kC - 1 - m)] = h < args.heads ? exp2f(args.log2g[h] * (float)m) : 0.f;
  }
}

// Out of line: the first pass keeps its registers.
template <int D>
__device__ __noinline__ void second_pass(const LaMaps& maps, const LaArgs& args, uint32_t tmem, int which, int group, int batch) {
  constexpr int NH = kC / D;
  extern __shared__ __align__(1024) unsigned char sm[];
  const LaShared<NH> sh(sm);
  if (threadIdx.x == 0) start_barriers<NH>(sh.bar + kBars);
  whole_weights<NH>(sh.wt, args, group, args.pass[which].reverse);
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  decay_pass<D, true>(maps, args, sm, tmem, which, group, batch);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(la_threads(kC / D), 1)
    decay_tc_kernel(const __grid_constant__ LaMaps maps, const __grid_constant__ LaArgs args) {
  constexpr int NH = kC / D;
  extern __shared__ __align__(1024) unsigned char sm[];
  const LaShared<NH> sh(sm);
  int* failed = sh.failed;
  const int tid = threadIdx.x, warp = tid >> 5, groups = (args.heads + NH - 1) / NH;
  int which = blockIdx.z, group = blockIdx.y % groups, batch = blockIdx.y / groups;
  if (smem_u32(sm) & 1023u) {           // the swizzled tiles' alignment
    if (tid == 0) atomicExch(args.err, SRNL_E_CUDA);
    return;
  }

  if (tid == 0) {
    *failed = *sh.again = 0;
    start_barriers<NH>(sh.bar);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (args.longest_first) {
    // the CTAs do not all run at once: batch is the one with so many longer sequences
    int* len = reinterpret_cast<int*>(sm);
    const int per = groups * gridDim.z, id = blockIdx.z * gridDim.y + blockIdx.y, rank = id / per;
    which = id % per / groups;
    group = id % groups;
    for (int i = tid; i < args.B; i += la_threads(NH)) len[i] = args.lengths[i];
    __syncthreads();
    for (int i = tid; i < args.B; i += la_threads(NH)) {
      const int mine = len[i];
      int before = 0;
      for (int j = 0; j < args.B; ++j) before += len[j] > mine || (len[j] == mine && j < i);
      if (before == rank) *sh.tmem_slot = i;
    }
    __syncthreads();
    batch = *sh.tmem_slot;
    fence_async();
    __syncthreads();
  }
  whole_weights<NH>(sh.wt, args, group, args.pass[which].reverse);
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sh.tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t tmem = *sh.tmem_slot;
  decay_pass<D, false>(maps, args, sm, tmem, which, group, batch);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(sh.again) != 0 && *reinterpret_cast<volatile int*>(failed) == 0)
    second_pass<D>(maps, args, tmem, which, group, batch);
  if (*reinterpret_cast<volatile int*>(failed)) {   // a wait gave up: report, and let the copies in flight land
    if (tid == 0) atomicExch(args.err, SRNL_E_TIMEOUT);
    const unsigned long long t0 = global_ns();
    for (int i = 0; i < (1 << 20) && global_ns() - t0 < 1000000ull; ++i) {}
  }
  if (warp == 2) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ------------------------------------------------------------------ the segments' states
// What a segment adds to the state, from zero: sum_j g^(tokens behind j) b_j c_j^T.  The weights
// reach to the segment's end, so the chunks' products add up as they are: in the formers' fp32 registers,
// not in TMEM, where a segment of 128 chunks with a decay next to one came out 3.7e-5 of its norm too
// small (now 0.4e-6; 1 x 16384, 16 heads of 128, returned state included: 114 us either way).  Eight
// formers have the registers for it, and form as fast as sixteen.
constexpr int kSegStages = 3;
enum { sFull = 0, sFree = kSegStages, sParts = 2 * kSegStages, sDone = sParts + 2, sTaken = sDone + 2, sBars };   // parts and done: one for each buffer

template <int D>
__global__ void __launch_bounds__(kSegThreads, 1)
    decay_segment_kernel(const __grid_constant__ LaMaps maps, const __grid_constant__ LaArgs args) {
  constexpr int NH = kC / D;
  extern __shared__ __align__(1024) unsigned char sm[];
  float* wt = reinterpret_cast<float*>(sm + 2 * kSegStages * kTile);   // stages of b, c; then [NH][kC]
  unsigned long long* bar = reinterpret_cast<unsigned long long*>(wt + NH * kC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + sBars);
  int* failed = reinterpret_cast<int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int which = blockIdx.z, seg = blockIdx.x, groups = (args.heads + NH - 1) / NH;
  const int group = blockIdx.y % groups, batch = blockIdx.y / groups;
  const int rev = args.pass[which].reverse, dr = args.d;
  const bool exact = args.pass[which].zn != nullptr;
  if (smem_u32(sm) & 1023u) {
    if (tid == 0) atomicExch(args.err, SRNL_E_CUDA);
    return;
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    *failed = 0;
    for (int i = 0; i < sBars; ++i) mbar_init(&bar[i], (i >= sParts && i < sDone) || i == sTaken ? kSegFormers : i >= sFree && i < sParts ? kSegFormers + 1 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < NH * kC; i += kSegThreads) {   // weights of a whole chunk
    const int h = group * NH + i / kC, m = i % kC;
    wt[i - m + (rev ? m : kC - 1 - m)] = h < args.heads ? exp2f(args.log2g[h] * (float)m) : 0.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t tmem = *tmem_slot, tP = tmem + 128;   // the sum, then two buffers of three parts
  int n = args.T;
  if (args.lengths != nullptr) n = min(max(args.lengths[batch], 0), args.T);
  const int begin = seg * args.seg_len, end = min(begin + args.seg_len, n);
  const int chunks = end > begin ? (end - begin + kC - 1) / kC : 0;

  if (warp == 0) {
    if (lane == 0)
      for (int k = 0; k < chunks; ++k) {
        const Chunk c = chunk_of(begin + k * kC, end, n, rev);
        const int s = k % kSegStages;
        if (!mbar_pass(&bar[sFree + s], (k / kSegStages & 1) ^ 1, failed)) break;
        mbar_expect(&bar[sFull + s], 2 * kTile);
        for (int i = 0; i < 2; ++i)
          for (int h = 0; h < 2; ++h)
            tma_load_4d(smem_u32(sm + (2 * s + i) * kTile) + h * kBoxBytes, &maps.m[which][1 + i], 2 * group + h, c.token0, batch,
                        &bar[sFull + s]);
      }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t iZ = idesc_mn(128, 128, false, true);
      for (int k = 0; k < chunks; ++k) {
        const int s = k % kSegStages;
        const uint64_t dc = desc_mn_major(smem_u32(sm + (2 * s + 1) * kTile), kBoxBytes);
        mbar_pass(&bar[sFull + s], k / kSegStages & 1, failed);
        mbar_pass(&bar[sParts + (k & 1)], k >> 1 & 1, failed);
        if (k > 0) mbar_pass(&bar[sTaken], (k - 1) & 1, failed);
        tmem_fence_after();
        for (int part = exact ? 2 : 1; part >= 0; --part)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma_k16_tmem_a(tmem, tP + (k & 1) * 192 + part * 64 + i * 8, dc + (uint64_t)i * 128, iZ,
                            part < (exact ? 2 : 1) || i > 0);
        mma_commit(&bar[sDone + (k & 1)]);
        mma_commit(&bar[sFree + s]);
      }
    }
  } else if (warp >= 4) {
    // 32 channels and a share of the tokens a warp; of the sum, those channels' rows and a share of the columns
    constexpr int kCols = D / (kSegFormers / 4);
    const int q = warp & 3, share = (warp - 4) >> 2, h = NH == 2 ? q >> 1 : 0, head = group * NH + h;
    const float lg = head < args.heads ? args.log2g[head] : 0.f;
    float sum[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) sum[j] = 0.f;
    auto take = [&](int k) {   // chunk k's products
      mbar_pass(&bar[sDone + (k & 1)], k >> 1 & 1, failed);
      __syncwarp();
      tmem_fence_after();
#pragma unroll
      for (int cb = 0; cb < kCols / 32; ++cb) {
        float v[32];
        tmem_ld32(v, tmem + ((uint32_t)(32 * q) << 16) + (NH == 2 ? h * 64 : 0) + share * kCols + cb * 32);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[32 * cb + j] += v[j];
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    };
    for (int k = 0; k < chunks; ++k) {
      const int s = k % kSegStages, t0 = begin + k * kC;
      const Chunk c = chunk_of(t0, end, n, rev);
      unsigned char *b = sm + 2 * s * kTile, *cc = b + kTile;
      float f = 1.f;
      if (c.cnt < kC) {
        asm volatile("bar.sync 2, %0;" ::"n"(32 * kSegFormers) : "memory");
        for (int i = tid - 128; i < NH * kC; i += kSegThreads - 128) {
          const int row = i % kC, o = rev ? kC - 1 - row : row;
          const float l = group * NH + i / kC < args.heads ? args.log2g[group * NH + i / kC] : 0.f;
          wt[i] = o < c.cnt && group * NH + i / kC < args.heads ? exp2f(l * (float)(c.cnt - 1 - o)) : 0.f;
        }
        asm volatile("bar.sync 2, %0;" ::"n"(32 * kSegFormers) : "memory");
      } else {   // a whole chunk's weights, decayed over the tokens behind it
        f = exp2f(lg * (float)(end - t0 - kC));
      }
      if (k > 1) mbar_pass(&bar[sDone + (k & 1)], ((k >> 1) & 1) ^ 1, failed);   // the buffer's last products are done
      mbar_pass(&bar[sFull + s], k / kSegStages & 1, failed);
      tmem_fence_after();
      if (!rev && c.cnt < kC) {
        clear_rows(cc, c.cnt, tid - 128, kSegThreads - 128);
        fence_async();
      }
      form_tmem<kC / 32 * 4 / kSegFormers>(smem_u32(b), tP + (k & 1) * 192, q, share * (kC * 4 / kSegFormers), wt + h * kC, f,
                                           exact ? kThree : kTwo, lane);
      tmem_wait_st();
      warp_arrive(&bar[sParts + (k & 1)], lane);
      if (lane == 0) mbar_arrive(&bar[sFree + s]);
      if (k > 0) {
        take(k - 1);
        warp_arrive(&bar[sTaken], lane);
      }
    }
    if (chunks > 0) take(chunks - 1);
    const int r = 32 * q + lane;
    float* dst = args.seg_state + ((((int64_t)which * args.B + batch) * args.heads + head) * args.segs + seg) * dr * dr +
                 (int64_t)(r % D) * dr + share * kCols;
    if (head < args.heads && r % D < dr && share * kCols < dr)
#pragma unroll
      for (int j = 0; j < kCols; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(failed)) {
    if (tid == 0) atomicExch(args.err, SRNL_E_TIMEOUT);
    const unsigned long long t0 = global_ns();
    for (int i = 0; i < (1 << 20) && global_ns() - t0 < 1000000ull; ++i) {}
  }
  if (warp == 2) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// What each segment adds -> the state each segment starts from, in place; z0 is the first one's.
__global__ void __launch_bounds__(256) decay_start_kernel(const __grid_constant__ LaArgs args) {
  const int D = args.d;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int i = blockIdx.x * 256 + threadIdx.x, which = blockIdx.z, head = blockIdx.y % args.heads, batch = blockIdx.y / args.heads;
  if (i >= D * D) return;
  const LaPass& P = args.pass[which];
  const int64_t sq = (int64_t)batch * args.heads + head;
  int n = args.T;
  if (args.lengths != nullptr) n = min(max(args.lengths[batch], 0), args.T);
  float cur = P.z0 != nullptr ? P.z0[sq * D * D + (P.z0_t ? (i % D) * D + i / D : i)] : 0.f;
  float* at = args.seg_state + ((int64_t)which * args.B * args.heads + sq) * args.segs * D * D + i;
  const float lg = args.log2g[head];
  // g^m as its difference from one where that is small, as where the state is updated chunk by chunk
  auto factor = [&](int m) {
    const float e = lg * (float)m;
    return e > -1.f ? make_float2(expm1f(e * 0.69314718055994531f), 1.f) : make_float2(exp2f(e), 0.f);
  };
  const float2 whole = factor(args.seg_len);
  constexpr int kAhead = 8;   // loads in flight
  for (int s0 = 0; s0 < args.segs; s0 += kAhead) {
    float add[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) add[j] = s0 + j + 1 < args.segs ? at[(int64_t)(s0 + j) * D * D] : 0.f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int s = s0 + j;
      if (s >= args.segs) break;
      const int len = min(max(n - s * args.seg_len, 0), args.seg_len);
      at[(int64_t)s * D * D] = cur;
      // z0 of a reversed pass meets its first token undecayed
      if (len > 0) {
        const bool lead = P.reverse && s == 0;
        const float2 f = len == args.seg_len && !lead ? whole : factor(lead ? len - 1 : len);
        cur = fmaf(f.x, cur, f.y * cur) + add[j];
      }
    }
  }
}

constexpr size_t la_smem(int d) { return 7 * (size_t)kTile + (size_t)(kC / d) * kC * 4 + 2 * kBars * 8 + 32 + 1024; }

template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, static_cast<P>(args)...);
}

template <int D>
cudaError_t launch_tc(LaArgs& a, const LaMaps& m, cudaStream_t s) {
  constexpr int NH = kC / D;
  const int groups = (a.heads + NH - 1) / NH;
  if (a.segs > 1) {
    cudaError_t e = launch_next(decay_segment_kernel<D>, dim3(a.segs - 1, a.B * groups, a.passes), kSegThreads, la_smem(D), s, m, a);
    if (e == cudaSuccess)
      e = launch_next(decay_start_kernel, dim3((a.d * a.d + 255) / 256, a.B * a.heads, a.passes), 256, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return launch_next(decay_tc_kernel<D>, dim3(a.segs, a.B * groups, a.passes), la_threads(NH), la_smem(D), s, m, a);
}

}  // namespace

int la_groups(int heads, int d) { return d == 128 ? heads : (heads + 1) / 2; }

int la_tc_segments(int T, int seqs, int sms) {
  // As many segments as fill the SMs once.  Between half the SMs and all of them, or above, that is one:
  // the segments' states are most of a pass by themselves, so that two waves of half the length, or a
  // second half of the SMs, do not pay for them (4096 tokens, one head of 128, whole, in 2 and in 3
  // segments: 80 sequences 129, 176, 162 us; 112: 128, 191, 216; 148: 138, 230, 260; 75 of 8192: 240,
  // 309, 269; backward of 8 x 2048, 16 heads of 64, 192 passes of a sequence: 116, 151, 169).
  const int chunks = (T + kC - 1) / kC, want = sms / seqs;
  // two chunks a segment at least, and six chunks: below, the two launches before the pass cost more
  // than the chunks that follow one another (512 tokens, 4 heads of 64: 15.6 us whole, 18.6 cut; 1024:
  // 28 and 19.7; 2048: 45 and 20)
  const int most = chunks < 6 ? 1 : chunks / 2;
  return want < 1 ? 1 : want < most ? want : most;
}

cudaError_t launch_la_tc(LaArgs& a, int sms, cudaStream_t s) {
  const int chunks = (a.T + kC - 1) / kC;
  const int want = la_tc_segments(a.T, a.B * la_groups(a.heads, a.d) * a.passes, sms);
  a.seg_len = (chunks + want - 1) / want * kC;
  a.segs = (a.T + a.seg_len - 1) / a.seg_len;
  a.longest_first = a.lengths != nullptr && a.segs == 1 && a.B <= kMaxSorted && a.B * la_groups(a.heads, a.d) * a.passes > sms;
  const TensorMapEncoder enc = ffn_tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  LaMaps m;
  memset(&m, 0, sizeof m);
  const int piece = a.d < 64 ? a.d : 64;   // channels of a piece; a 32-wide head's is half of its box
  for (int i = 0; i < a.passes; ++i) {
    const LaPass& p = a.pass[i];
    const bf16* base[4] = {p.a, p.b, p.c, p.out};
    const int64_t ld[4] = {p.lda, p.ldb, p.ldc, p.ldo};
    for (int j = 0; j < 4; ++j) {
      const cuuint64_t token = (cuuint64_t)ld[j] * 2;
      const cuuint64_t dim[4] = {(cuuint64_t)piece, (cuuint64_t)a.heads * a.d / piece, (cuuint64_t)a.T, (cuuint64_t)a.B};
      const cuuint64_t str[3] = {(cuuint64_t)piece * 2, token, a.B > 1 ? token * a.T : token};
      const cuuint32_t box[4] = {64u, 1u, j == 3 ? 32u : (cuuint32_t)kC, 1u}, est[4] = {1u, 1u, 1u, 1u};   // out: a warp's rows
      if (enc(&m.m[i][j], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<bf16*>(base[j]), dim, str, box, est,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
  }
  return a.d == 128 ? launch_tc<128>(a, m, s) : launch_tc<64>(a, m, s);
}

cudaError_t prepare_la_tc(int d) {
  const int n = (int)la_smem(d == 128 ? 128 : 64);
  if (d != 128) {
    cudaError_t e = cudaFuncSetAttribute(decay_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
    return e == cudaSuccess ? cudaFuncSetAttribute(decay_segment_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, n) : e;
  }
  cudaError_t e = cudaFuncSetAttribute(decay_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
  return e == cudaSuccess ? cudaFuncSetAttribute(decay_segment_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, n) : e;
}

}  // namespace srnl
