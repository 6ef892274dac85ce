// Gated feed-forward branch with its backward pass (sm_100a), bf16 with fp32 accumulation, for
// training and serving the layers around the SRNL operator.
//
//   gate = x Wg^T, up = x Wu^T, h = act(gate) * up, y = h Wd^T + res
//   dh = dy Wd, dgate = dh * up * act'(gate), dup = dh * act(gate),
//   dx = dgate Wg + dup Wu, dWg = dgate^T x, dWu = dup^T x, dWd = dy^T h
//
// One matrix-product kernel serves all six products; what differs is which way its operands
// lie and what its epilogue does:
//   kGlu      both projections of a 256-token x 128-channel tile at once: Wg's rows are the first
//             half of the product's N and Wu's the second, so act(gate) * up is formed from two
//             accumulators of the same thread, and neither projection is written unless asked
//   kPlain    (+ res), to bf16: y
//   kGrad     the same for dx (its K runs over dgate Wg, then dup Wu) and the weights' gradients (both
//             operands read as they lie, tokens along K), all in one launch
//   kGluBack  dh stays in TMEM: the epilogue reads gate and up and writes dgate, dup and h
//
// The kernel is persistent; a pair of CTAs (cta_group::2) makes 256 x BN tiles.  In each CTA one
// thread fills a ring of 64-wide K stages by TMA (128-byte swizzle; a ragged edge reads as
// zeros), one thread of the leading CTA issues the products into one of two accumulators in
// TMEM, and eight warps empty the other.  Results leave by TMA from per-warp staging tiles,
// which clips them at the edges.  8192 rows, 2048 x 5632: forward 455 to 470 us (1245 to 1205 TF/s), backward
// 975 to 1025 (1165 to 1105 TF/s), bound by the tensor cores under the power limit, but for kGluBack, whose
// epilogue moves 461 MB; 12544 rows, 256 x 1024, both pre-activations kept: 41 us, bound by the epilogue.
//
// Roundings: h, dgate and dup are rounded to bf16 between the products, as the tensor cores
// take them; everything else is rounded once, on output.  gate and up are kept in bf16 for the
// backward pass, whose definition takes them so.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>

#include "srnl_common.cuh"
#include "srnl_internal.h"
#include "srnl_scan.h"
#include "srnl_tma.cuh"
#include "srnl_umma.cuh"

namespace srnl {

TensorMapEncoder ffn_tensor_map_encoder() {
  static TensorMapEncoder enc = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      enc = reinterpret_cast<TensorMapEncoder>(fn);
  });
  return enc;
}

namespace {

using bf16_t = __nv_bfloat16;

constexpr int kTileM = 256;        // rows of a pair's tile (128 per CTA)
constexpr int kTileK = 64;         // K per stage
constexpr int kEpiWarps = 8;
constexpr int kFfnThreads = 32 * (4 + kEpiWarps);
constexpr int kBox = 4096;         // a warp's staging tile: 32 rows x 64 bf16
constexpr uint32_t kABytes = 128 * kTileK * 2;

enum Epi { kPlain = 0, kGlu = 1, kGluBack = 2, kGrad = 3 };

// Staging tiles per warp and ring stages: what the epilogue has in flight against how far the
// loads run ahead, within 227 KB.
__host__ __device__ constexpr int epi_boxes(int epi) { return epi == kPlain || epi == kGrad ? 2 : 3; }
__host__ __device__ constexpr uint32_t stage_bytes(int bn) { return kABytes + (uint32_t)(bn / 2) * kTileK * 2; }
__host__ __device__ constexpr int ring_stages(int epi, int bn) {
  return (int)((226 * 1024 - 2048 - kEpiWarps * epi_boxes(epi) * kBox) / stage_bytes(bn));
}
constexpr size_t ffn_smem(int epi, int bn) {
  return 1024 + (size_t)ring_stages(epi, bn) * stage_bytes(bn) + kEpiWarps * epi_boxes(epi) * kBox + 512;   // 512: the barriers
}

struct FfnMaps {
  CUtensorMap a[5], b[4], o[4];
  CUtensorMap in[2];   // kGluBack: gate, up; kPlain: res
};

// One product of a launch: its output and operands, by their places in the maps.  Where k1 is not
// zero the sum goes on over the next two operands; a_mn: A's rows run along K in memory.
struct FfnProduct {
  int first;             // tile it begins with
  int M, N, tiles_m, tiles_n;
  int k0, k1;            // stages of the first and of the second operand pair
  int a, b, o, a_mn;
  int parts;             // K is cut into so many, each a tile of its own; one number above 1 in a launch
  int slot;              // tiles of cut products before its own
};

struct FfnArgs {
  FfnProduct product[4];
  int products, tiles;
  int slots;             // tiles of cut products
  int save, res;         // kGlu: gate and up are kept; kPlain: in[0] is added
  const bf16_t* res_at;  // the same as in[0]
  float* partial;        // the sums of a cut product's parts: [tile][CTA][warp][part][32 rows x columns]
  unsigned* arrived;     // [tile][CTA][warp], zeros between launches
  int* err;
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 same(float v) { return make_float2(v, v); }

// act(v) and its derivative for two values.  The epilogues are bound by the instructions they
// issue, so the arithmetic goes in pairs and both activations need one exponential and one
// reciprocal a value.  GELU's Phi(-z) for z >= 0 is exp(-z^2 / 2) times a polynomial in
// t = 1 / (1 + p z) without a constant term, fitted to erfc(z / sqrt 2) / 2 for the least relative
// error over 0 <= z <= 13.3 (a linear program over a grid, for each p): under 4e-6 of the value
// everywhere, against 2^-9 of the bf16 that it is rounded to.  Phi(z) is one minus that; the lower
// tail is taken as it is, since 1 - (1 - Phi(-z)) would leave nothing of it (v = -5: tens of percent).
// Below -13.2 the exponential is under fp32's normal numbers and GELU is zero, as SiLU is below -87.3.
// Projections of 12544 x 256 x 1024 with both pre-activations kept: 51 us with erff, 34 us value by
// value, 30 us so.
template <int ACT>
__device__ __forceinline__ void activation(float2 v, float2& f, float2& df) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (ACT == SRNL_ACT_SILU) {
    const float2 x = __fmul2_rn(v, same(-kLog2e));
    const float2 d = __fadd2_rn(make_float2(exp2_approx(x.x), exp2_approx(x.y)), same(1.f));
    const float2 p = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    f = __fmul2_rn(v, p);
    df = __ffma2_rn(f, __ffma2_rn(p, same(-1.f), same(1.f)), p);
  } else {
    const float2 z = make_float2(fabsf(v.x), fabsf(v.y));
    const float2 d = __ffma2_rn(z, same(0.30744928730f), same(1.f));
    const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    const float2 x = __fmul2_rn(__fmul2_rn(v, v), same(-0.5f * kLog2e));
    const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
    float2 c = __ffma2_rn(t, same(-0.07599032306f), same(0.19261357328f));
    c = __ffma2_rn(t, c, same(0.00438559623f));
    c = __ffma2_rn(t, c, same(0.13768646389f));
    c = __ffma2_rn(t, c, same(0.11837624300f));
    c = __ffma2_rn(t, c, same(0.12292661570f));
    c = __fmul2_rn(__fmul2_rn(t, c), e);                 // Phi(-|v|)
    const float2 r = __ffma2_rn(c, same(-1.f), same(1.f));
    const float2 p = make_float2(v.x < 0.f ? c.x : r.x, v.y < 0.f ? c.y : r.y);
    f = __fmul2_rn(v, p);
    df = __ffma2_rn(__fmul2_rn(v, same(0.3989422804014327f)), e, p);
  }
}

// A launch's tiles product by product; a product's in bands of 8 along M, M fastest within a
// band: the pairs that run together share their operands' rows in L2.
struct Tile {
  int tm, tn, n, part;   // n: its number in the product
};
template <int EPI, bool CUT>
__device__ __forceinline__ const FfnProduct& tile_of(int t, const FfnArgs& args, Tile& tile) {
  constexpr int kBand = 8;
  int i = 0;
  if (EPI == kGrad)
    while (i + 1 < args.products && t >= args.product[i + 1].first) ++i;
  const FfnProduct& p = args.product[i];
  t -= p.first;
  tile.part = 0;
  if (CUT && p.parts > 1) {
    tile.part = t % p.parts;
    t /= p.parts;
  }
  tile.n = t;
  const int band = t / (kBand * p.tiles_n), first = band * kBand;
  const int rows = min(kBand, p.tiles_m - first), in = t - band * kBand * p.tiles_n;
  tile.tm = first + in % rows;
  tile.tn = in / rows;
  return p;
}

// The stage that a part of a cut product begins with.
template <bool CUT>
__device__ __forceinline__ int stage_of(const FfnProduct& p, int part) {
  return CUT ? (p.k0 + p.k1) * part / p.parts : part ? p.k0 + p.k1 : 0;
}

// B lies K-major forward (weights' rows along K) and MN-major backward.  A lies K-major but for the
// weights' gradients, which share a launch (kGrad) with the input's.  CUT: the K of some products
// comes in parts; a kernel of its own, since the others lost 6 us at 1531 x 520 x 1384 to code that
// they do not run.
template <int EPI, int ACT, int BN, bool CUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFfnThreads, 1)
    ffn_product_kernel(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnArgs args) {
  constexpr bool BMN = EPI == kGluBack || EPI == kGrad;
  constexpr int S = ring_stages(EPI, BN);
  constexpr uint32_t kStage = stage_bytes(BN);
  constexpr int kBRows = BN / 2;   // of B per CTA
  constexpr int kHalf = BN / 2;    // accumulator columns per epilogue half
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* boxes = smem + S * kStage;
  unsigned long long* bars = reinterpret_cast<unsigned long long*>(boxes + kEpiWarps * epi_boxes(EPI) * kBox);
  unsigned long long *full = bars, *empty = bars + S, *tfull = bars + 2 * S, *tempty = bars + 2 * S + 2;
  unsigned long long* inbar = bars + 2 * S + 4;   // kGluBack: [warp][2], gate and up have arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(inbar + 2 * kEpiWarps);
  int* failed = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = args.tiles;

  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    *failed = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(&inbar[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  // Launched while the kernel before may still run: everything above touches only this CTA.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1u;   // the ring starts empty
      const uint32_t lead = map_rank(smem_u32(full), 0), ring = smem_u32(smem);
      for (int t = pair; t < tiles; t += pairs) {
        Tile T;
        const FfnProduct& P = tile_of<EPI, CUT>(t, args, T);
        const int k0 = P.k0, end = stage_of<CUT>(P, T.part + 1);
        const bool a_mn = EPI == kGrad && P.a_mn;
        const int m0 = T.tm * kTileM + (int)rank * 128;
        const int n0 = EPI == kGlu ? T.tn * (BN / 2) : T.tn * BN + (int)rank * kBRows;
        for (int it = stage_of<CUT>(P, T.part); it < end; ++it) {
          const int two = it >= k0;
          const int k = (it - (two ? k0 : 0)) * kTileK;
          const CUtensorMap* am = &maps.a[P.a + two];
          const CUtensorMap* bm = &maps.b[EPI == kGlu ? (int)rank : P.b + two];
          if (!mbar_pass(&empty[s], ph, failed)) break;
          if (rank == 0) mbar_expect(&full[s], 2 * kStage);
          const uint32_t bar = lead + (uint32_t)s * 8, as = ring + s * kStage, bs = as + kABytes;
          if (a_mn) {
#pragma unroll
            for (int i = 0; i < 2; ++i) tma_load_pair(as + i * 8192, am, m0 + 64 * i, k, bar);
          } else {
            tma_load_pair(as, am, k, m0, bar);
          }
          if constexpr (BMN) {
#pragma unroll
            for (int i = 0; i < kBRows / 64; ++i) tma_load_pair(bs + i * 8192, bm, n0 + 64 * i, k, bar);
          } else {
            tma_load_pair(bs, bm, k, n0, bar);
          }
          if (++s == S) { s = 0; ph ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      int s = 0, buf = 0;
      uint32_t ph = 0u, tph = 1u;   // the accumulators start empty
      const uint32_t ring = smem_u32(smem);
      const uint64_t bd0 = BMN ? desc_mn_major(ring + kABytes, 8192) : desc_k_major(ring + kABytes);
      for (int t = pair; t < tiles; t += pairs) {
        Tile T;
        const FfnProduct& P = tile_of<EPI, CUT>(t, args, T);
        const int ktot = stage_of<CUT>(P, T.part + 1) - stage_of<CUT>(P, T.part);
        const bool a_mn = EPI == kGrad && P.a_mn;
        const uint32_t idesc = a_mn ? idesc_mn(kTileM, BN, true, BMN) : idesc_mn(kTileM, BN, false, BMN);
        const uint64_t ad0 = a_mn ? desc_mn_major(ring, 8192) : desc_k_major(ring), astep = a_mn ? 128 : 2;
        mbar_pass(&tempty[buf], tph, failed);
        tmem_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * BN);
        for (int it = 0; it < ktot; ++it) {
          if (!mbar_pass(&full[s], ph, failed)) break;
          tmem_fence_after();
          const uint64_t ad = ad0 + (uint64_t)(s * (kStage >> 4)), bd = bd0 + (uint64_t)(s * (kStage >> 4));
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)
            mma_pair(acc, ad + k * astep, bd + (uint64_t)(k * (BMN ? 2048 : 32) >> 4),
                     idesc, it > 0 || k > 0);
          mma_commit_pair(&empty[s]);
          if (++s == S) { s = 0; ph ^= 1u; }
        }
        mma_commit_pair(&tfull[buf]);
        if (++buf == 2) { buf = 0; tph ^= 1u; }
      }
    }
  } else if (warp >= 4) {
    const int ew = warp - 4, quarter = ew & 3, half = ew >> 2;
    unsigned char* box = boxes + ew * epi_boxes(EPI) * kBox;
    const uint32_t done = map_rank(smem_u32(tempty), 0);
    int buf = 0, turn = 0;
    uint32_t ph = 0u;
    // bf16 pairs of 32 columns into a staging tile's columns 32 c .. : 16-byte units, swizzled as
    // its map has it (rows of 128 bytes, or of 64 in the 32-column tiles)
    constexpr bool kNarrow = EPI == kGlu;
    auto stage32 = [&](unsigned char* b, int c, const uint32_t (&w)[16]) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(kNarrow ? b + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)
                                          : b + lane * 128 + (((4 * c + j) ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    };
    // kGluBack and kPlain work in pieces of 32 rows, of 32 columns (2 KB tiles, 64-byte swizzle) and
    // 64.  What a piece reads, gate and up or the residual, arrives by TMA a piece ahead; the results
    // (dgate and dup; the sum) are written over it and leave by TMA, h beside them.
    constexpr int kCols = EPI == kGluBack ? 32 : 64, kPieces = kHalf / kCols, kPiece = kCols * 64;
    constexpr int kBuf = (EPI == kGluBack ? 3 : 1) * kPiece;
    const bool reads = EPI == kGluBack || (EPI == kPlain && !CUT && args.res != 0);
    unsigned long long* mybar = inbar + 2 * ew;
    auto fetch = [&](int t, int c, int b) {   // lane 0: piece c of tile t into buffer b
      Tile T;
      tile_of<EPI, CUT>(t, args, T);
      const int row = T.tm * kTileM + (int)rank * 128 + quarter * 32, col = T.tn * BN + half * kHalf + kCols * c;
      mbar_expect(&mybar[b], (EPI == kGluBack ? 2 : 1) * kPiece);
      for (int i = 0; i < (EPI == kGluBack ? 2 : 1); ++i)
        tma_load_own(smem_u32(box + b * kBuf + i * kPiece), &maps.in[i], col, row, &mybar[b]);
    };
    int piece = 0;   // pieces so far: buffer piece & 1, phase (piece >> 1) & 1
    if (reads && lane == 0 && pair < tiles) fetch(pair, 0, 0);
    // before a piece: the other buffer's results have left, the next piece may come
    auto ahead = [&](int t, int c, int b) {
      if (lane == 0) {
        if (reads) {
          bulk_wait_read<0>();
          if (c + 1 < kPieces) fetch(t, c + 1, b ^ 1);
          else if (t + pairs < tiles) fetch(t + pairs, 0, b ^ 1);
        } else {
          bulk_wait_read<1>();   // nothing comes: this buffer alone has to be free
        }
      }
      __syncwarp();
    };
    for (int t = pair; t < tiles; t += pairs) {
      Tile T;
      const FfnProduct& P = tile_of<EPI, CUT>(t, args, T);
      const int tn = T.tn, row0 = T.tm * kTileM + (int)rank * 128 + quarter * 32;
      const uint32_t acc = tmem + (uint32_t)(buf * BN) + ((uint32_t)(32 * quarter) << 16);
      mbar_pass(&tfull[buf], ph, failed);
      tmem_fence_after();
      if constexpr (EPI == kGlu) {
        // this half's BN / 4 hidden channels: gate in its columns, up BN / 2 further
        constexpr int kHid = BN / 4, kTile32 = 2048;
        // 32 channels at a time through 2 KB tiles: h alone takes six of them in turn, h, gate and
        // up together one of two sets of three
#pragma unroll
        for (int c = 0; c < kHid / 32; ++c) {
          const int col = tn * (BN / 2) + half * kHid + 32 * c;
          unsigned char* b = box + turn * kTile32;
          if (lane == 0) {
            if (args.save) bulk_wait_read<1>();
            else bulk_wait_read<5>();
          }
          __syncwarp();
          float g[32], u[32];
          uint32_t w[16];
          tmem_ld32(g, acc + half * kHid + 32 * c);
          tmem_ld32(u, acc + kHalf + half * kHid + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 f, d;
            activation<ACT>(make_float2(g[2 * i], g[2 * i + 1]), f, d);
            f = __fmul2_rn(f, make_float2(u[2 * i], u[2 * i + 1]));
            w[i] = pack_bf16(f.x, f.y);
          }
          stage32(b, 0, w);
          if (args.save) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16(g[2 * i], g[2 * i + 1]);
            stage32(b + kTile32, 0, w);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16(u[2 * i], u[2 * i + 1]);
            stage32(b + 2 * kTile32, 0, w);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (col < P.N && row0 < P.M)
              for (int o = 0; o < (args.save ? 3 : 1); ++o) tma_store(&maps.o[o], smem_u32(b + o * kTile32), col, row0);
            bulk_commit();
          }
          turn += args.save ? 3 : 1;
          if (turn == 6) turn = 0;
        }
      } else if constexpr (EPI == kGluBack) {
#pragma unroll 1
        for (int c = 0; c < kPieces; ++c, ++piece) {
          const int b = piece & 1, col = tn * BN + half * kHalf + 32 * c;
          unsigned char* at = box + b * 3 * kPiece;
          ahead(t, c, b);
          float v[32];
          tmem_ld32(v, acc + half * kHalf + 32 * c);
          mbar_pass(&mybar[b], (piece >> 1) & 1, failed);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            unsigned char* p = at + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4);
            const uint4 g4 = *reinterpret_cast<const uint4*>(p), u4 = *reinterpret_cast<const uint4*>(p + kPiece);
            const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
            uint32_t dg[4], du[4], hh[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = make_float2(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]), u = make_float2(bf16_lo(uw[i]), bf16_hi(uw[i]));
              float2 f, d;
              activation<ACT>(make_float2(bf16_lo(gw[i]), bf16_hi(gw[i])), f, d);
              d = __fmul2_rn(__fmul2_rn(x, u), d);
              dg[i] = pack_bf16(d.x, d.y);
              d = __fmul2_rn(x, f);
              du[i] = pack_bf16(d.x, d.y);
              f = __fmul2_rn(f, u);
              hh[i] = pack_bf16(f.x, f.y);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
            *reinterpret_cast<uint4*>(p + kPiece) = make_uint4(du[0], du[1], du[2], du[3]);
            *reinterpret_cast<uint4*>(p + 2 * kPiece) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (col < P.N && row0 < P.M)
              for (int o = 0; o < 3; ++o) tma_store(&maps.o[o], smem_u32(at + o * kPiece), col, row0);
            bulk_commit();
          }
        }
      } else {
        // of a cut product: this part's sums go to memory; who comes last adds up all parts, in
        // their order, and goes on with the sum
        const bool cut = CUT && P.parts > 1;
        const int64_t slot = ((int64_t)(P.slot + T.n) * 2 + rank) * kEpiWarps + ew;
        float4* mine = reinterpret_cast<float4*>(args.partial + slot * P.parts * (32 * kHalf)) + lane;
        constexpr int kPart = 32 * kHalf / 4;
        bool finish = true;
        if (cut) {
          finish = false;
          if (row0 < P.M) {
#pragma unroll 1
            for (int c = 0; c < kHalf / 32; ++c) {
              float v[32];
              tmem_ld32(v, acc + half * kHalf + 32 * c);
              tmem_wait_ld();
              if (row0 + lane < P.M)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  mine[T.part * kPart + (c * 8 + j) * 32] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
            __threadfence();
            __syncwarp();
            unsigned before = 0;
            if (lane == 0) before = atomicAdd(&args.arrived[slot], 1u);
            finish = __shfl_sync(0xFFFFFFFFu, before, 0) == (unsigned)P.parts - 1;
            if (finish) {
              __threadfence();
              if (lane == 0) args.arrived[slot] = 0;
            }
          }
        }
#pragma unroll 1
        for (int c = 0; c < kPieces && finish; ++c, ++piece) {
          const int b = piece & 1, col = tn * BN + half * kHalf + 64 * c;
          unsigned char* at = box + b * kBuf;
          ahead(t, c, b);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v[32];
            uint32_t w[16];
            if (!cut) {
              tmem_ld32(v, acc + half * kHalf + 64 * c + 32 * k);
              if (reads && k == 0) mbar_pass(&mybar[b], (piece >> 1) & 1, failed);
              tmem_wait_ld();
            } else {
              const bool on = row0 + lane < P.M;
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.f;
              if (on) {
                const float4* from = mine + (2 * c + k) * 8 * 32;
#pragma unroll 2
                for (int p = 0; p < P.parts; ++p, from += kPart) {
                  float4 x[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j) x[j] = __ldcg(from + j * 32);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    v[4 * j] += x[j].x; v[4 * j + 1] += x[j].y; v[4 * j + 2] += x[j].z; v[4 * j + 3] += x[j].w;
                  }
                }
                if (EPI == kPlain && args.res) {
                  const bf16_t* r = args.res_at + (int64_t)(row0 + lane) * P.N + col + 32 * k;
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (col + 32 * k + 8 * j < P.N) {
                      const uint4 q = *reinterpret_cast<const uint4*>(r + 8 * j);
                      const uint32_t rw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                      for (int i = 0; i < 4; ++i) {
                        v[8 * j + 2 * i] += bf16_lo(rw[i]);
                        v[8 * j + 2 * i + 1] += bf16_hi(rw[i]);
                      }
                    }
                }
              }
            }
            if (reads) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 r4 = *reinterpret_cast<const uint4*>(at + lane * 128 + (((4 * k + j) ^ (lane & 7)) << 4));
                const uint32_t r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  v[8 * j + 2 * i] += bf16_lo(r[i]);
                  v[8 * j + 2 * i + 1] += bf16_hi(r[i]);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            stage32(at, k, w);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (col < P.N && row0 < P.M) tma_store(&maps.o[P.o], smem_u32(at), col, row0);
            bulk_commit();
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(done + (uint32_t)buf * 8);
      if (++buf == 2) { buf = 0; ph ^= 1u; }
    }
    if (lane == 0) bulk_wait_all();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(failed)) {   // a wait gave up: let the copies in flight land, then report
    if (threadIdx.x == 0) atomicExch(args.err, SRNL_E_TIMEOUT);
    const unsigned long long t0 = global_ns();
    for (int i = 0; i < (1 << 20) && global_ns() - t0 < 1000000ull; ++i) {}
  }
  cluster_sync();   // neither CTA leaves while the other may still signal it
  if (warp == 2) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ------------------------------------------------------------------ few rows
// A handful of rows, as in serving one token of each sequence: the time is the weights' bytes,
// so the kernels are built to stream them.  Weights' rows are the left operand of m16n8k16, the
// tokens its columns: 8 rows of Wg and the same 8 of Wu in the first kernel, 16 of Wd in the
// second; a block's warps split K.  A sum over K may run in any order, so a lane takes 8
// consecutive values of K in one 16-byte load of each row and the two products of a 32-wide piece
// use them as they lie; the tokens are loaded by the same rule, and nothing passes through shared
// memory but the warps' sums.  Small blocks (8 channels; 5 to an SM) come out even over the SMs:
// 5632 channels are 704 of them.  4 rows, 2048 x 5632 (69 MB): 16.8 us, 4.1 TB/s; 32 rows: 34 us, where
// the tiles' kernel takes 35.
constexpr int kFewRows = 32;

__device__ __forceinline__ uint4 load_once(const bf16_t* p) {   // weights are met once: not kept in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void mma_rows(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// GLU: out = act(x W^T) * (x W2^T), 8 channels a block, and the two products themselves where
// asked; else out = x W^T (+ res), 16 channels.  NT: columns of 8 tokens; U: 32-wide pieces of K
// in flight.
template <bool GLU> __host__ __device__ constexpr int few_warps() { return GLU ? 8 : 16; }

template <bool GLU, int ACT, int NT>
__global__ void __launch_bounds__(few_warps<GLU>() * 32, GLU && NT == 1 ? 5 : 2)
    ffn_few_rows_kernel(const bf16_t* __restrict__ x, const bf16_t* __restrict__ W, const bf16_t* __restrict__ W2,
                        const bf16_t* __restrict__ res, bf16_t* __restrict__ out, bf16_t* __restrict__ gate,
                        bf16_t* __restrict__ up, int rows, int N, int K) {
  constexpr int kWarps = few_warps<GLU>(), U = GLU ? 2 : NT == 4 ? 2 : 4;
  __shared__ float part[kWarps][16][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, kk = (lane & 3) * 8;
  const int n0 = blockIdx.x * (GLU ? 8 : 16);
  // the lane's two rows of the left operand
  const bool on0 = n0 + g < N, on1 = GLU ? on0 : n0 + g + 8 < N;
  const bf16_t *w0 = W + (int64_t)(n0 + g) * K, *w1 = GLU ? W2 + (int64_t)(n0 + g) * K : W + (int64_t)(n0 + g + 8) * K;
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 a[U][2], b[U][NT];
  auto weights = [&](int u, int k) {
    a[u][0] = k < K && on0 ? load_once(w0 + k) : zero;
    a[u][1] = k < K && on1 ? load_once(w1 + k) : zero;
  };
  // the second kernel's first weights come while the first one ends: that one waited for all before
  // it, so nothing writes them any more (4 rows, 2048 x 5632: 17.7 -> 16.7 us; at 16 rows the
  // registers do not suffice, and it cost 2 us)
  constexpr bool kEarly = !GLU && NT == 1;
  if constexpr (kEarly)
#pragma unroll
    for (int u = 0; u < U; ++u) weights(u, (warp + u * kWarps) * 32 + kk);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  for (int k0 = warp * 32; k0 < K; k0 += kWarps * 32 * U) {   // the same passes in every lane: the products are the warp's
    if constexpr (NT == 1) {   // all of them before the tokens, which L1 holds
      if (!kEarly || k0 != warp * 32)
#pragma unroll
        for (int u = 0; u < U; ++u) weights(u, k0 + u * kWarps * 32 + kk);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kWarps * 32 + kk;
      if constexpr (NT > 1) weights(u, k);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = t * 8 + g;
        b[u][t] = k < K && r < rows ? *reinterpret_cast<const uint4*>(x + (int64_t)r * K + k) : zero;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_rows(acc[t], a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y, b[u][t].x, b[u][t].y);
        mma_rows(acc[t], a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w, b[u][t].z, b[u][t].w);
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][g + (e >> 1) * 8][t * 8 + (lane & 3) * 2 + (e & 1)] = acc[t][e];
  __syncthreads();
  constexpr int kChan = GLU ? 8 : 16;
  for (int i = threadIdx.x; i < kChan * rows; i += kWarps * 32) {
    const int c = i % kChan, r = i / kChan, n = n0 + c;
    if (n >= N) continue;
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      v += part[w][c][r];
      if (GLU) u += part[w][c + 8][r];
    }
    const int64_t at = (int64_t)r * N + n;
    if constexpr (GLU) {
      float2 f, d;
      activation<ACT>(make_float2(v, v), f, d);
      out[at] = __float2bfloat16_rn(f.x * u);
      if (gate != nullptr) {
        gate[at] = __float2bfloat16_rn(v);
        up[at] = __float2bfloat16_rn(u);
      }
    } else {
      out[at] = __float2bfloat16_rn(res != nullptr ? v + __bfloat162float(res[at]) : v);
    }
  }
}

// ------------------------------------------------------------------ host side
// bf16 [outer][inner] row-major, boxes of `cols` inner values (64: 128-byte swizzle, 32: 64-byte)
// x `rows`.
bool ffn_map(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, int rows, int cols = 64) {
  const TensorMapEncoder enc = ffn_tensor_map_encoder();
  const cuuint64_t dim[2] = {(cuuint64_t)inner, (cuuint64_t)outer}, str[1] = {(cuuint64_t)inner * 2};
  const cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)rows}, est[2] = {1u, 1u};
  return enc != nullptr &&
         enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dim, str, box, est,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int ceil_div(int64_t a, int b) { return (int)((a + b - 1) / b); }

// Launch that may begin while the kernel before on the stream runs out; the kernel itself waits
// for that one's results (griddepcontrol.wait) before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
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

template <int EPI, int ACT>
cudaError_t launch_product(int bn, const FfnMaps& maps, const FfnArgs& a, int sms, cudaStream_t s) {
  const int pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
  const dim3 grid(2 * pairs);
  if constexpr (EPI == kPlain || EPI == kGrad) {
    if (a.slots > 0)
      return bn == 256 ? launch_after(ffn_product_kernel<EPI, ACT, 256, true>, grid, kFfnThreads, ffn_smem(EPI, 256), s, maps, a)
                       : launch_after(ffn_product_kernel<EPI, ACT, 128, true>, grid, kFfnThreads, ffn_smem(EPI, 128), s, maps, a);
  }
  return bn == 256 ? launch_after(ffn_product_kernel<EPI, ACT, 256, false>, grid, kFfnThreads, ffn_smem(EPI, 256), s, maps, a)
                   : launch_after(ffn_product_kernel<EPI, ACT, 128, false>, grid, kFfnThreads, ffn_smem(EPI, 128), s, maps, a);
}

template <int EPI, int ACT, bool CUT = false>
cudaError_t prepare_product() {
  constexpr cudaFuncAttribute kSmem = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(ffn_product_kernel<EPI, ACT, 256, CUT>, kSmem, (int)ffn_smem(EPI, 256));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(ffn_product_kernel<EPI, ACT, 128, CUT>, kSmem, (int)ffn_smem(EPI, 128));
  return e;
}

// One more product of a launch, its tiles after those before it.  cols: columns of its tiles.
void add_product(FfnArgs& a, int64_t M, int64_t N, int cols, int64_t K, bool two, int am, int bm, int om, bool a_mn,
                 int parts = 1) {
  FfnProduct& p = a.product[a.products++];
  p.first = a.tiles;
  p.M = (int)M; p.N = (int)N;
  p.tiles_m = ceil_div(M, kTileM); p.tiles_n = ceil_div(N, cols);
  p.k0 = ceil_div(K, kTileK); p.k1 = two ? p.k0 : 0;
  p.a = am; p.b = bm; p.o = om; p.a_mn = a_mn;
  p.parts = parts;
  p.slot = a.slots;
  if (parts > 1) a.slots += p.tiles_m * p.tiles_n;
  a.tiles += p.tiles_m * p.tiles_n * parts;
}

// Most stages that a pair of CTAs has in a launch.  Tiles go to the pairs in turn: each pair has
// n / pairs of a product's n, and one more from where the product begins, around the pairs; the
// busiest is one that some product begins with.
int64_t longest_pair(const FfnArgs& a, int pairs) {
  int64_t all = 0, most = 0;
  for (int i = 0; i < a.products; ++i) {
    const FfnProduct& p = a.product[i];
    all += (int64_t)(p.tiles_m * p.tiles_n * p.parts / pairs) * ceil_div(p.k0 + p.k1, p.parts);
    int64_t more = 0;
    for (int j = 0; j < a.products; ++j) {
      const FfnProduct& q = a.product[j];
      const int from = (p.first - q.first) % pairs, n = q.tiles_m * q.tiles_n * q.parts % pairs;
      if ((from < 0 ? from + pairs : from) < n) more += ceil_div(q.k0 + q.k1, q.parts);
    }
    most = more > most ? more : most;
  }
  return all + most;
}

// Parts that K may come in, and what a cut costs, in stages of a 256-column tile: in any case, and
// for each part of such a tile.
constexpr int kParts[] = {2, 3, 4, 6, 8, 12, 16}, kCutStages = 12, kPartStages = 3;

template <bool GLU, int ACT>
cudaError_t launch_few_rows(const bf16_t* x, const bf16_t* W, const bf16_t* W2, const bf16_t* res, bf16_t* out, bf16_t* gate,
                            bf16_t* up, int rows, int N, int K, cudaStream_t s) {
  const dim3 grid((unsigned)(GLU ? (N + 7) / 8 : (N + 15) / 16));
  const int t = few_warps<GLU>() * 32;
  if (rows <= 8) return launch_after(ffn_few_rows_kernel<GLU, ACT, 1>, grid, t, 0, s, x, W, W2, res, out, gate, up, rows, N, K);
  if (rows <= 16) return launch_after(ffn_few_rows_kernel<GLU, ACT, 2>, grid, t, 0, s, x, W, W2, res, out, gate, up, rows, N, K);
  return launch_after(ffn_few_rows_kernel<GLU, ACT, 4>, grid, t, 0, s, x, W, W2, res, out, gate, up, rows, N, K);
}

// Columns of the pairs' tiles: 256, or 128 where that fills the SMs better (`wide`, `narrow`: the
// launch either way).  A 128-column tile reads as much of A for half the work.  It takes about 0.85
// of a 256-column one where the rounds of tiles follow one another (8192 x 2048 x 11264: 409 us in
// 7 rounds of them, 259 us in 4) and two thirds in a single round (512 x 5632 x 2048, with the
// projections before it: 58 us against 65; 1024 rows: 70 us, against 74 in 256 columns and two
// parts).  Where K is short and the epilogue counts, narrow tiles lose as much (projections and hidden
// gradients in 256 against 128 columns, GELU: forward of 12544 x 256 x 1024 35 us against 39, both
// pre-activations kept 41 against 47, backward 81 against 84; of 25088 rows 57, 71, 137 against 71, 86, 142;
// 50176 x 128 x 512 51, 64, 130 against 62, 77, 133).
int64_t launch_cost(const FfnArgs& a, int bn, int sms) {
  return (bn == 256 ? 12 : a.tiles <= sms / 2 ? 8 : 10) * longest_pair(a, sms / 2);
}
int pick_bn(const FfnArgs& wide, const FfnArgs& narrow, int sms) {
  return launch_cost(narrow, 128, sms) < launch_cost(wide, 256, sms) ? 128 : 256;
}

// Fewest stages of a cut product.
int least_stages(const FfnArgs& a) {
  int k = INT_MAX;
  for (int i = 0; i < a.products; ++i)
    if (a.product[i].parts > 1 && a.product[i].k0 + a.product[i].k1 < k) k = a.product[i].k0 + a.product[i].k1;
  return k;
}

// The launch `build(cols, what, parts)` with the columns and the parts of K that take least; `what`:
// the group of products that is cut, of `groups`.  A long sum over few tiles leaves most SMs idle; a
// cut one pays for its partial sums, which go through L2 and are added up by whoever comes last
// (output product of 2048 x 5632, 64 rows, with the projections before it: 44 us uncut, 39, 36.5 and
// 35.5 in 2, 3 and 4 parts; of 520 x 1384, 22 stages: 15.6 uncut, 16.5 in 2; the weights' gradients of
// 12544 x 256 x 1024, in the whole backward pass: 96 us uncut, 76 to 81).
template <typename Build>
FfnArgs pick_launch(int sms, int groups, int& bn, const Build& build) {
  FfnArgs best{};
  int64_t least = INT64_MAX;
  const auto take = [&](const FfnArgs& a, int cols, int64_t cost) {
    if (cost >= least) return;
    least = cost;
    best = a;
    bn = cols;
  };
  for (int cols = 256; cols >= 128; cols -= 128) {
    const FfnArgs a = build(cols, 0, 1);
    take(a, cols, launch_cost(a, cols, sms));
  }
  for (int cols = 256; cols >= 128; cols -= 128)
    for (int what = 0; what < groups; ++what)
      for (const int parts : kParts) {
        if (least <= 12 * (kCutStages + kPartStages)) return best;   // no cut costs less
        const FfnArgs a = build(cols, what, parts);
        if (a.slots * parts > sms / 2 || least_stages(a) < parts) break;   // the workspace; no part is empty
        take(a, cols, launch_cost(a, cols, sms) + 12 * (kCutStages + kPartStages * parts * cols / 256));
      }
  return best;
}

}  // namespace
}  // namespace srnl

// ------------------------------------------------------------------ C ABI
struct srnl_ffn {
  srnl_ffn_config cfg{};
  int device = 0, sms = 0;
  // workspace, bf16 [max_rows][hidden]: the branch's hidden rows; in training also dgate, dup
  __nv_bfloat16 *hid = nullptr, *dgate = nullptr, *dup = nullptr;
  float* partial = nullptr;       // a tile of 256 x 256 sums for each pair of SMs
  unsigned* arrived = nullptr;    // a counter for each of their warps
  int* dev_err = nullptr;
  char err[256] = "";
};

namespace {

using bf16 = __nv_bfloat16;
thread_local char g_ffn_create_error[256] = "";

srnl_status ffn_fail(srnl_ffn* h, srnl_status st, const char* msg) {
  snprintf(h != nullptr ? h->err : g_ffn_create_error, 256, "%s", msg);
  return st;
}

srnl_status ffn_cuda_fail(srnl_ffn* h, cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return ffn_fail(h, e == cudaErrorMemoryAllocation ? SRNL_E_NOMEM : SRNL_E_CUDA, msg);
}

void ffn_free(srnl_ffn* h) {
  void* ptrs[] = {h->hid, h->dgate, h->dup, h->partial, h->arrived, h->dev_err};
  for (void* p : ptrs)
    if (p != nullptr) cudaFree(p);
}

struct Span {
  const void* p;
  size_t n;
  const char* name;
};

// Alignment of every given buffer, and no output over an input or another output.
srnl_status ffn_check(srnl_ffn* h, const Span* in, int ni, const Span* out, int no) {
  char msg[256];
  auto over = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && x < y + b.n && y < x + a.n;
  };
  for (int i = 0; i < ni + no; ++i) {
    const Span& s = i < ni ? in[i] : out[i - ni];
    if (reinterpret_cast<uintptr_t>(s.p) & 15u) {
      snprintf(msg, sizeof msg, "%s must be 16-byte aligned", s.name);
      return ffn_fail(h, SRNL_E_INVAL, msg);
    }
  }
  for (int i = 0; i < no; ++i)
    for (int j = 0; j < ni + i; ++j) {
      const Span& s = j < ni ? in[j] : out[j - ni];
      if (over(out[i], s)) {
        snprintf(msg, sizeof msg, "%s overlaps %s", out[i].name, s.name);
        return ffn_fail(h, SRNL_E_INVAL, msg);
      }
    }
  int cur = -1;
  const cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return ffn_cuda_fail(h, e, "cudaGetDevice");
  if (cur != h->device) return ffn_fail(h, SRNL_E_INVAL, "the current device is not the handle's device");
  return SRNL_OK;
}

}  // namespace

extern "C" {

srnl_status srnl_ffn_create(srnl_ffn** out, const srnl_ffn_config* cfg) {
  using namespace srnl;
  if (out == nullptr) return ffn_fail(nullptr, SRNL_E_INVAL, "out is NULL");
  *out = nullptr;
  if (cfg == nullptr) return ffn_fail(nullptr, SRNL_E_INVAL, "cfg is NULL");
  if (cfg->dim <= 0 || cfg->hidden <= 0 || cfg->max_rows <= 0)
    return ffn_fail(nullptr, SRNL_E_INVAL, "dim, hidden and max_rows must be positive");
  if (cfg->activation != SRNL_ACT_SILU && cfg->activation != SRNL_ACT_GELU)
    return ffn_fail(nullptr, SRNL_E_INVAL, "activation must be SRNL_ACT_SILU or SRNL_ACT_GELU");
  if (cfg->act_dtype != SRNL_BF16) return ffn_fail(nullptr, SRNL_E_UNSUPPORTED, "the branch takes bf16 activations");
  if (cfg->dim % 8 != 0 || cfg->hidden % 8 != 0)
    return ffn_fail(nullptr, SRNL_E_UNSUPPORTED, "dim and hidden must be multiples of 8");
  if (cfg->dim > 65536 || cfg->hidden > 65536)
    return ffn_fail(nullptr, SRNL_E_UNSUPPORTED, "dim and hidden must be at most 65536");
  if (cfg->max_rows > (1 << 24)) return ffn_fail(nullptr, SRNL_E_UNSUPPORTED, "max_rows must be at most 2^24");
  srnl_ffn* h = new (std::nothrow) srnl_ffn;
  if (h == nullptr) return ffn_fail(nullptr, SRNL_E_NOMEM, "host allocation failed");
  h->cfg = *cfg;
  const size_t bytes = (size_t)cfg->max_rows * cfg->hidden * 2;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) e = cudaMalloc(&h->hid, bytes);
  if (e == cudaSuccess && cfg->training) e = cudaMalloc(&h->dgate, bytes);
  if (e == cudaSuccess && cfg->training) e = cudaMalloc(&h->dup, bytes);
  const size_t pairs = (size_t)(h->sms / 2);
  if (e == cudaSuccess) e = cudaMalloc(&h->partial, pairs * kTileM * 256 * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&h->arrived, pairs * 2 * kEpiWarps * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMemset(h->arrived, 0, pairs * 2 * kEpiWarps * sizeof(unsigned));
  if (e == cudaSuccess) e = cudaMalloc(&h->dev_err, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(h->dev_err, 0, sizeof(int));
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);   // a call's stream need not wait for the one these ran on
  if (e == cudaSuccess) e = prepare_product<kGlu, SRNL_ACT_SILU>();
  if (e == cudaSuccess) e = prepare_product<kGlu, SRNL_ACT_GELU>();
  if (e == cudaSuccess) e = prepare_product<kPlain, 0>();
  if (e == cudaSuccess) e = prepare_product<kPlain, 0, true>();
  if (e == cudaSuccess) e = prepare_product<kGluBack, SRNL_ACT_SILU>();
  if (e == cudaSuccess) e = prepare_product<kGluBack, SRNL_ACT_GELU>();
  if (e == cudaSuccess) e = prepare_product<kGrad, 0>();
  if (e == cudaSuccess) e = prepare_product<kGrad, 0, true>();
  if (e == cudaSuccess && ffn_tensor_map_encoder() == nullptr) e = cudaErrorNotSupported;
  if (e != cudaSuccess) {
    const srnl_status st = ffn_cuda_fail(nullptr, e, "feed-forward create");
    ffn_free(h);
    delete h;
    return st;
  }
  *out = h;
  return SRNL_OK;
}

srnl_status srnl_ffn_forward(srnl_ffn* h, const void* x, const srnl_ffn_params* p, const void* res, void* y,
                             void* gate, void* up, int rows, void* stream) {
  using namespace srnl;
  if (h == nullptr) return ffn_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  const srnl_ffn_config& c = h->cfg;
  if (rows < 0 || rows > c.max_rows) return ffn_fail(h, SRNL_E_INVAL, "rows must be between 0 and max_rows");
  if (rows == 0) return SRNL_OK;
  if (x == nullptr || y == nullptr || p == nullptr || p->W_gate == nullptr || p->W_up == nullptr || p->W_down == nullptr)
    return ffn_fail(h, SRNL_E_INVAL, "x, y or a weight is NULL");
  if ((gate == nullptr) != (up == nullptr)) return ffn_fail(h, SRNL_E_INVAL, "gate and up are kept together or not at all");
  const int64_t M = rows, D = c.dim, F = c.hidden;
  const size_t nx = (size_t)M * D * 2, nf = (size_t)M * F * 2, nw = (size_t)D * F * 2;
  const Span in[] = {{x, nx, "x"}, {p->W_gate, nw, "W_gate"}, {p->W_up, nw, "W_up"}, {p->W_down, nw, "W_down"}, {res, nx, "res"}};
  const Span out[] = {{y, nx, "y"}, {gate, nf, "gate"}, {up, nf, "up"}};
  const srnl_status st = ffn_check(h, in, 5, out, 3);
  if (st != SRNL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows <= kFewRows) {
    const auto w = [](const void* q) { return static_cast<const bf16*>(q); };
    bf16 *gk = static_cast<bf16*>(gate), *uk = static_cast<bf16*>(up);
    cudaError_t e = c.activation == SRNL_ACT_SILU
        ? launch_few_rows<true, SRNL_ACT_SILU>(w(x), w(p->W_gate), w(p->W_up), nullptr, h->hid, gk, uk, rows, (int)F, (int)D, s)
        : launch_few_rows<true, SRNL_ACT_GELU>(w(x), w(p->W_gate), w(p->W_up), nullptr, h->hid, gk, uk, rows, (int)F, (int)D, s);
    if (e == cudaSuccess)
      e = launch_few_rows<false, 0>(h->hid, w(p->W_down), nullptr, w(res), static_cast<bf16*>(y), nullptr, nullptr, rows, (int)D, (int)F, s);
    return e == cudaSuccess ? SRNL_OK : ffn_cuda_fail(h, e, "feed-forward few-row launch");
  }
  FfnMaps m;
  memset(&m, 0, sizeof m);
  FfnArgs a[2] = {};   // tiles of 256 and of 128 columns
  for (int i = 0; i < 2; ++i) {
    add_product(a[i], M, F, 128 >> i, D, false, 0, 0, 0, false);
    a[i].save = gate != nullptr;
    a[i].err = h->dev_err;
  }
  int bn = pick_bn(a[0], a[1], h->sms);
  bool ok = ffn_map(&m.a[0], x, D, M, 128) && ffn_map(&m.b[0], p->W_gate, D, F, bn / 2) &&
            ffn_map(&m.b[1], p->W_up, D, F, bn / 2) && ffn_map(&m.o[0], h->hid, F, M, 32, 32) &&
            (gate == nullptr || (ffn_map(&m.o[1], gate, F, M, 32, 32) && ffn_map(&m.o[2], up, F, M, 32, 32)));
  if (!ok) return ffn_fail(h, SRNL_E_CUDA, "a tensor map could not be encoded");
  cudaError_t e = c.activation == SRNL_ACT_SILU ? launch_product<kGlu, SRNL_ACT_SILU>(bn, m, a[bn == 128], h->sms, s)
                                                : launch_product<kGlu, SRNL_ACT_GELU>(bn, m, a[bn == 128], h->sms, s);
  if (e != cudaSuccess) return ffn_cuda_fail(h, e, "feed-forward projections launch");
  const FfnArgs b = pick_launch(h->sms, 1, bn, [&](int cols, int, int parts) {
    FfnArgs l{};
    add_product(l, M, D, cols, F, false, 0, 0, 0, false, parts);
    l.res = res != nullptr;
    l.res_at = static_cast<const bf16*>(res);
    l.partial = h->partial;
    l.arrived = h->arrived;
    l.err = h->dev_err;
    return l;
  });
  ok = (res == nullptr || ffn_map(&m.in[0], res, D, M, 32)) && ffn_map(&m.a[0], h->hid, F, M, 128) &&
       ffn_map(&m.b[0], p->W_down, F, D, bn / 2) && ffn_map(&m.o[0], y, D, M, 32);
  if (!ok) return ffn_fail(h, SRNL_E_CUDA, "a tensor map could not be encoded");
  e = launch_product<kPlain, 0>(bn, m, b, h->sms, s);
  return e == cudaSuccess ? SRNL_OK : ffn_cuda_fail(h, e, "feed-forward output launch");
}

srnl_status srnl_ffn_backward(srnl_ffn* h, const void* x, const void* gate, const void* up, const void* dy,
                              const srnl_ffn_params* p, void* dx, const srnl_ffn_grads* grads, int rows, void* stream) {
  using namespace srnl;
  if (h == nullptr) return ffn_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  h->err[0] = 0;
  const srnl_ffn_config& c = h->cfg;
  if (!c.training) return ffn_fail(h, SRNL_E_INVAL, "the backward pass needs a handle created with training set");
  if (rows < 0 || rows > c.max_rows) return ffn_fail(h, SRNL_E_INVAL, "rows must be between 0 and max_rows");
  srnl_ffn_grads g{};
  if (grads != nullptr) g = *grads;
  const int64_t M = rows, D = c.dim, F = c.hidden;
  const size_t nx = (size_t)M * D * 2, nf = (size_t)M * F * 2, nw = (size_t)D * F * 2;
  if (rows > 0 && (x == nullptr || gate == nullptr || up == nullptr || dy == nullptr || p == nullptr ||
                   p->W_gate == nullptr || p->W_up == nullptr || p->W_down == nullptr))
    return ffn_fail(h, SRNL_E_INVAL, "x, gate, up, dy or a weight is NULL");
  srnl_ffn_params w{};
  if (p != nullptr) w = *p;
  const Span in[] = {{x, nx, "x"}, {gate, nf, "gate"}, {up, nf, "up"}, {dy, nx, "dy"},
                     {w.W_gate, nw, "W_gate"}, {w.W_up, nw, "W_up"}, {w.W_down, nw, "W_down"}};
  const Span out[] = {{dx, nx, "dx"}, {g.W_gate, nw, "grads.W_gate"}, {g.W_up, nw, "grads.W_up"}, {g.W_down, nw, "grads.W_down"}};
  const srnl_status st = ffn_check(h, in, 7, out, 4);
  if (st != SRNL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // sums over no tokens
    void* const outs[] = {g.W_gate, g.W_up, g.W_down};
    for (void* o : outs) {
      const cudaError_t e = o != nullptr ? cudaMemsetAsync(o, 0, nw, s) : cudaSuccess;
      if (e != cudaSuccess) return ffn_cuda_fail(h, e, "gradient reset");
    }
    return SRNL_OK;
  }
  if (dx == nullptr && g.W_gate == nullptr && g.W_up == nullptr && g.W_down == nullptr) return SRNL_OK;
  FfnMaps m;
  memset(&m, 0, sizeof m);
  // dgate, dup and h from dh = dy Wd
  FfnArgs a[2] = {};
  for (int i = 0; i < 2; ++i) {
    add_product(a[i], M, F, 256 >> i, D, false, 0, 0, 0, false);
    a[i].err = h->dev_err;
  }
  int bn = pick_bn(a[0], a[1], h->sms);
  bool ok = ffn_map(&m.a[0], dy, D, M, 128) && ffn_map(&m.b[0], w.W_down, F, D, 64) &&
            ffn_map(&m.o[0], h->dgate, F, M, 32, 32) && ffn_map(&m.o[1], h->dup, F, M, 32, 32) &&
            ffn_map(&m.o[2], h->hid, F, M, 32, 32) && ffn_map(&m.in[0], gate, F, M, 32, 32) && ffn_map(&m.in[1], up, F, M, 32, 32);
  if (!ok) return ffn_fail(h, SRNL_E_CUDA, "a tensor map could not be encoded");
  cudaError_t e = c.activation == SRNL_ACT_SILU ? launch_product<kGluBack, SRNL_ACT_SILU>(bn, m, a[bn == 128], h->sms, s)
                                                : launch_product<kGluBack, SRNL_ACT_GELU>(bn, m, a[bn == 128], h->sms, s);
  if (e != cudaSuccess) return ffn_cuda_fail(h, e, "feed-forward backward launch");
  // what is asked for of dx and the weights' gradients in one launch: the longest sums first, the
  // others' tiles fill up the SMs behind them
  const bool weights = g.W_gate != nullptr || g.W_up != nullptr || g.W_down != nullptr;
  const FfnArgs b = pick_launch(h->sms, 1 + (dx != nullptr && weights), bn, [&](int cols, int what, int parts) {
    FfnArgs l{};
    const int pd = dx == nullptr || what == 1 ? 1 : parts, pw = dx == nullptr || what == 1 ? parts : 1;
    if (dx != nullptr) add_product(l, M, D, cols, F, true, 0, 0, 0, false, pd);
    if (g.W_gate != nullptr) add_product(l, F, D, cols, M, false, 2, 2, 1, true, pw);
    if (g.W_up != nullptr) add_product(l, F, D, cols, M, false, 3, 2, 2, true, pw);
    if (g.W_down != nullptr) add_product(l, D, F, cols, M, false, 4, 3, 3, true, pw);
    l.partial = h->partial;
    l.arrived = h->arrived;
    l.err = h->dev_err;
    return l;
  });
  ok = ffn_map(&m.a[0], h->dgate, F, M, 128) && ffn_map(&m.a[1], h->dup, F, M, 128) && ffn_map(&m.a[2], h->dgate, F, M, 64) &&
       ffn_map(&m.a[3], h->dup, F, M, 64) && ffn_map(&m.a[4], dy, D, M, 64) && ffn_map(&m.b[0], w.W_gate, D, F, 64) &&
       ffn_map(&m.b[1], w.W_up, D, F, 64) && ffn_map(&m.b[2], x, D, M, 64) && ffn_map(&m.b[3], h->hid, F, M, 64) &&
       (dx == nullptr || ffn_map(&m.o[0], dx, D, M, 32)) && (g.W_gate == nullptr || ffn_map(&m.o[1], g.W_gate, D, F, 32)) &&
       (g.W_up == nullptr || ffn_map(&m.o[2], g.W_up, D, F, 32)) && (g.W_down == nullptr || ffn_map(&m.o[3], g.W_down, F, D, 32));
  if (!ok) return ffn_fail(h, SRNL_E_CUDA, "a tensor map could not be encoded");
  e = launch_product<kGrad, 0>(bn, m, b, h->sms, s);
  if (e != cudaSuccess) return ffn_cuda_fail(h, e, "feed-forward gradients launch");
  return SRNL_OK;
}

srnl_status srnl_ffn_device_status(srnl_ffn* h) {
  if (h == nullptr) return ffn_fail(nullptr, SRNL_E_INVAL, "handle is NULL");
  int v = 0;
  const cudaError_t e = cudaMemcpy(&v, h->dev_err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return ffn_cuda_fail(h, e, "status read");
  return v == 0 ? SRNL_OK : ffn_fail(h, static_cast<srnl_status>(v), "a bounded in-kernel wait gave up");
}

const char* srnl_ffn_last_error(const srnl_ffn* h) { return h != nullptr ? h->err : g_ffn_create_error; }

void srnl_ffn_destroy(srnl_ffn* h) {
  if (h == nullptr) return;
  int prev = -1;
  if (cudaGetDevice(&prev) == cudaSuccess && prev != h->device) cudaSetDevice(h->device);
  cudaDeviceSynchronize();
  ffn_free(h);
  if (prev >= 0 && prev != h->device) cudaSetDevice(prev);
  delete h;
}

}  // extern "C"
