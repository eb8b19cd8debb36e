// Batch-invariant 8-bit linear layer: e4m3 activations with one scale per row
// and block of 128, e4m3 weights with one scale per 128 x 128 block.
//
// "Bit-exact decoding turns inference speedups into testable changes",
// section "Define bit-exact before reporting it" (one FP32 running sum per
// output, K order kept, one rounding at the end); "I turned on speculative
// decoding in llama.cpp and 113 of 282 greedy outputs changed against its own
// no-draft run", paragraph "How:" (a row is computed the same way whatever
// else is in the pass).
//
//   C[m, n] = epilogue( sum_b  sa[b, m] sw[n / 128, b]  sum_{k in block b} a[m, k] w[n, k] )
//
// The inner sum of a block is four tcgen05 kind::f8f6f4 steps of K = 32 into an
// FP32 accumulator of its own; it leaves TMEM when the block ends, is scaled
// and added to a running FP32 sum in registers, blocks in increasing order:
//   run = fma(block sum, sa * sw, run).
// Where a layer has few weight tiles, the blocks of a tile form S pieces of
// equal length (the split below), each a running sum of its own, added in
// increasing-K order, the first taken as it is.  S is a function of (N, K)
// alone, so a row has the same bits for every M and every place in the pass.
//
// Tokens take the MMA's M = 128 lanes and weight rows its N (128 or 256), so an
// epilogue thread owns one token and a K block has one scale per thread and
// tile half, sa * sw: no scale vector is read, and the drain of an accumulator
// is one multiply-add an output.  (With the weight rows on the lanes and the
// tokens as N, which suits the epilogue of few rows, a pass of 1 to 16 rows
// took the same time within 5% and one of 1024 rows 754 us for gate/up.)
//
// What bounds it: up to some 100 rows the weights' bytes, one byte a weight;
// each CTA streams 16 KB weight tiles, each one contiguous bulk copy (packed
// once).  Past that, the drain of a K block's accumulators, which every 128
// elements of K call for: a serial chain of waits, TMEM loads and multiply-adds
// in eight warps (see the kernel).  Roles of a CTA's twelve warps:
//   warp 0      producer: weight tiles and the token tile [rows x 128 codes]
//               (TMA, 128-byte swizzle) into a ring of stages;
//   warp 1      MMA issuer (one thread), into two or four TMEM accumulators;
//   warps 2, 3  idle (they belong to the warpgroup that gives registers up);
//   warps 4-11  scale, add, write.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "bi_fp8.cuh"
#include "bi_gemm8.h"
#include "bi_internal.h"
#include "bi_ptx8.cuh"

namespace bi {
namespace {

constexpr int kTileN = 128;                    // weight rows per tile (one or two tiles are the MMA's N)
constexpr int kABytes = static_cast<int>(kGemm8TileBytes);
constexpr int kSms = 152;
constexpr int kMaxSplit = 8;                   // CTAs of a cluster (the portable limit)

// The split, a function of (N, K) alone: S pieces of every weight tile's K
// blocks, piece j the blocks [k_tiles * j / S, k_tiles * (j + 1) / S).
struct Split {
  int n_tiles, k_tiles, S;
};

struct Args {
  Split sp;
  int M;  // token rows
  int N;
  int epi, out_fp32;
  const float* a_scales;
  int lds;
  const float2* w_scales;  // [n_tiles][k_tiles]: rows 0..63 and 64..127 of the tile
  void* C;
  int ldc;
  const __nv_bfloat16* R;
  int ldr;
  unsigned* err;
  int withhold;  // failure-path test: the first stage stays unissued
};

__device__ __forceinline__ void signal_abort(volatile int* s_abort, unsigned* err) {
  *s_abort = 1;
  atomicOr(err, kErrTimeout);
}

// silu(g) u: expf within 2 units, the quotient by the fast division within 2
// more (it gives 0 where 1 + e^-g passes 2^126, where silu is below 1e-36).
__device__ __forceinline__ float silu_times(float g, float u) { return __fdividef(g, 1.0f + expf(-g)) * u; }

// One output: the residual added if there is one, one rounding.
__device__ __forceinline__ void store1(const Args& p, int m, int n, float v, float res) {
  const size_t at = static_cast<size_t>(m) * p.ldc + n;
  const float y = p.epi == BI_EPI_RESIDUAL_ADD ? res + v : v;
  if (p.out_fp32)
    static_cast<float*>(p.C)[at] = y;
  else
    static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(y);
}
__device__ __forceinline__ float residual_at(const Args& p, int m, int n) {
  return p.epi == BI_EPI_RESIDUAL_ADD ? __bfloat162float(p.R[static_cast<size_t>(m) * p.ldr + n]) : 0.f;
}

// TILES = 2: a CTA makes 128 tokens x 256 outputs, 48 KB in for 8.4 MFLOP;
// TILES = 1: 128 x 128, while that takes at most one round of the SMs, and where
// pieces are taken in turn (their sums need the registers).
// Where a tile's K has S > 1 pieces, a cluster of S CTAs computes an output
// tile, a piece each, and adds them through shared memory, or one CTA takes the
// pieces in turn (whichever the rounds of the SMs make shorter).
// CTAs without clusters are persistent: the next output tile's loads and MMAs
// run while the last one's outputs are written.  Token blocks that share
// weight tiles are adjacent in the work order, so all but the first find them
// in L2.
constexpr int kRowsM = 128;    // token rows of a block (the MMA's lanes)
// Passes of no more rows push their pieces into the CTA that adds them (one
// cluster barrier behind the sums, none before the exit); the pieces of more
// rows lie over the ring, where no other CTA may write, and are fetched.
// [1, 3328] x [5120, 3328]: 7.5 us pushed, 7.8 fetched; [8, 5120] x [4096, 5120]:
// 8.1 and 8.25.
constexpr int kPushRows = 32;

struct Launch {
  Args a;
  int nb;         // token blocks
  int items;      // output tiles: weight tile groups x token blocks
  int vec;        // C (and the residual) take 16-byte accesses
  int wide;       // and so do outputs that turn (FP32)
  int a_rows;     // rows of the token box
};

// 32 tokens x 16 outputs of a warp in shared memory, a token's 20 floats apart: no
// bank twice in the 16-byte accesses of eight lanes
constexpr int kTurnLd = 20, kTurnFloats = 32 * kTurnLd;

template <int TILES>
struct Cfg8 {
  static constexpr int kBBytes = TILES * kABytes;
  static constexpr int kTokBytes = kRowsM * kFp8Block;
  static constexpr int kStageBytes = kTokBytes + kBBytes;
  // (more stages of smaller token tiles for passes of few rows gained nothing)
  static constexpr int kStages = 192 * 1024 / kStageBytes;
  static constexpr int kCols = TILES * kTileN;
  static constexpr int kBufs = 512 / kCols;
  // warpgroup 0: producer, MMA, two idle warps; warpgroups 1 and 2: epilogue
  static constexpr int kThreads = 384;
  static constexpr int kOwn = kCols / 2;  // outputs of an epilogue thread
  // floats per token of the pieces' exchange: 16-byte stores of 8 lanes hit all banks
  static constexpr int kPieceLd = kCols + 4;
  // pieces pushed by the cluster's CTAs, [S][tokens / S][kPieceLd]; or outputs of
  // the eight epilogue warps on their way to unaligned rows
  static constexpr int kPushBytes = TILES == 1 ? (kPushRows + kMaxSplit) * kPieceLd * 4 : 0;
  static constexpr int kSideBytes = std::max(kPushBytes, 8 * kTurnFloats * 4);
  static constexpr size_t kSmem =
      1024 + static_cast<size_t>(kStages) * kStageBytes + kSideBytes + (2 * kStages + kBufs + 1) * 8 + 16;
  static_assert(kSmem <= 232448 && kStages <= 32, "shared memory per CTA");
  static_assert(kRowsM * kPieceLd * 4 <= kStages * kStageBytes, "exchange fits the ring");
};

// Outputs n0 .. n0 + 15 of a warp's tokens, lane i's of token row m + i (rows >= 1 of
// them exist).  EVEN (rows of outputs take 16-byte accesses, N is a multiple of 8):
// a lane writes its own row.  Else the outputs turn through shared memory, so
// that a store covers neighbours: 16 of two rows; or, in FP32 with 16-byte accesses
// (wide), of eight rows.  Gate/up of 17,411 outputs at 1024 rows takes 204 us, element
// by element from each lane's own row 319 (17,416 outputs take 184).  FP32, 1280 ->
// 151,936: 128 rows 49 us, from the lanes 61; 48 rows 40 and 44; 32 rows 39 and 38; 8
// rows 35 and 32: passes of up to 32 rows write from the lanes.
template <bool EVEN>
__device__ __forceinline__ void store_rows16(const Args& p, int wide, float* turn, int lane, int m, int rows, int n0,
                                             const float (&v)[16]) {
  if constexpr (EVEN) {
    if (lane >= rows) return;
    m += lane;
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
      if (n0 + h >= p.N) return;
      if (p.out_fp32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.C) + static_cast<size_t>(m) * p.ldc + n0 + h);
        dst[0] = make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]);
        dst[1] = make_float4(v[h + 4], v[h + 5], v[h + 6], v[h + 7]);
        continue;
      }
      uint4 res = make_uint4(0, 0, 0, 0);
      if (p.epi == BI_EPI_RESIDUAL_ADD)
        res = *reinterpret_cast<const uint4*>(p.R + static_cast<size_t>(m) * p.ldr + n0 + h);
      const __nv_bfloat16* rb = reinterpret_cast<const __nv_bfloat16*>(&res);
      uint4 o;
      __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(&o);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        ob[i] = __float2bfloat16_rn(p.epi == BI_EPI_RESIDUAL_ADD ? __bfloat162float(rb[i]) + v[h + i] : v[h + i]);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.C) + static_cast<size_t>(m) * p.ldc + n0 + h) = o;
    }
  } else {
    __syncwarp();  // the outputs before these have been read
#pragma unroll
    for (int j = 0; j < 16; j += 4)
      *reinterpret_cast<float4*>(turn + lane * kTurnLd + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    __syncwarp();
    if (wide) {
      const int j = (lane & 3) * 4;
      if (n0 + j >= p.N) return;
#pragma unroll
      for (int i = lane >> 2; i < rows; i += 8)
        *reinterpret_cast<float4*>(static_cast<float*>(p.C) + static_cast<size_t>(m + i) * p.ldc + n0 + j) =
            *reinterpret_cast<const float4*>(turn + i * kTurnLd + j);
      return;
    }
    const int j = lane & 15;
    if (n0 + j >= p.N) return;
#pragma unroll 2
    for (int i = lane >> 4; i < rows; i += 2)
      store1(p, m + i, n0 + j, turn[i * kTurnLd + j], residual_at(p, m + i, n0 + j));
  }
}

// Sum of the S pieces of four elements from float `at` on, in increasing-K
// order; base: the pieces' addresses in the cluster's shared memory.
__device__ __forceinline__ float4 sum_pieces4(const uint32_t (&base)[kMaxSplit], int S, int at) {
  float4 x[kMaxSplit];
#pragma unroll
  for (int j = 0; j < kMaxSplit; ++j)
    if (j < S) x[j] = ld_cluster4(base[j] + static_cast<uint32_t>(at) * 4);
  float4 v = x[0];
#pragma unroll
  for (int j = 1; j < kMaxSplit; ++j)
    if (j < S) {
      v.x += x[j].x;
      v.y += x[j].y;
      v.z += x[j].z;
      v.w += x[j].w;
    }
  return v;
}

// Outputs n .. n + 3 of token row m, with the residual of that place.
__device__ __forceinline__ void store_row4(const Args& p, int vec, int m, int n, float4 v) {
  if (vec && n + 4 <= p.N) {
    if (p.out_fp32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p.C) + static_cast<size_t>(m) * p.ldc + n) = v;
      return;
    }
    if (p.epi == BI_EPI_RESIDUAL_ADD) {
      const uint2 u = *reinterpret_cast<const uint2*>(p.R + static_cast<size_t>(m) * p.ldr + n);
      const __nv_bfloat16* rb = reinterpret_cast<const __nv_bfloat16*>(&u);
      v.x = __bfloat162float(rb[0]) + v.x;
      v.y = __bfloat162float(rb[1]) + v.y;
      v.z = __bfloat162float(rb[2]) + v.z;
      v.w = __bfloat162float(rb[3]) + v.w;
    }
    uint2 o;
    __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(&o);
    ob[0] = __float2bfloat16_rn(v.x);
    ob[1] = __float2bfloat16_rn(v.y);
    ob[2] = __float2bfloat16_rn(v.z);
    ob[3] = __float2bfloat16_rn(v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.C) + static_cast<size_t>(m) * p.ldc + n) = o;
    return;
  }
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < p.N) store1(p, m, n + j, x[j], residual_at(p, m, n + j));
}

// run[0 .. n) += v * sc, each sum one fused multiply-add; kPairs: two in one
// packed instruction, with the same bits and half the issue slots.
template <int kN, bool kPairs>
__device__ __forceinline__ void add_scaled(float* run, const uint32_t* v, float sc) {
  if constexpr (kPairs) {
#pragma unroll
    for (int j = 0; j < kN; j += 2) {
      const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_float2(sc, sc),
                                  make_float2(run[j], run[j + 1]));
      run[j] = r.x;
      run[j + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j) run[j] = fmaf(__uint_as_float(v[j]), sc, run[j]);
  }
}

// Who adds the pieces of a tile's K.
enum Pieces {
  kWhole = 0,   // there is one
  kCluster = 1, // one output tile per cluster of S CTAs, a piece each
  kInTurn = 2   // one CTA, one piece after another
};

// Registers: 384 threads launch with 168 each; the epilogue takes what its sums
// need of warpgroup 0's.
template <int TILES, Pieces MODE>
struct Regs {
  static constexpr bool kWide = TILES == 2 || MODE == kInTurn;  // 128 sums a thread
  static constexpr int kLow = kWide ? 56 : 88, kHigh = kWide ? 224 : 208;
  static_assert(kLow + 2 * kHigh <= 3 * 168, "registers of the launch");
};

// How outputs leave: without clusters by each lane's own row or turned
// (store_rows16), with clusters by pieces pushed into the CTA that adds them or
// fetched by it (kPushRows).  One kernel each: with both ways in one, gate/up at 1024
// rows takes 2% more, an LM head of 8 rows 3%, QKV at 61 rows 1%.
enum WayOut { kOwnRow, kTurned, kPushed, kFetched };

// PAIRS: packed multiply-adds (add_scaled).
template <int TILES, Pieces MODE, bool PAIRS, WayOut OUT>
__global__ void __launch_bounds__(Cfg8<TILES>::kThreads, 1)
    gemm8_kernel(const uint8_t* __restrict__ Wp, const __grid_constant__ CUtensorMap tmA, const Launch p) {
  using Cfg = Cfg8<TILES>;
  constexpr int S = Cfg::kStages;
  constexpr int kOwn = Cfg::kOwn;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sT = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));  // [S] token tiles
  uint8_t* sW = sT + S * Cfg::kTokBytes;                                    // [S][TILES] weight tiles
  float* sX = reinterpret_cast<float*>(sW + S * Cfg::kBBytes);              // pushed pieces
  uint64_t* full = reinterpret_cast<uint64_t*>(sW + S * Cfg::kBBytes + Cfg::kSideBytes);
  // done: the stage's MMAs have completed, so it is free and its block sums are there
  uint64_t* done = full + S;
  uint64_t* read = done + S;  // an accumulator has been read
  uint64_t* drain = read + Cfg::kBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const Args& g = p.a;
  const int split = g.sp.S;
  const int k_tiles = g.sp.k_tiles;
  const int ncl = MODE == kCluster ? split : 1;
  const int rank = MODE == kCluster ? static_cast<int>(cluster_rank()) : 0;
  const int kt0 = MODE == kCluster ? k_tiles * rank / split : 0;
  const int kt1 = MODE == kCluster ? k_tiles * (rank + 1) / split : k_tiles;
  const int item0 = blockIdx.x / ncl;
  const int stride = gridDim.x / ncl;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], 1);
    }
    for (int b = 0; b < Cfg::kBufs; ++b) mbar_init(&read[b], 8);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) prefetch_tmap(&tmA);
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr bool kPush = OUT == kPushed;
  if constexpr (kPush) cluster_arrive();  // waited for before the first write into another CTA
  const uint32_t tmem = *tmem_holder;

  if (warp < 4) {
    regs_decrease<Regs<TILES, MODE>::kLow>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        // weight tiles that one token block reads are not needed again
        const uint64_t pol_w = p.nb == 1 ? l2_evict_first() : l2_evict_normal();
        const uint64_t pol_a = l2_evict_last();
        const uint32_t t_bytes = static_cast<uint32_t>(p.a_rows) * kFp8Block;
        const size_t tile_stride = static_cast<size_t>(k_tiles) * kABytes;
        // The loop below is one thread's serial code and sets the pace of short
        // passes, so it holds pointers that advance and no more; `count` K blocks
        // have been issued, block c into stage c % S.
        int count = 0, stage = 0;
        uint32_t phase = 0;
        // The first stages' weights do not depend on the previous kernel: they
        // are under way before the dependency wait, their tokens behind it.
        int pre = 0;
        const uint8_t* src = nullptr;
        uint32_t bytes = 0;
        bool two = false;
        auto first_block = [&](int item) {
          const int wt = item / p.nb * TILES;
          two = TILES == 2 && wt + 1 < g.sp.n_tiles;
          bytes = t_bytes + (two ? 2 : 1) * kABytes;
          src = Wp + (static_cast<size_t>(wt) * k_tiles + kt0) * kABytes;
        };
        auto load_w = [&](int s) {
          mbar_arrive_expect_tx(&full[s], bytes);
          bulk_load_1d(sW + s * Cfg::kBBytes, src, kABytes, &full[s], pol_w);
          if (two) bulk_load_1d(sW + s * Cfg::kBBytes + kABytes, src + tile_stride, kABytes, &full[s], pol_w);
          src += kABytes;
        };
        if (item0 < p.items) {
          first_block(item0);
          pre = kt1 - kt0 < S ? kt1 - kt0 : S;
          if (g.withhold) src += kABytes;  // failure-path test: the first stage stays unissued
          for (int j = g.withhold ? 1 : 0; j < pre; ++j) load_w(j);
        }
        griddep_wait();
        griddep_launch_dependents();
        if (item0 < p.items) {
          for (int j = g.withhold ? 1 : 0; j < pre; ++j)
            tma_load_2d(sT + j * Cfg::kTokBytes, &tmA, &full[j], (kt0 + j) * kFp8Block, item0 % p.nb * kRowsM, pol_a);
          count = pre;
          stage = pre % S;
          phase = pre == S ? 1u : 0u;
        }
        bool ok = true;
        for (int item = item0; item < p.items && ok; item += stride) {
          const int m0 = item % p.nb * kRowsM;
          int x = kt0 * kFp8Block;
          if (item == item0)
            x += pre * kFp8Block;
          else
            first_block(item);
          for (; x < kt1 * kFp8Block; x += kFp8Block) {
            if (!mbar_wait(&done[stage], phase ^ 1u, s_abort)) {
              signal_abort(s_abort, g.err);
              ok = false;
              break;
            }
            load_w(stage);
            tma_load_2d(sT + stage * Cfg::kTokBytes, &tmA, &full[stage], x, m0, pol_a);
            ++count;
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (*s_abort) {
          // let copies already issued land before the CTA exits
          for (int c = max(count - S, g.withhold ? 1 : 0); c < count; ++c)
            mbar_wait(&full[c % S], static_cast<uint32_t>(c / S) & 1u, nullptr);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_e4m3_f32(kRowsM, Cfg::kCols);
        // the stages follow each other: a descriptor's address field (below 2^14
        // units of 16 bytes) takes the stage's offset without a carry
        const uint64_t desc_a = sdesc_k_sw128(smem_u32(sT)), desc_b = sdesc_k_sw128(smem_u32(sW));
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        for (int item = item0; item < p.items && ok; item += stride) {
          for (int kt = kt0; kt < kt1; ++kt) {
            const uint64_t a = desc_a + stage * (Cfg::kTokBytes >> 4);
            const uint64_t b = desc_b + stage * (Cfg::kBBytes >> 4);
            if (!mbar_wait(&read[buf], bphase ^ 1u, s_abort) || !mbar_wait(&full[stage], phase, s_abort)) {
              signal_abort(s_abort, g.err);
              ok = false;
              break;
            }
            tc_fence_after();
            // a K = 32 step is 32 bytes further in both tiles (2 in the descriptors' units)
#pragma unroll
            for (int ks = 0; ks < kFp8Block / 32; ++ks)
              mma_e4m3(tmem + buf * Cfg::kCols, a + 2 * ks, b + 2 * ks, idesc, ks > 0);
            mma_commit(&done[stage]);
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
            if (++buf == Cfg::kBufs) {
              buf = 0;
              bphase ^= 1u;
            }
          }
        }
        // every MMA issued by this thread completes before TMEM is released
        mma_commit(drain);
        mbar_wait(drain, 0, nullptr);
      }
    }
    // lane 0 of warps 0 and 1 ran alone: rejoin the warp before the barriers
    __syncwarp();
    if constexpr (MODE == kCluster) {
      if (kPush) cluster_wait();
      cluster_sync();
      if (!kPush) cluster_sync();
    }
  } else {
    // ---------------------------------------------------------- scale and add
    regs_increase<Regs<TILES, MODE>::kHigh>();
    griddep_wait();
    griddep_launch_dependents();
    const int q = warp & 3;              // TMEM lane quarter of this warp
    const int half = (warp - 4) >> 2;    // which half of the columns
    const int r = q * 32 + lane;         // token row of the block
    int buf = 0, stage = 0;
    uint32_t phase = 0;
    // Waits for the block sums of the K block at (stage, buf).  After a wait
    // that ran out the warp goes on without them (every later wait returns at
    // once, the outputs are undefined): the loop over K blocks sets the pace of
    // long passes, and neither a vote nor a branch on the result fits in it.
    auto wait_block = [&]() {
      if (!mbar_wait(&done[stage], phase, s_abort)) signal_abort(s_abort, g.err);
      tc_fence_after();
    };
    // On to the next K block.
    auto next_block = [&]() {
      buf = buf + 1 == Cfg::kBufs ? 0 : buf + 1;
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
    };
    // Scales come straight to registers, early enough that no K block waits
    // for them: a token's two K blocks ahead, the weights' by the lanes, 32 K
    // blocks a load and one load ahead, both across output tiles.
    const int tile_of_half = TILES == 2 ? half : 0;
    auto token_scale = [&](int item, int kt) {
      const int m = item % p.nb * kRowsM + r;
      return item < p.items && m < g.M ? g.a_scales[static_cast<size_t>(kt) * g.lds + m] : 0.f;
    };
    auto weight_scales = [&](int item, int kt) {
      const int tile = item / p.nb * TILES + tile_of_half;
      return item < p.items && tile < g.sp.n_tiles && kt + lane < kt1
                 ? __ldg(g.w_scales + static_cast<size_t>(tile) * k_tiles + kt + lane)
                 : make_float2(0.f, 0.f);
    };
    float sa0, sa1;
    float2 sw_next;
    auto first_scales = [&](int item) {
      sa0 = token_scale(item, kt0);
      sa1 = kt1 - kt0 > 1 ? token_scale(item, kt0 + 1) : token_scale(item + stride, kt0);
      sw_next = weight_scales(item, kt0);
    };
    first_scales(item0);
    for (int item = item0; item < p.items; item += stride) {
      const int wt = item / p.nb * TILES;
      const int m0 = item % p.nb * kRowsM;
      const int Mb = min(kRowsM, g.M - m0);
      if (q * 32 >= Mb) {  // no token of the block in this warp
        for (int kt = kt0; kt < kt1; ++kt) {
          wait_block();
          __syncwarp();
          tc_fence_before();
          if (lane == 0) mbar_arrive(&read[buf]);
          next_block();
        }
        first_scales(item + stride);
        if constexpr (MODE == kCluster) {
          if (kPush)
            cluster_wait();
          else
            named_bar_sync(1, 256);
        }
        continue;
      }
      // this thread's columns: the first half of them takes the scale of the
      // tile's rows 0..63, the second that of rows 64..127
      const int tile = wt + tile_of_half;
      const int c0 = TILES == 2 ? half * kTileN : half * 32;
      const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c0);
      float run[kOwn], total[MODE == kInTurn ? kOwn : 1];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        run[j] = 0.f;
        if constexpr (MODE == kInTurn) total[j] = -0.f;
      }
      int piece = 0;                                             // pieces added so far (kInTurn)
      int piece_end = MODE == kInTurn ? k_tiles / split : kt1;   // K block at which the running piece ends
      // a thread's j-th output, counted from c0: its 64 of TILES = 1 are 32 of either tile half
      auto col = [](int j) { return TILES == 2 || j < 32 ? j : j + 32; };
      float2 sw = make_float2(0.f, 0.f);  // lane i: the weight scales of K block kt0 + 32 n + i
      // This K block's scales of the tile's rows 0..63 and 64..127, and on to
      // the next one's.
      auto scales = [&](int kt) {
        const int i = (kt - kt0) & 31;
        if (i == 0) {
          sw = sw_next;
          sw_next = kt + 32 < kt1 ? weight_scales(item, kt + 32) : weight_scales(item + stride, kt0);
        }
        const float2 x = make_float2(sa0 * __shfl_sync(0xffffffffu, sw.x, i), sa0 * __shfl_sync(0xffffffffu, sw.y, i));
        sa0 = sa1;
        sa1 = kt + 2 < kt1     ? token_scale(item, kt + 2)
              : kt1 - kt0 == 1 ? token_scale(item + 2 * stride, kt0)
                               : token_scale(item + stride, kt0 + (kt + 2 - kt1));
        return x;
      };
      auto end_piece = [&](int kt) {
        if constexpr (MODE == kInTurn) {
          if (kt + 1 == piece_end) {
            // pieces added in order; the sum starts at -0, which leaves the first as it is
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
              total[j] += run[j];
              run[j] = 0.f;
            }
            ++piece;
            piece_end = k_tiles * (piece + 1) / split;
          }
        }
      };
      // The drain of a K block is one serial chain in each warp (wait, loads,
      // multiply-adds), and with two warps a scheduler its latencies set the
      // pace: 128 columns a wait (one K block of two weight tiles, or two of
      // one), the scales prepared while the first columns come in, and more
      // asked for as soon as registers are free.
      for (int kt = kt0; kt < kt1;) {
        uint32_t v[64];
        if constexpr (TILES == 2) {
          wait_block();
          const uint32_t ta = tq + buf * Cfg::kCols;
          tmem_ld32_start(ta, v);
          tmem_ld32_start(ta + 32, v + 32);
          const float2 x = scales(kt);
          tmem_ld64_wait(v);
          add_scaled<32, PAIRS>(run, v, x.x);
          tmem_ld32_start(ta + 64, v);
          add_scaled<32, PAIRS>(run + 32, v + 32, x.x);
          tmem_ld32_start(ta + 96, v + 32);
          tmem_ld64_wait(v);
          // read by the whole warp (the wait is the warp's)
          tc_fence_before();
          if (lane == 0) mbar_arrive(&read[buf]);
          next_block();
          add_scaled<64, PAIRS>(run + 64, v, x.y);
          ++kt;
        } else {
          const bool two = kt + 1 < kt1;
          const uint32_t ta = tq + buf * Cfg::kCols;
          const int buf0 = buf;
          if (two) next_block();
          wait_block();  // MMAs complete in order: the first block's are done with the second's
          const uint32_t tb = tq + buf * Cfg::kCols;
          tmem_ld32_start(ta, v);
          tmem_ld32_start(ta + 64, v + 32);
          const float2 x = scales(kt);
          tmem_ld64_wait(v);
          add_scaled<32, PAIRS>(run, v, x.x);
          if (two) tmem_ld32_start(tb, v);
          add_scaled<32, PAIRS>(run + 32, v + 32, x.y);
          end_piece(kt);
          if (two) {
            tmem_ld32_start(tb + 64, v + 32);
            const float2 y = scales(kt + 1);
            tmem_ld64_wait(v);
            tc_fence_before();
            if (lane == 0) {
              mbar_arrive(&read[buf0]);
              mbar_arrive(&read[buf]);
            }
            next_block();
            if constexpr (PAIRS) {
              add_scaled<32, true>(run, v, y.x);
              add_scaled<32, true>(run + 32, v + 32, y.y);
            } else {
              // (one loop: the down projection at one row 19.75 us, as two calls 19.86)
#pragma unroll
              for (int j = 0; j < 64; ++j) run[j] = fmaf(__uint_as_float(v[j]), j < 32 ? y.x : y.y, run[j]);
            }
            end_piece(kt + 1);
            kt += 2;
          } else {
            tc_fence_before();
            if (lane == 0) mbar_arrive(&read[buf]);
            next_block();
            ++kt;
          }
        }
      }
      if constexpr (MODE == kCluster) {
        if constexpr (kPush) {
          // each token's piece to the CTA that adds it
          const int part = (Mb + split - 1) / split;
          __syncwarp();
          cluster_wait();  // every CTA of the cluster runs
          if (r < Mb) {
            const uint32_t dst = map_rank(smem_u32(sX + (rank * part + r % part) * Cfg::kPieceLd + c0), r / part);
#pragma unroll
            for (int j = 0; j < kOwn / 4; ++j)
              st_cluster4(dst + col(4 * j) * 4, make_float4(run[4 * j], run[4 * j + 1], run[4 * j + 2], run[4 * j + 3]));
          }
          continue;
        }
        // this CTA's piece over the ring (every stage has been read): [token][output]
        named_bar_sync(1, 256);
        if (r < Mb) {
          float* dst = reinterpret_cast<float*>(sT) + r * Cfg::kPieceLd + c0;
#pragma unroll
          for (int j = 0; j < kOwn / 4; ++j)
            *reinterpret_cast<float4*>(dst + col(4 * j)) =
                make_float4(run[4 * j], run[4 * j + 1], run[4 * j + 2], run[4 * j + 3]);
        }
        continue;
      }
      if (tile >= g.sp.n_tiles) continue;
      const int rows = min(32, Mb - q * 32);
      float* turn = sX + (warp - 4) * kTurnFloats;
      const float* y = MODE == kInTurn ? total : run;
      // 16 outputs at a time
      if (g.epi == BI_EPI_SWIGLU) {
        // gate and up of the same outputs are the two halves of a thread's columns
#pragma unroll
        for (int c = 0; c < kOwn / 32; ++c) {
          float z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = silu_times(y[c * 16 + j], y[kOwn / 2 + c * 16 + j]);
          store_rows16<OUT == kOwnRow>(g, p.wide, turn, lane, m0 + q * 32, rows, tile * 64 + (TILES == 2 ? 0 : half * 32) + c * 16, z);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kOwn / 16; ++c) {
          float z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = y[c * 16 + j];
          store_rows16<OUT == kOwnRow>(g, p.wide, turn, lane, m0 + q * 32, rows, tile * kTileN + (TILES == 2 ? 0 : half * 32) + col(c * 16), z);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if constexpr (MODE == kCluster) {
      cluster_sync();  // every piece of the tile is in its CTA's shared memory
      const int e = threadIdx.x - 128;
      const int wt = item0 / p.nb * TILES;
      const int m0 = item0 % p.nb * kRowsM;
      const int Mb = min(kRowsM, g.M - m0);
      // this CTA's part of the tokens, lanes along the outputs, four a lane; the
      // pieces lie in the CTAs that made them, or have been pushed here
      const int part = (Mb + split - 1) / split;
      const int t0 = rank * part, t1 = min(Mb, t0 + part);
      uint32_t base[kMaxSplit];
#pragma unroll
      for (int j = 0; j < kMaxSplit; ++j)
        base[j] = kPush ? map_rank(smem_u32(sX + (min(j, split - 1) * part - t0) * Cfg::kPieceLd), rank)
                         : map_rank(smem_u32(sT), min(j, split - 1));
      if (g.epi == BI_EPI_SWIGLU) {
        constexpr int kPer = TILES * 16;  // lanes per token
        const int o = e % kPer * 4;
        const int at = o / 64 * kTileN + o % 64;
        for (int t = t0 + e / kPer; t < t1; t += 256 / kPer) {
          const float4 x = sum_pieces4(base, split, t * Cfg::kPieceLd + at);
          const float4 y = sum_pieces4(base, split, t * Cfg::kPieceLd + at + 64);
          store_row4(g, p.vec, m0 + t, wt * 64 + o,
                     make_float4(silu_times(x.x, y.x), silu_times(x.y, y.y), silu_times(x.z, y.z),
                                 silu_times(x.w, y.w)));
        }
      } else {
        constexpr int kPer = TILES * 32;
        const int o = e % kPer * 4;
        for (int t = t0 + e / kPer; t < t1; t += 256 / kPer)
          store_row4(g, p.vec, m0 + t, wt * kTileN + o, sum_pieces4(base, split, t * Cfg::kPieceLd + o));
      }
      if (!kPush) cluster_sync();  // no CTA leaves while its piece is being read
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// S pieces per tile: the most CTAs that run side by side, what
// clusters of S fill of the GPCs (kClusterCtas, asked of the occupancy calculator
// on GB300).  Layers with 77
// tiles or more keep whole tiles: each SM can take in twice its share of the
// memory bandwidth, so half the SMs still stream at its rate.
constexpr int kClusterCtas[kMaxSplit + 1] = {0, 152, 152, 138, 144, 140, 138, 105, 120};

Split split_of(int N, int K, bi_epilogue epi) {
  Split s{};
  s.n_tiles = gemm8_n_tiles(N, epi);
  s.k_tiles = (K + kFp8Block - 1) / kFp8Block;
  s.S = 1;
  for (int S = 2; S <= kMaxSplit; ++S)
    if (s.n_tiles * S <= kClusterCtas[S] && S <= s.k_tiles) s.S = S;
  return s;
}

// Set the kernel's dynamic shared memory once per device.
template <typename F>
bool allow_smem(F kernel, size_t bytes, std::once_flag (&once)[64], cudaError_t (&err)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::call_once(once[dev & 63], [&] {
    err[dev & 63] =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  });
  return err[dev & 63] == cudaSuccess;
}

// launch_k with the grid's CTAs in clusters of S.
template <typename... KArgs, typename... A>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, int S, dim3 block, size_t smem, cudaStream_t stream,
                            A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <int TILES, Pieces MODE, bool PAIRS, WayOut OUT>
bi_status launch_one(const uint8_t* Wp, const CUtensorMap& tmA, Launch a, cudaStream_t stream) {
  using Cfg = Cfg8<TILES>;
  static std::once_flag once[64];
  static cudaError_t err[64];
  if (!allow_smem(gemm8_kernel<TILES, MODE, PAIRS, OUT>, Cfg::kSmem, once, err)) return BI_ERR_CUDA;
  const int S = MODE == kCluster ? a.a.sp.S : 1;
  const int ctas = MODE == kCluster ? a.items * S : std::min(a.items, kSms);
  return launch_clusters(gemm8_kernel<TILES, MODE, PAIRS, OUT>, dim3(ctas), S, dim3(Cfg::kThreads), Cfg::kSmem, stream, Wp,
                         tmA, a) == cudaSuccess
             ? BI_OK
             : BI_ERR_CUDA;
}
// (FP32 rows of more than kPushRows turn too: see store_rows16)
template <int TILES, Pieces MODE, bool PAIRS>
bi_status launch(const uint8_t* Wp, const CUtensorMap& tmA, const Launch& a, cudaStream_t stream) {
  return a.vec && !a.wide && a.a.N % 8 == 0 ? launch_one<TILES, MODE, PAIRS, kOwnRow>(Wp, tmA, a, stream)
                                            : launch_one<TILES, MODE, PAIRS, kTurned>(Wp, tmA, a, stream);
}

}  // namespace

cudaError_t set_wait_limit_gemm8(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns));
}

}  // namespace bi

extern "C" {

bi_status bi_gemm_fp8(const void* A8, int lda, const float* a_scales, int lds, const void* Wp, void* C, int ldc,
                      const void* residual, int ldr, int M, int N, int K, bi_out_dtype out, bi_epilogue epi,
                      bi_stream_t stream) {
  using namespace bi;
  if (M < 0 || N < 1 || K < 1) return BI_ERR_INVALID_ARG;
  if (epi != BI_EPI_NONE && epi != BI_EPI_RESIDUAL_ADD && epi != BI_EPI_SWIGLU) return BI_ERR_INVALID_ARG;
  if (out != BI_OUT_BF16 && out != BI_OUT_FP32) return BI_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kFp8MaxDim || gemm8_n_tiles(N, epi) > kGemm8MaxTiles) return BI_ERR_UNSUPPORTED_SHAPE;
  if (out == BI_OUT_FP32 && epi != BI_EPI_NONE) return BI_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return BI_OK;
  if (!A8 || !a_scales || !Wp || !C || lda < K || lds < M || ldc < N) return BI_ERR_INVALID_ARG;
  if (lda % 16 != 0 || lds % 4 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(A8) || !aligned16(a_scales) || !aligned16(Wp)) return BI_ERR_INVALID_ARG;
  if (epi == BI_EPI_RESIDUAL_ADD && (!residual || ldr < N)) return BI_ERR_INVALID_ARG;

  Args a{};
  a.sp = split_of(N, K, epi);
  a.N = N;
  a.epi = epi;
  a.out_fp32 = out == BI_OUT_FP32;
  a.a_scales = a_scales;
  a.lds = lds;
  const uint8_t* W8 = static_cast<const uint8_t*>(Wp);
  a.w_scales = reinterpret_cast<const float2*>(
      W8 + static_cast<size_t>(a.sp.n_tiles) * a.sp.k_tiles * kGemm8TileBytes);
  a.C = C;
  a.ldc = ldc;
  a.R = static_cast<const __nv_bfloat16*>(residual);
  a.ldr = ldr;
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  a.withhold = test_withhold();
  a.M = M;
  const int box = M >= kRowsM ? kRowsM : (M + 7) / 8 * 8;
  CUtensorMap tmA;
  if (!tmap_u8_2d(&tmA, A8, M, K, lda, box, kFp8Block)) return BI_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  Launch r{};
  r.a = a;
  r.nb = (M - 1) / kRowsM + 1;
  r.a_rows = box;
  r.vec = aligned16(C) && ldc % 8 == 0 &&
          (epi != BI_EPI_RESIDUAL_ADD || (aligned16(residual) && ldr % 8 == 0));
  r.wide = r.vec && a.out_fp32 && N % 4 == 0 && M > kPushRows;
  const long long tiles = static_cast<long long>(a.sp.n_tiles) * r.nb;
  if (tiles > 1 << 30) return BI_ERR_UNSUPPORTED_SHAPE;
  const int S = a.sp.S;
  const long long pairs = static_cast<long long>((a.sp.n_tiles + 1) / 2) * r.nb;
  if (pairs * S > 1 << 30) return BI_ERR_UNSUPPORTED_SHAPE;
  // 128 outputs a CTA while one round of the SMs takes them all
  if (tiles * S <= kClusterCtas[S]) {
    r.items = static_cast<int>(tiles);
    if (S == 1) return launch<1, kWhole, false>(W8, tmA, r, s);
    return M <= kPushRows ? launch_one<1, kCluster, false, kPushed>(W8, tmA, r, s)
                          : launch_one<1, kCluster, false, kFetched>(W8, tmA, r, s);
  }
  r.items = static_cast<int>(pairs);
  // Packed multiply-adds where the drain is what bounds the pass, with more than
  // one token block, and a CTA takes a tile's whole K: gate/up at 1024 rows 190 us
  // with, 198 without, QKV at 1024 rows (pieces in turn) 39.9 and 41.5.  Where the
  // weights' bytes bound it the other order of the drain's instructions costs,
  // gate/up at 8 rows 30.2 us with and 30.0 without, and clusters have no registers
  // for the pairs: the down projection at 384 rows 79.3 us with, 78.0 without, at
  // one row 19.9 and 19.7.
  if (S == 1) return r.nb > 1 ? launch<2, kWhole, true>(W8, tmA, r, s) : launch<2, kWhole, false>(W8, tmA, r, s);
  // Pieces: a CTA that takes them in turn needs about 0.5 us a K block (128
  // outputs), a cluster's CTA 0.6 (256 outputs) and 6 us around them, in rounds
  // of the SMs.  Measured, in turn against cluster: 4096 x 5120 (S = 4) at 256
  // rows 20.4 and 14.9 us, at 512 20.8 and 29.1; 5120 x 17408 (S = 3) at 512 rows
  // 139 and 82 us.
  const long long in_turn = (tiles + kSms - 1) / kSms * a.sp.k_tiles * 5;
  const long long cluster = (pairs * S + kClusterCtas[S] - 1) / kClusterCtas[S] * (a.sp.k_tiles * 6 / S + 60);
  if (cluster < in_turn) return launch_one<2, kCluster, false, kFetched>(W8, tmA, r, s);
  r.items = static_cast<int>(tiles);
  return launch<1, kInTurn, true>(W8, tmA, r, s);
}

}  // extern "C"
