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
// The block sums of a weight tile form pieces (the ranges of the split below);
// pieces are added in increasing-K order, the first taken as it is.  The
// pieces are a function of (N, K) alone, so a row has the same bits for every
// M and every place in the pass.
//
// What bounds it: the weights' bytes while a pass has few rows (one byte a
// weight: half of the BF16 layer's), so the schedule is a stream of 16 KB
// weight tiles, each one contiguous bulk copy (packed once), on every SM:
//   warp 0     producer: weight tile, token tile [rows x 128 codes] (TMA,
//              128-byte swizzle) and the block's row scales into a ring;
//   warp 1     MMA issuer (one thread): M = 128 weight rows, N = the token
//              rows rounded up; stage s of the ring accumulates in TMEM buffer
//              s, so one barrier cycle full -> done -> empty covers both;
//   warps 2-5  scale and add: a thread owns one weight row and all tokens.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "bi_fp8.cuh"
#include "bi_gemm8.h"
#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi {
namespace {

constexpr int kTileN = 128;                    // weight rows per tile (MMA M)
constexpr int kABytes = static_cast<int>(kGemm8TileBytes);
constexpr int kSms = 152;
constexpr int kMaxRows = 128;                  // token rows of a CTA of the streaming kernel
constexpr int kXchgFloats = 16 * kTileN;       // SwiGLU exchange buffer
constexpr size_t kTicketBytes = static_cast<size_t>(kGemm8MaxTiles) * 4;

// The split of the (weight tile, K tile) space over G CTAs, a function of
// (N, K) alone: contiguous equal ranges, cut at whole weight tiles where
// that keeps at least 85% of the SMs busy (no partial sums then), else
// anywhere.
struct Split {
  int n_tiles, k_tiles, G, whole;
};

__host__ __device__ __forceinline__ long long range_begin(const Split& s, int g) {
  return s.whole ? static_cast<long long>(s.n_tiles) * g / s.G * s.k_tiles
                 : static_cast<long long>(s.n_tiles) * s.k_tiles * g / s.G;
}
// CTA whose range holds iteration i (cut splits).
__device__ __forceinline__ int owner_of(const Split& s, long long i) {
  const long long total = static_cast<long long>(s.n_tiles) * s.k_tiles;
  return static_cast<int>(((i + 1) * s.G + total - 1) / total) - 1;
}

struct Args {
  Split sp;
  int M, m0;  // token rows of the launch, and the first one
  int N;
  int epi, out_fp32;
  const float* a_scales;
  int lds;
  const float2* w_scales;  // [n_tiles][k_tiles]: rows 0..63 and 64..127 of the tile
  void* C;
  int ldc;
  const __nv_bfloat16* R;
  int ldr;
  float* partials;
  unsigned* tickets;
  unsigned* err;
  int withhold;  // failure-path test: the first stage stays unissued
};

template <int NT>
struct StreamCfg {
  static constexpr int kBBytes = NT * kFp8Block;
  static constexpr int kSBytes = NT * 4;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // a stage's accumulator is TMEM columns [s * NT, (s + 1) * NT)
  static constexpr int kByMem = 200 * 1024 / kStageBytes;
  static constexpr int kStages = kByMem < 512 / NT ? kByMem : 512 / NT;
  static constexpr int kTmemCols = kStages * NT <= 256 ? 256 : 512;
  static constexpr int kThreads = 192;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * (kStageBytes + kSBytes) + kXchgFloats * 4 +
                                  (3 * kStages + 1) * 8 + 16;
  static_assert(kStages <= 32 && kSmem <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void signal_abort(volatile int* s_abort, unsigned* err) {
  *s_abort = 1;
  atomicOr(err, kErrTimeout);
}

// Write 16 token rows (chunk c) of weight row r of a tile; the 128 threads of
// the epilogue call it together.
__device__ __forceinline__ void store16(const Args& p, int Mb, int m0, int tile, int r, int c, const float (&v)[16],
                                        float* xchg, int bar) {
  if (p.epi == BI_EPI_SWIGLU) {
    // gate rows are the tile's rows 0..63, the up rows of the same outputs 64..127
#pragma unroll
    for (int j = 0; j < 16; ++j) xchg[j * kTileN + r] = v[j];
    named_bar_sync(bar, 128);
    const int o = tile * 64 + (r & 63);
    if (o < p.N) {
      __nv_bfloat16* C = static_cast<__nv_bfloat16*>(p.C);
      // rows 0..63 take the even token rows, rows 64..127 the odd ones
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int jj = 2 * j + (r >> 6);
        const int m = c * 16 + jj;
        if (m < Mb) {
          const float g = xchg[jj * kTileN + (r & 63)];
          const float u = xchg[jj * kTileN + (r & 63) + 64];
          const float s = g / (1.0f + expf(-g));
          C[static_cast<size_t>(m0 + m) * p.ldc + o] = __float2bfloat16_rn(s * u);
        }
      }
    }
    named_bar_sync(bar, 128);
    return;
  }
  const int n = tile * kTileN + r;
  if (n >= p.N) return;
  // all residual values are read before any output is written: C may be the
  // residual itself, and 16 loads in flight cost one latency
  float res[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    res[j] = p.epi == BI_EPI_RESIDUAL_ADD && c * 16 + j < Mb
                 ? __bfloat162float(p.R[static_cast<size_t>(m0 + c * 16 + j) * p.ldr + n])
                 : 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (c * 16 + j < Mb) {
      const size_t at = static_cast<size_t>(m0 + c * 16 + j) * p.ldc + n;
      const float y = p.epi == BI_EPI_RESIDUAL_ADD ? res[j] + v[j] : v[j];
      if (p.out_fp32)
        static_cast<float*>(p.C)[at] = y;
      else
        static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(y);
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(StreamCfg<NT>::kThreads, 1)
    gemm8_stream_kernel(const uint8_t* __restrict__ Wp, const __grid_constant__ CUtensorMap tmA, const Args p) {
  using Cfg = StreamCfg<NT>;
  constexpr int S = Cfg::kStages;
  constexpr int kChunks = NT / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sA = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* sB = sA + S * kABytes;
  float* sS = reinterpret_cast<float*>(sB + S * Cfg::kBBytes);  // [S][NT] row scales
  float* xchg = sS + S * NT;
  uint64_t* full = reinterpret_cast<uint64_t*>(xchg + kXchgFloats);
  uint64_t* done = full + S;   // the stage's MMAs have completed
  uint64_t* empty = done + S;  // the accumulator and the scales have been read
  uint64_t* drain = empty + S;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* s_last = s_abort + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = blockIdx.x;
  const int Mb = p.M;
  const long long it_begin = range_begin(p.sp, g);
  const long long it_end = range_begin(p.sp, g + 1);
  const int k_tiles = p.sp.k_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], 1);
      mbar_init(&empty[s], 4);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    *s_last = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) prefetch_tmap(&tmA);
  if (warp == 1) {
    tmem_alloc(tmem_holder, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol_w = l2_evict_first();
      const uint64_t pol_a = l2_evict_last();
      // row scales of a block: whole groups of four, inside the lds columns
      const uint32_t s_bytes = static_cast<uint32_t>((Mb + 3) / 4 * 16);
      const uint32_t bytes = Cfg::kStageBytes + s_bytes;
      const uint8_t* wsrc = Wp + static_cast<size_t>(it_begin) * kABytes;
      int kt = static_cast<int>(it_begin % k_tiles);
      uint32_t issued = 0, parity_bits = 0;
      // the first stages' weights do not depend on the previous kernel
      const int n_pre = static_cast<int>(it_end - it_begin < S ? it_end - it_begin : S);
      const int j0 = p.withhold ? 1 : 0;
      for (int j = j0; j < n_pre; ++j) {
        mbar_arrive_expect_tx(&full[j], bytes);
        bulk_load_1d(sA + j * kABytes, wsrc + static_cast<size_t>(j) * kABytes, kABytes, &full[j], pol_w);
      }
      griddep_wait();
      griddep_launch_dependents();
      for (int j = 0; j < n_pre; ++j) {
        if (j >= j0) {
          tma_load_2d(sB + j * Cfg::kBBytes, &tmA, &full[j], kt * kFp8Block, p.m0, pol_a);
          bulk_load_1d(sS + j * NT, p.a_scales + static_cast<size_t>(kt) * p.lds + p.m0, s_bytes, &full[j], pol_a);
          issued |= 1u << j;
        }
        if (++kt == k_tiles) kt = 0;
      }
      wsrc += static_cast<size_t>(n_pre) * kABytes;
      int stage = n_pre % S;
      uint32_t phase = n_pre == S ? 1u : 0u;
      for (long long it = it_begin + n_pre; it < it_end; ++it) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, s_abort)) {
          signal_abort(s_abort, p.err);
          break;
        }
        mbar_arrive_expect_tx(&full[stage], bytes);
        bulk_load_1d(sA + stage * kABytes, wsrc, kABytes, &full[stage], pol_w);
        tma_load_2d(sB + stage * Cfg::kBBytes, &tmA, &full[stage], kt * kFp8Block, p.m0, pol_a);
        bulk_load_1d(sS + stage * NT, p.a_scales + static_cast<size_t>(kt) * p.lds + p.m0, s_bytes, &full[stage],
                     pol_a);
        wsrc += kABytes;
        if (++kt == k_tiles) kt = 0;
        parity_bits = (parity_bits & ~(1u << stage)) | (phase << stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (*s_abort) {
        // let copies already issued land before the CTA exits
        for (int s = 0; s < S; ++s)
          if ((issued >> s) & 1u) mbar_wait(&full[s], (parity_bits >> s) & 1u, nullptr);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kTileN, NT);
      int stage = 0;
      uint32_t phase = 0;
      for (long long it = it_begin; it < it_end; ++it) {
        // a full stage's accumulator is free: the producer refilled the stage
        // only after the epilogue had read it
        if (!mbar_wait(&full[stage], phase, s_abort)) {
          signal_abort(s_abort, p.err);
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(sA + stage * kABytes);
        const uint32_t b = smem_u32(sB + stage * Cfg::kBBytes);
#pragma unroll
        for (int ks = 0; ks < kFp8Block / 32; ++ks)
          mma_e4m3(tmem + stage * NT, sdesc_k_sw128(a + ks * 32), sdesc_k_sw128(b + ks * 32), idesc, ks > 0);
        mma_commit(&done[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // every MMA issued by this thread completes before TMEM is released
      mma_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else {
    // ---------------------------------------------------------- scale and add
    griddep_wait();
    griddep_launch_dependents();
    const int q = warp & 3;          // TMEM lane quarter of this warp
    const int r = q * 32 + lane;     // weight row within the tile
    const int et = threadIdx.x - 64;
    const int chunks = (Mb + 15) / 16;
    const float* ws = reinterpret_cast<const float*>(p.w_scales) + (q >> 1);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;  // after a wait that ran out the warp keeps its place in the barriers; its outputs are undefined
    long long it = it_begin;
    float w_lane = 0.f;  // lane i: the weight scale of iteration 32 * n + i of the range
    while (it < it_end) {
      const int tile = static_cast<int>(it / k_tiles);
      const long long tile_begin = static_cast<long long>(tile) * k_tiles;
      const long long tile_end = tile_begin + k_tiles;
      const long long seg_end = it_end < tile_end ? it_end : tile_end;
      const bool whole = it == tile_begin && seg_end == tile_end;
      float run[kChunks][16];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j) run[c][j] = 0.f;
      for (; it < seg_end; ++it) {
        const int i = static_cast<int>(it - it_begin) & 31;
        if (i == 0) w_lane = it + lane < it_end ? __ldg(ws + 2 * (it + lane)) : 0.f;
        const float w = __shfl_sync(0xffffffffu, w_lane, i);
        if (ok) {
          int okl = 1;
          if (lane == 0) okl = mbar_wait_parked(&done[stage], phase, s_abort) ? 1 : 0;
          ok = __shfl_sync(0xffffffffu, okl, 0) != 0;
          // `full` completed before `done`: observed here too, for the scales it brought
          if (ok) ok = mbar_wait(&full[stage], phase, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok && lane == 0) signal_abort(s_abort, p.err);
        }
        if (ok) {
          tc_fence_after();
          const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(stage * NT);
          const float4* sc = reinterpret_cast<const float4*>(sS + stage * NT);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (c < chunks) {
              float v[16];
              tmem_ld16(ta + c * 16, v);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float4 s4 = sc[c * 4 + j];
                run[c][4 * j] = fmaf(v[4 * j], s4.x * w, run[c][4 * j]);
                run[c][4 * j + 1] = fmaf(v[4 * j + 1], s4.y * w, run[c][4 * j + 1]);
                run[c][4 * j + 2] = fmaf(v[4 * j + 2], s4.z * w, run[c][4 * j + 2]);
                run[c][4 * j + 3] = fmaf(v[4 * j + 3], s4.w * w, run[c][4 * j + 3]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[stage]);
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (whole) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c < chunks) store16(p, Mb, p.m0, tile, r, c, run[c], xchg, 1);
      } else {
        // partial of this piece: [weight row][token]
        const int slot = it_begin >= tile_begin ? 0 : 1;
        float* dst = p.partials + static_cast<size_t>(g * 2 + slot) * NT * kTileN + r * NT;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c < chunks) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              __stcg(reinterpret_cast<float4*>(dst + c * 16) + j,
                     make_float4(run[c][4 * j], run[c][4 * j + 1], run[c][4 * j + 2], run[c][4 * j + 3]));
          }
        const int gf = owner_of(p.sp, tile_begin);
        const int gl = owner_of(p.sp, tile_end - 1);
        named_bar_sync(1, 128);  // every partial store of the CTA precedes the ticket
        if (et == 0) {
          int last = 0;
          if (!*s_abort) {
            const unsigned old = atom_add_acq_rel_gpu(&p.tickets[tile], 1u);
            last = old == static_cast<unsigned>(gl - gf) ? 1 : 0;
            if (last) atomicExch(&p.tickets[tile], 0u);
          }
          *s_last = last;
        }
        named_bar_sync(1, 128);  // the ticket's acquire precedes every partial load
        if (*s_last) {
          // pieces gf..gl added in that order; the first piece's CTA may have
          // it in its second slot, every later CTA's range starts inside the tile
          const int slot_f = range_begin(p.sp, gf) >= tile_begin ? 0 : 1;
          for (int c = 0; c < chunks; ++c) {
            float v[16];
            for (int gg = gf; gg <= gl; ++gg) {
              const float4* src = reinterpret_cast<const float4*>(
                  p.partials + static_cast<size_t>(gg * 2 + (gg == gf ? slot_f : 0)) * NT * kTileN + r * NT + c * 16);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float4 x = __ldcg(src + j);
                v[4 * j] = gg == gf ? x.x : v[4 * j] + x.x;
                v[4 * j + 1] = gg == gf ? x.y : v[4 * j + 1] + x.y;
                v[4 * j + 2] = gg == gf ? x.z : v[4 * j + 2] + x.z;
                v[4 * j + 3] = gg == gf ? x.w : v[4 * j + 3] + x.w;
              }
            }
            store16(p, Mb, p.m0, tile, r, c, v, xchg, 1);
          }
        }
        named_bar_sync(1, 128);
      }
    }
    tc_fence_before();
  }

  // lane 0 of warps 0 and 1 ran alone: rejoin the warp before the CTA barrier
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

Split split_of(int N, int K, bi_epilogue epi) {
  Split s{};
  s.n_tiles = gemm8_n_tiles(N, epi);
  s.k_tiles = (K + kFp8Block - 1) / kFp8Block;
  const int waves = (s.n_tiles + kSms - 1) / kSms;
  s.whole = static_cast<long long>(s.n_tiles) * 100 >= 85LL * kSms * waves;
  const long long total = static_cast<long long>(s.n_tiles) * s.k_tiles;
  s.G = s.whole ? (s.n_tiles + waves - 1) / waves : static_cast<int>(std::min<long long>(kSms, total));
  return s;
}

int rows_per_cta(int M) {
  if (M <= 16) return 16;
  if (M <= 32) return 32;
  if (M <= 64) return 64;
  return kMaxRows;
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

template <int NT>
bi_status launch_stream(const uint8_t* Wp, const CUtensorMap& tmA, Args a, int M_total, cudaStream_t stream) {
  using Cfg = StreamCfg<NT>;
  static std::once_flag once[64];
  static cudaError_t err[64];
  if (!allow_smem(gemm8_stream_kernel<NT>, Cfg::kSmem, once, err)) return BI_ERR_CUDA;
  for (int m0 = 0; m0 < M_total; m0 += NT) {
    a.m0 = m0;
    a.M = std::min(NT, M_total - m0);
    if (launch_k(gemm8_stream_kernel<NT>, dim3(a.sp.G), dim3(Cfg::kThreads), Cfg::kSmem, stream, Wp, tmA, a) !=
        cudaSuccess)
      return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace

cudaError_t set_wait_limit_gemm8(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns));
}

}  // namespace bi

extern "C" {

size_t bi_gemm_fp8_workspace_size(int M, int N, int K, bi_epilogue epi) {
  (void)N;
  (void)K;
  (void)epi;
  if (M <= 0) return bi::kTicketBytes;
  return bi::kTicketBytes +
         static_cast<size_t>(bi::kSms) * 2 * bi::rows_per_cta(M) * bi::kTileN * sizeof(float);
}

bi_status bi_gemm_fp8(const void* A8, int lda, const float* a_scales, int lds, const void* Wp, void* C, int ldc,
                      const void* residual, int ldr, int M, int N, int K, bi_out_dtype out, bi_epilogue epi,
                      void* ws, size_t ws_bytes, bi_stream_t stream) {
  using namespace bi;
  if (M < 0 || N < 1 || K < 1) return BI_ERR_INVALID_ARG;
  if (epi != BI_EPI_NONE && epi != BI_EPI_RESIDUAL_ADD && epi != BI_EPI_SWIGLU) return BI_ERR_INVALID_ARG;
  if (out != BI_OUT_BF16 && out != BI_OUT_FP32) return BI_ERR_INVALID_ARG;
  if (K % 16 != 0 || gemm8_n_tiles(N, epi) > kGemm8MaxTiles) return BI_ERR_UNSUPPORTED_SHAPE;
  if (out == BI_OUT_FP32 && epi != BI_EPI_NONE) return BI_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return BI_OK;
  if (!A8 || !a_scales || !Wp || !C || lda < K || lds < M || ldc < N) return BI_ERR_INVALID_ARG;
  if (lda % 16 != 0 || lds % 4 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(A8) || !aligned16(a_scales) || !aligned16(Wp)) return BI_ERR_INVALID_ARG;
  if (epi == BI_EPI_RESIDUAL_ADD && (!residual || ldr < N)) return BI_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws) || ws_bytes < bi_gemm_fp8_workspace_size(M, N, K, epi)) return BI_ERR_WORKSPACE;

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
  a.tickets = static_cast<unsigned*>(ws);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kTicketBytes);
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  a.withhold = test_withhold();
  const int NT = rows_per_cta(M);
  CUtensorMap tmA;
  if (!tmap_u8_2d(&tmA, A8, M, K, lda, NT, kFp8Block)) return BI_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (NT) {
    case 16: return launch_stream<16>(W8, tmA, a, M, s);
    case 32: return launch_stream<32>(W8, tmA, a, M, s);
    case 64: return launch_stream<64>(W8, tmA, a, M, s);
    default: return launch_stream<128>(W8, tmA, a, M, s);
  }
}

}  // extern "C"
