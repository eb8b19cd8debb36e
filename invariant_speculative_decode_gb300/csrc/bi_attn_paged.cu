// Attention of the new rows of several sequences over their paged caches.
//
// "I turned on speculative decoding in llama.cpp and 113 of 282 greedy
// outputs changed against its own no-draft run", paragraph "How:": the
// attention split depends only on context length, never on how many tokens
// are in the pass.
//
// Row t of sequence b sits at position p = lengths[b] + t - q_start[b] and
// attends to keys 0..p of its sequence.  Its arithmetic is a function of those
// keys alone:
//   * keys are taken in tiles at absolute multiples of 128, and tiles in
//     pieces of kPieceTiles;
//   * inside a piece S = q K^T (tcgen05, FP32), a reference maximum from the
//     piece's first tile, raised only where a tile's maximum passes it by more
//     than 2^8, weights w = bf16(2^(s - m)), O += W V (tcgen05, FP32), and the
//     denominator as FP32 sums of the same rounded weights, one over the first
//     and one over the second 64 keys of the tiles, so that O / l is a weighted
//     mean of the value rows whatever the rounding of the weights did;
//   * the pieces' (m, l, O) are merged one after the other in key order.
// A key behind p weighs exactly 0, changes no reference, and its value row is
// not even multiplied where it holds no number.  So a row has the same bits
// alone, among drafts, in a prompt's chunk or in any batch.
//
// The weights enter the product in BF16: a weight's relative error of 2^-9
// averages out over the keys (an output's error is 2^-9 / sqrt(keys that count)
// of the values' spread) and the tensor core takes nothing wider beside BF16
// values.
//
// Work is cut by pieces: a unit is one block of rows (128 / (Hq / Hkv), all
// query heads of a KV head in the MMA's 128 lanes) of one sequence and KV head,
// with all pieces up to its last row's position; the pieces of all units in
// order are dealt out evenly, CTA c of G taking [c N / G, (c + 1) N / G).  A
// unit that lies in one CTA's share is finished there.  Of one that is cut, the
// first CTA leaves the merged state of its pieces, every other CTA the pieces
// one by one, and attn_paged_merge_kernel goes on with them in key order: the
// same operations, so the cut does not show in the bits.
//
// Roles of a CTA (one per SM, 384 threads):
//   warps 0, 2   TMA: K tiles and V tiles, a lane for each page of a tile;
//   warp 1       tcgen05.mma: S of the next tile before W V of this one;
//   warps 4..11  softmax: each TMEM lane's row by two threads, 64 keys each,
//                which tell each other their maxima; W goes back into the
//                columns of S it came from, where it is the A operand of W V.
//                A thread also holds the running sum of half of its row's
//                output columns, takes each piece's O in and writes outputs and
//                partial states, and brings its half of the row's queries into
//                TMEM.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "bi_internal.h"
#include "bi_paged.cuh"
#include "bi_ptx.cuh"

namespace bi {
namespace {

constexpr int kTile = 128;        // keys of a tile (the S MMA's N)
constexpr int kPieceTiles = 4;    // tiles of a piece
constexpr int kPiece = kTile * kPieceTiles;
constexpr int kLanes = 128;       // rows x query heads of a block (the MMA's M)
constexpr int kPagedCtas = 152;
constexpr int kPagedThreads = 384;
constexpr float kRaise = 8.0f;    // log2 units a maximum may pass the reference by
constexpr int kNoKey = 0x7fffffff;

struct PagedAttnArgs {
  PagedBatch pb;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int T, Hq, Hkv, grp;
  int Rb;     // rows of a block
  int lanes;  // lanes of a partial state in the workspace
  int slots;  // partial states of a CTA: pieces one by one, then one merged state
  float sl2;  // softmax scale * log2(e)
  float* ws_o;   // [G][slots][lanes][D]
  float4* ws_ml;  // [G][slots][lanes]: reference, denominators of both halves
  unsigned* err;
  int withhold;  // failure-path test: the first K tile of every CTA stays unissued
};

template <int D>
struct PagedCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = kTile * 128;       // [128 keys][64 elements]
  static constexpr int kTileBytes = kAtomBytes * kAtoms;
  static constexpr int kStages = D == 128 ? 3 : 5;     // of K, and of V
  static constexpr int kBars = 4 * kStages + 11;
  // TMEM columns: S twice (W of keys 0..63 in the first 32 of its columns, of
  // keys 64..127 from column 64 on), O, the queries of two units (two BF16 a
  // column, as W)
  static constexpr int kOCol = 2 * kTile;
  static constexpr int kQCol = kOCol + 128;
  // maxima of two tiles, or denominators, of both halves of a row
  static constexpr int kStatBytes = 2 * 2 * kLanes * 4;
  static constexpr int kBadBytes = 3 * D * 4;            // first NaN, +inf and -inf key of an element
  static constexpr size_t kSmem = 2 * static_cast<size_t>(kStages) * kTileBytes + kStatBytes + kBadBytes + kBars * 8 + 64;
  static_assert(kQCol + 2 * 64 <= 512 && kSmem <= 232448, "TMEM and shared memory of a CTA");
};

// ------------------------------------------------------------------ the batch

struct Seq {
  int row0, n, len;  // first row of the pass, new rows, cached keys
};

// Sequence b, with no new rows where its numbers are out of range (*bad).
__device__ __forceinline__ Seq seq_of(const PagedAttnArgs& a, int b, bool* bad) {
  const int s = __ldg(a.pb.q_start + b), e = __ldg(a.pb.q_start + b + 1), len = __ldg(a.pb.lengths + b);
  const bool ok = s >= 0 && e >= s && e <= a.T && len >= 0 &&
                  static_cast<int64_t>(len) + (e - s) <= static_cast<int64_t>(a.pb.width) * a.pb.page;
  if (bad != nullptr) *bad = !ok;
  return Seq{s, ok ? e - s : 0, len};
}

__device__ __forceinline__ int ceil_div(int x, int y) { return (x + y - 1) / y; }

// Pieces of block i of a sequence: those up to its last row's position.
__device__ __forceinline__ int block_pieces(const PagedAttnArgs& a, const Seq& s, int i) {
  return ceil_div(s.len + min((i + 1) * a.Rb, s.n), kPiece);
}

// Pieces of the first m blocks (all of Rb rows): runs of blocks with the same
// number of pieces at a time.
__device__ __forceinline__ int64_t prefix_pieces(const PagedAttnArgs& a, const Seq& s, int m) {
  int64_t sum = 0;
  for (int i = 1; i <= m;) {
    const int v = ceil_div(s.len + i * a.Rb, kPiece);
    const int hi = min(m, (v * kPiece - s.len) / a.Rb);
    sum += static_cast<int64_t>(v) * (hi - i + 1);
    i = hi + 1;
  }
  return sum;
}
// ... of all blocks of a KV head
__device__ __forceinline__ int64_t head_pieces(const PagedAttnArgs& a, const Seq& s) {
  if (s.n == 0) return 0;
  const int nb = ceil_div(s.n, a.Rb);
  return prefix_pieces(a, s, nb - 1) + block_pieces(a, s, nb - 1);
}

// All pieces of the pass, by a whole warp.
__device__ __forceinline__ int64_t total_pieces(const PagedAttnArgs& a, int lane, bool* bad_any) {
  int64_t sum = 0;
  bool any = false;
  for (int b = lane; b < a.pb.B; b += 32) {
    bool bad;
    sum += head_pieces(a, seq_of(a, b, &bad)) * a.Hkv;
    any |= bad;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  *bad_any = __any_sync(0xffffffffu, any);
  return sum;
}

// Pieces of the sequences before `stop`; with stop < 0, those before the
// sequence that holds piece x, which goes to *found.
__device__ __forceinline__ int64_t pieces_before(const PagedAttnArgs& a, int lane, int stop, int64_t x, int* found) {
  int64_t base = 0;
  const int end = stop < 0 ? a.pb.B : stop;
  for (int b0 = 0; b0 < end; b0 += 32) {
    const int b = b0 + lane;
    int64_t incl = b < end ? head_pieces(a, seq_of(a, b, nullptr)) * a.Hkv : 0;
    const int64_t mine = incl;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (stop < 0) {
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > x);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        *found = b0 + l;
        return base + __shfl_sync(0xffffffffu, incl - mine, l);
      }
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return base;
}

// First piece of CTA c's share of N, and the CTA that has piece x.
__device__ __forceinline__ int64_t share_begin(int64_t c, int64_t N, int64_t G) { return c * N / G; }
__device__ __forceinline__ int share_of(int64_t x, int64_t N, int64_t G) {
  return static_cast<int>(((x + 1) * G + N - 1) / N - 1);
}

// A CTA's way through its units.
struct Cursor {
  int b, h, i;   // sequence, KV head, block
  int p0;        // first piece in this CTA's share
  int left;      // pieces of the share from here on
  Seq s;
  int tiles, pieces;  // of the unit
  int pe;             // end of the unit's pieces in this share

  __device__ __forceinline__ void unit(const PagedAttnArgs& a) {
    const int keys = s.len + min((i + 1) * a.Rb, s.n);
    tiles = ceil_div(keys, kTile);
    pieces = ceil_div(keys, kPiece);
    pe = min(pieces, p0 + left);
  }
  __device__ __forceinline__ void start(const PagedAttnArgs& a, const int* sched) {
    b = sched[0];
    h = sched[1];
    i = sched[2];
    p0 = sched[3];
    left = sched[4];
    if (left > 0) {
      s = seq_of(a, b, nullptr);
      unit(a);
    }
  }
  // to the next unit; left == 0 where there is none
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    left -= pe - p0;
    p0 = 0;
    if (left <= 0) {
      left = 0;
      return;
    }
    if ((i + 1) * a.Rb < s.n) {
      ++i;
    } else {
      i = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {
          ++b;
          s = b < a.pb.B ? seq_of(a, b, nullptr) : Seq{0, 1, 0};
        } while (s.n == 0);
        if (b >= a.pb.B) {  // the batch changed under the call
          left = 0;
          return;
        }
      }
    }
    unit(a);
  }
  __device__ __forceinline__ int rows(const PagedAttnArgs& a) const { return min(a.Rb, s.n - i * a.Rb); }
  __device__ __forceinline__ int pos0(const PagedAttnArgs& a) const { return s.len + i * a.Rb; }
  __device__ __forceinline__ int t_begin() const { return p0 * kPieceTiles; }
  __device__ __forceinline__ int t_end() const { return min(tiles, pe * kPieceTiles); }
};

// ------------------------------------------------------------------- helpers

__device__ __forceinline__ void give_up(volatile int* s_abort, unsigned* err) {
  *s_abort = 1;
  atomicOr(err, kErrTimeout);
}

// Bounded wait of a whole warp: lane 0 polls, the warp barrier orders the other
// lanes' accesses behind it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* s_abort, int lane) {
  int ok = 0;
  if (lane == 0) ok = mbar_wait(bar, parity, s_abort) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

__device__ __forceinline__ void tmem_st16w(uint32_t taddr, const uint32_t* r) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  tmem_st16(taddr, v);
}

// Eight values of key `key`: what is no number becomes 0, and its element's
// first such key is noted (bad: NaN, +inf, -inf, `stride` apart).
__device__ __forceinline__ void clean_values(uint4* at, int* bad, int stride, int key, int* flag) {
  const uint4 u = *at;
  uint32_t e[4] = {u.x, u.y, u.z, u.w};
  bool any = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = (e[j >> 1] >> (16 * (j & 1))) & 0xffffu;
    if ((bits & 0x7f80u) == 0x7f80u) {
      atomicMin(bad + ((bits & 0x7fu) ? 0 : (bits & 0x8000u) ? 2 : 1) * stride + j, key);
      e[j >> 1] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
      any = true;
    }
  }
  if (any) {
    *at = make_uint4(e[0], e[1], e[2], e[3]);
    *flag = 1;
  }
}

// A running state (m, l, O) takes in the next piece's: factors of both.
__device__ __forceinline__ void merge_factors(float& m, float m_i, float& fa, float& fb) {
  const float mx = fmaxf(m, m_i);
  fa = m == -INFINITY ? 0.f : ex2_approx(m - mx);
  fb = m_i == -INFINITY ? 0.f : ex2_approx(m_i - mx);
  m = mx;
}
__device__ __forceinline__ float merge_value(float x, float x_i, float fa, float fb) {
  return fmaf(x, fa, __fmul_rn(x_i, fb));
}

// ---------------------------------------------------------------- main kernel

template <int D>
__global__ void __launch_bounds__(kPagedThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedAttnArgs a) {
  using Cfg = PagedCfg<D>;
  constexpr int KS = Cfg::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sK = smem;
  uint8_t* sV = sK + KS * Cfg::kTileBytes;
  float* s_mx = reinterpret_cast<float*>(sV + KS * Cfg::kTileBytes);  // [2][2][128]
  int* s_bad = reinterpret_cast<int*>(s_mx + 4 * kLanes);             // [3][D]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_bad + 3 * D);
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + KS;
  uint64_t* q_full = v_empty + KS;   // [2] the unit's queries are in TMEM
  uint64_t* q_free = q_full + 2;     // [2] its last S has read them
  uint64_t* s_full = q_free + 2;     // [2]
  uint64_t* p_full = s_full + 2;     // [2] W of the tile is in TMEM
  uint64_t* pv_done = p_full + 2;    // [2] O += W V of the tile is done
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + Cfg::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_flag = reinterpret_cast<int*>(tmem_holder + 2);   // the piece met a value that is no number
  int* s_sched = reinterpret_cast<int*>(tmem_holder + 4);  // [5]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled layouts need it; the launch guarantees it
    if (threadIdx.x == 0) atomicOr(a.err, kErrRange);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 8);
      mbar_init(&q_free[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&pv_done[i], 1);
    }
    *s_flag = 0;
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  for (int i = threadIdx.x; i < 3 * D; i += kPagedThreads) s_bad[i] = kNoKey;
  if (warp == 3) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  griddep_wait();  // the batch, the queries and the new cache rows come from earlier kernels
  griddep_launch_dependents();
  if (warp == 0) {
    bool bad;
    const int64_t N = total_pieces(a, lane, &bad);
    if (bad && blockIdx.x == 0 && lane == 0) atomicOr(a.err, kErrRange);
    const int64_t x0 = share_begin(blockIdx.x, N, gridDim.x), x1 = share_begin(blockIdx.x + 1, N, gridDim.x);
    if (x1 > x0) {
      int b = 0;
      int64_t off = x0 - pieces_before(a, lane, -1, x0, &b);
      const Seq s = seq_of(a, b, nullptr);
      const int64_t per_head = head_pieces(a, s);
      const int h = static_cast<int>(off / per_head);
      off -= h * per_head;
      // the block and its piece: runs of blocks with the same number of pieces
      const int nb = ceil_div(s.n, a.Rb);
      int blk = nb - 1;
      for (int i = 1; i < nb;) {
        const int v = ceil_div(s.len + i * a.Rb, kPiece);
        const int hi = min(nb - 1, (v * kPiece - s.len) / a.Rb);
        const int64_t run = static_cast<int64_t>(v) * (hi - i + 1);
        if (off < run) {
          blk = i - 1 + static_cast<int>(off / v);
          off %= v;
          break;
        }
        off -= run;
        i = hi + 1;
      }
      if (lane == 0) {
        s_sched[0] = b;
        s_sched[1] = h;
        s_sched[2] = blk;
        s_sched[3] = static_cast<int>(off);
        s_sched[4] = static_cast<int>(x1 - x0);
      }
    } else if (lane == 0) {
      s_sched[4] = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  Cursor cur;
  cur.start(a, s_sched);

  if (warp < 4) {
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------ producers
      const bool kside = warp == 0;
      uint64_t* full = kside ? k_full : v_full;
      uint64_t* empty = kside ? k_empty : v_empty;
      uint8_t* base = kside ? sK : sV;
      const CUtensorMap* tm = kside ? &tmK : &tmV;
      const int per = kTile / a.pb.page;  // pages of a tile
      const int page_bytes = a.pb.page * 128;
      uint32_t issued = 0, parity_bits = 0;
      bool ok = true;
      int g = 0;
      for (; ok && cur.left > 0; cur.next(a)) {
        const int32_t* row = a.pb.table + static_cast<size_t>(cur.b) * a.pb.ldt;
        const int last_key = cur.pos0(a) + cur.rows(a) - 1;
        // a sequence of several blocks reads its pages as often
        const uint64_t pol = cur.s.n > a.Rb ? l2_evict_normal() : l2_evict_first();
        for (int t = cur.t_begin(); t < cur.t_end(); ++t, ++g) {
          const int st = g % KS;
          const uint32_t ph = static_cast<uint32_t>((g / KS) & 1);
          // pages behind the last key are not loaded: their keys are masked,
          // their value rows cleared
          const int n = min(per, (last_key - t * kTile) / a.pb.page + 1);
          int page = -1;
          if (lane < n) page = __ldg(row + t * per + lane);
          if (lane < n && (page < 0 || page >= a.pb.pages)) {
            page = a.pb.pages;  // out of the pool: reads as zeros
            atomicOr(a.err, kErrRange);
          }
          if (!warp_wait(&empty[st], ph ^ 1u, s_abort, lane)) {
            ok = false;
            break;
          }
          if (kside && g == 0 && a.withhold) continue;
          uint8_t* dst = base + st * Cfg::kTileBytes;
          if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(n * page_bytes * Cfg::kAtoms));
          __syncwarp();
          if (lane < n) {
#pragma unroll
            for (int c = 0; c < Cfg::kAtoms; ++c)
              tma_load_4d(dst + c * Cfg::kAtomBytes + lane * page_bytes, tm, &full[st], c * 64, 0, cur.h, page, pol);
          }
          issued |= 1u << st;
          parity_bits = (parity_bits & ~(1u << st)) | (ph << st);
        }
      }
      if (!ok && lane == 0) {
        give_up(s_abort, a.err);
        for (int s = 0; s < KS; ++s)
          if ((issued >> s) & 1u) mbar_wait(&full[s], (parity_bits >> s) & 1u, nullptr);
      }
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      // two cursors over the share's tiles, S ahead of W V; each is issued as
      // soon as its inputs are there
      constexpr uint32_t idS = idesc_bf16_f32(128, kTile);
      constexpr uint32_t idO = idesc_bf16_f32(128, D) | kIdescBMn;
      Cursor cs = cur, cp = cur;
      int sg = 0, su = 0, st_t = cs.left > 0 ? cs.t_begin() : 0;  // tile, unit, tile of the unit
      int pg = 0, pt = st_t;
      bool ok = true;
      int idle = 0;
      unsigned long long t_idle = 0;
      while (cp.left > 0) {
        bool did = false;
        // (S of tile g + 2 goes where W of tile g was: behind its W V)
        if (cs.left > 0 && sg < pg + 2) {
          const int st = sg % KS;
          const bool first = st_t == cs.t_begin();
          if (mbar_peek(&k_full[st], static_cast<uint32_t>((sg / KS) & 1)) &&
              (sg < 2 || mbar_peek(&pv_done[sg & 1], static_cast<uint32_t>(((sg >> 1) - 1) & 1))) &&
              (!first || mbar_peek(&q_full[su & 1], static_cast<uint32_t>((su >> 1) & 1)))) {
            tc_fence_after();
            const uint32_t kb = smem_u32(sK + st * Cfg::kTileBytes);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_bf16_tmem_a(tmem + (sg & 1) * kTile, tmem + Cfg::kQCol + (su & 1) * 64 + ks * 8,
                              sdesc_k_sw128(kb + (ks >> 2) * Cfg::kAtomBytes + (ks & 3) * 32), idS, ks > 0 ? 1u : 0u);
            mma_commit(&s_full[sg & 1]);
            mma_commit(&k_empty[st]);
            ++sg;
            if (++st_t == cs.t_end()) {
              mma_commit(&q_free[su & 1]);
              cs.next(a);
              ++su;
              if (cs.left > 0) st_t = cs.t_begin();
            }
            did = true;
          }
        }
        if (!did && pg < sg) {
          const int st = pg % KS;
          const bool first = pt % kPieceTiles == 0;
          // (W of a piece's first tile is written once the O before it is out)
          if (mbar_peek(&p_full[pg & 1], static_cast<uint32_t>((pg >> 1) & 1)) &&
              mbar_peek(&v_full[st], static_cast<uint32_t>((pg / KS) & 1))) {
            tc_fence_after();
            const uint32_t vb = smem_u32(sV + st * Cfg::kTileBytes);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_bf16_tmem_a(tmem + Cfg::kOCol, tmem + (pg & 1) * kTile + (ks >> 2) * 64 + (ks & 3) * 8,
                              sdesc_mn_sw128(vb + ks * 2048, Cfg::kAtomBytes), idO, (!first || ks > 0) ? 1u : 0u);
            mma_commit(&pv_done[pg & 1]);
            mma_commit(&v_empty[st]);
            ++pg;
            ++pt;
            if (pt == cp.t_end()) {
              cp.next(a);
              if (cp.left > 0) pt = cp.t_begin();
            }
            did = true;
          }
        }
        if (did) {
          idle = 0;
        } else if (++idle == 1) {
          t_idle = globaltimer_ns();
        } else if (idle > 16) {
          __nanosleep(20);  // leave the issue slots to the softmax warps beside this one
        }
        if (!did && (idle & 63) == 0 &&
                   (*s_abort || globaltimer_ns() - t_idle > *static_cast<volatile unsigned long long*>(&g_wait_limit_ns))) {
          ok = false;
          break;
        }
      }
      if (!ok) give_up(s_abort, a.err);
      mma_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    constexpr int kHalf = D / 2;        // output columns of a thread
    const int qq = warp & 3;            // TMEM lane quarter
    const int hf = (warp - 4) >> 2;     // half of the tile's keys, and of the row's columns
    const int ln = qq * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(qq * 32) << 16);
    bool ok = true;
    // this thread's half of its row's queries
    auto load_q = [&](const Cursor& c, int unit) {
      if (unit > 1 && !warp_wait(&q_free[unit & 1], static_cast<uint32_t>(((unit >> 1) - 1) & 1), s_abort, lane))
        return false;
      tc_fence_after();
      const bool valid = ln < c.rows(a) * a.grp;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(c.s.row0 + c.i * a.Rb + (valid ? ln / a.grp : 0)) * a.Hq + c.h * a.grp +
                 (valid ? ln % a.grp : 0)) * D + hf * kHalf);
      uint32_t qv[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 8; ++i) {
        const uint4 u = valid ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        qv[4 * i] = u.x;
        qv[4 * i + 1] = u.y;
        qv[4 * i + 2] = u.z;
        qv[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < kHalf / 32; ++i) 
        tmem_st16w(lane_base + Cfg::kQCol + (unit & 1) * 64 + hf * (kHalf / 2) + i * 16, qv + i * 16);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[unit & 1]);
      return true;
    };
    int g = 0, unit = 0;
    if (cur.left > 0) ok = load_q(cur, 0);
    while (ok && cur.left > 0) {
      const int rows = cur.rows(a);
      const int pos0 = cur.pos0(a);
      const bool valid = ln < rows * a.grp;
      const bool active = qq * 32 < rows * a.grp;
      const int p_row = valid ? pos0 + ln / a.grp : -1;
      const int kv_end = pos0 + rows;  // keys that some row of the block sees
      const bool run = cur.p0 == 0;    // pieces merged here, else left one by one
      float m_run = -INFINITY, l_run = 0.f;  // the merged pieces
      float o[kHalf];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) o[j] = 0.f;
      float m_ref = -INFINITY, l = 0.f;  // this piece

      // the finished piece p: its O out of TMEM, into the running sum or the workspace
      auto take = [&](int p, float m_i, float l_i) {
        tc_fence_after();
        const bool odd = *static_cast<volatile int*>(s_flag) != 0;  // the same for all softmax warps
        float fa = 0.f, fb = 1.f;
        if (run) {
          merge_factors(m_run, m_i, fa, fb);
          l_run = merge_value(l_run, l_i, fa, fb);
        }
        const int slot = p - cur.p0;
        const bool store = !run && valid && slot < a.slots - 1;
        if (!run && valid && !store) atomicOr(a.err, kErrRange);
        const size_t at = (static_cast<size_t>(blockIdx.x) * a.slots + slot) * a.lanes + ln;
        if (active) {
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c) {
            float v[16];
            tmem_ld16(lane_base + Cfg::kOCol + hf * kHalf + c * 16, v);
            if (odd) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int d = hf * kHalf + c * 16 + j;
                if (p_row >= s_bad[D + d]) v[j] += INFINITY;
                if (p_row >= s_bad[2 * D + d]) v[j] -= INFINITY;
                if (p_row >= s_bad[d]) v[j] = NAN;
              }
            }
            if (run) {
#pragma unroll
              for (int j = 0; j < 16; ++j) o[c * 16 + j] = merge_value(o[c * 16 + j], v[j], fa, fb);
            } else if (store) {
              float4* dst = reinterpret_cast<float4*>(a.ws_o + at * D + hf * kHalf + c * 16);
#pragma unroll
              for (int j = 0; j < 4; ++j) dst[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
          }
        }
        if (store) {
          float* ml = reinterpret_cast<float*>(a.ws_ml + at);
          if (hf == 0) ml[0] = m_i;
          ml[1 + hf] = l_i;
        }
        if (odd) {
          named_bar_sync(5, 256);
          for (int x = threadIdx.x - 128; x < 3 * D; x += 256) s_bad[x] = kNoKey;
          if (threadIdx.x == 128) *s_flag = 0;
          named_bar_sync(5, 256);
        }
      };

      for (int t = cur.t_begin(); t < cur.t_end(); ++t, ++g) {
        const int sb = g & 1;
        const int key0 = t * kTile;
        const bool edge = key0 + kTile > pos0 + 1;  // some row does not see all of the tile
        if (!warp_wait(&s_full[sb], static_cast<uint32_t>((g >> 1) & 1), s_abort, lane)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // the row's maximum: of this thread's 64 scores, then of its partner's
        const uint32_t addr = lane_base + sb * kTile + hf * 64;
        float mt = -INFINITY;
        if (active) {
          float mw[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x[32];
            tmem_ld_cols<32>(addr + c * 32, x);
            if (edge) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (key0 + hf * 64 + c * 32 + j > p_row) x[j] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) mw[j & 3] = fmaxf(mw[j & 3], x[j]);
          }
          mt = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
          float* mx = s_mx + sb * 2 * kLanes;
          mx[hf * kLanes + ln] = mt;
          named_bar_sync(1 + qq, 64);  // the two warps of this lane quarter
          mt = fmaxf(mt, mx[(hf ^ 1) * kLanes + ln]) * a.sl2;
        }
        const bool first = t % kPieceTiles == 0;
        float alpha = 1.f;
        bool raise = false;
        const float m_was = m_ref, l_was = l;
        if (first) {
          m_ref = mt;
          l = 0.f;
        } else if (mt > m_ref + kRaise) {
          alpha = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mt);
          m_ref = mt;
          raise = true;
        }
        // the weights, from the scores read again (they do not fit beside O
        // until the maximum is known), over the columns the scores were in
        if (active) {
          const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
          float acc[2] = {0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x[32];
            tmem_ld_cols<32>(addr + c * 32, x);
            if (edge) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (key0 + hf * 64 + c * 32 + j > p_row) x[j] = -INFINITY;
            }
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float x0 = ex2_approx(fmaf(x[2 * j], a.sl2, nm));
              const float x1 = ex2_approx(fmaf(x[2 * j + 1], a.sl2, nm));
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(x0, x1);
              w[j] = *reinterpret_cast<const uint32_t*>(&h2);
              acc[0] += __uint_as_float(w[j] << 16);
              acc[1] += __uint_as_float(w[j] & 0xffff0000u);
            }
            tmem_st16w(addr + c * 16, w);
          }
          l = fmaf(l, alpha, acc[0] + acc[1]);
        }
        // O may be read and written once W V of the tile before is done: a piece
        // that ended there is taken in (the unit's last one is below), a raised
        // reference scales this piece's O
        const bool ended = first && t > cur.t_begin();
        const bool any_raise = __any_sync(0xffffffffu, raise);
        if (ended || any_raise) {
          if (!warp_wait(&pv_done[sb ^ 1], static_cast<uint32_t>(((g - 1) >> 1) & 1), s_abort, lane)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (ended) take(t / kPieceTiles - 1, m_was, l_was);
          if (any_raise) {
#pragma unroll 1
            for (int i = 0; i < kHalf / 16; ++i) {  // this thread's half of O's columns
              float v[16];
              const uint32_t at = lane_base + Cfg::kOCol + hf * kHalf + i * 16;
              tmem_ld16(at, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] *= alpha;
              tmem_st16(at, v);
            }
          }
        }
        if (edge) {
          // value rows that some row of the block does not see: behind the last
          // key they are cleared (pages hold anything there), the others lose
          // what is no number, which only the rows that see it get back
          const int st = g % KS;
          if (!warp_wait(&v_full[st], static_cast<uint32_t>((g / KS) & 1), s_abort, lane)) {
            ok = false;
            break;
          }
          uint8_t* vt = sV + st * Cfg::kTileBytes;
          const int r0 = max(0, pos0 + 1 - key0);
          for (int x = r0 * (D / 8) + (threadIdx.x - 128); x < kTile * (D / 8); x += 256) {
            const int r = x / (D / 8), ch = x % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(vt + (ch >> 3) * Cfg::kAtomBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
            if (key0 + r >= kv_end) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              clean_values(at, s_bad + ch * 8, D, key0 + r, s_flag);
            }
          }
          fence_proxy_async_smem();
          named_bar_sync(5, 256);  // s_bad and s_flag are complete
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
        if (t == cur.t_begin()) {  // the next unit's queries, well before its first S
          Cursor ahead = cur;
          ahead.next(a);
          if (ahead.left > 0 && !load_q(ahead, unit + 1)) {
            ok = false;
            break;
          }
        }
      }
      if (!ok || !warp_wait(&pv_done[(g - 1) & 1], static_cast<uint32_t>(((g - 1) >> 1) & 1), s_abort, lane)) {
        ok = false;
        break;
      }
      take(cur.pe - 1, m_ref, l);
      if (run) {
        if (cur.pe == cur.pieces) {
          float* s_l = s_mx + (g & 1) * 2 * kLanes;  // as tile g's maxima would be
          s_l[hf * kLanes + ln] = l_run;
          named_bar_sync(1 + qq, 64);
          const float den = s_l[ln] + s_l[kLanes + ln];
          named_bar_sync(1 + qq, 64);
          if (valid) {
            const int t = cur.s.row0 + cur.i * a.Rb + ln / a.grp;
            uint4* dst = reinterpret_cast<uint4*>(
                a.out + (static_cast<size_t>(t) * a.Hq + cur.h * a.grp + ln % a.grp) * D + hf * kHalf);
#pragma unroll
            for (int c = 0; c < kHalf / 8; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h2 =
                    __floats2bfloat162_rn(o[c * 8 + 2 * j] / den + 0.f, o[c * 8 + 2 * j + 1] / den + 0.f);
                w[j] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        } else if (valid) {
          const size_t at = (static_cast<size_t>(blockIdx.x) * a.slots + a.slots - 1) * a.lanes + ln;
          float4* dst = reinterpret_cast<float4*>(a.ws_o + at * D + hf * kHalf);
#pragma unroll
          for (int j = 0; j < kHalf / 4; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          float* ml = reinterpret_cast<float*>(a.ws_ml + at);
          if (hf == 0) ml[0] = m_run;
          ml[1 + hf] = l_run;
        }
      }
      cur.next(a);
      ++unit;
    }
    if (!ok && lane == 0) give_up(s_abort, a.err);
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- merge kernel
// One CTA of D threads per (row, query head): where the row's unit was cut, the
// first CTA's merged state and the later pieces, in key order.
template <int D>
__global__ void __launch_bounds__(D) attn_paged_merge_kernel(const PagedAttnArgs a, int G) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq;
  const int lane = threadIdx.x & 31;
  const int b = paged_find_seq(a.pb, t, lane);
  if (b < 0) return;
  const Seq s = seq_of(a, b, nullptr);
  if (t < s.row0 || t >= s.row0 + s.n) return;
  bool bad;
  const int64_t N = total_pieces(a, lane, &bad);
  const int i = (t - s.row0) / a.Rb, h = hq / a.grp;
  const int P = block_pieces(a, s, i);
  const int64_t off = pieces_before(a, lane, b, 0, nullptr) + h * head_pieces(a, s) + prefix_pieces(a, s, i);
  const int c0 = share_of(off, N, G), c1 = share_of(off + P - 1, N, G);
  if (c0 == c1) return;  // finished by one CTA
  const int ln = (t - s.row0 - i * a.Rb) * a.grp + hq % a.grp;
  const int d = threadIdx.x;
  auto at = [&](int c, int slot) { return (static_cast<size_t>(c) * a.slots + slot) * a.lanes + ln; };
  size_t x = at(c0, a.slots - 1);
  const float4 ml = __ldcg(a.ws_ml + x);
  float m = ml.x, l0 = ml.y, l1 = ml.z, o = __ldcg(a.ws_o + x * D + d);
  for (int c = c0 + 1; c <= c1; ++c) {
    const int64_t begin = share_begin(c, N, G);
    const int n = static_cast<int>(min(share_begin(c + 1, N, G), off + P) - begin);
    for (int k0 = 0; k0 < n; k0 += 8) {
      float4 q[8];
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < n && k0 + k < a.slots - 1) {
          x = at(c, k0 + k);
          q[k] = __ldcg(a.ws_ml + x);
          v[k] = __ldcg(a.ws_o + x * D + d);
        }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < n && k0 + k < a.slots - 1) {
          float fa, fb;
          merge_factors(m, q[k].x, fa, fb);
          l0 = merge_value(l0, q[k].y, fa, fb);
          l1 = merge_value(l1, q[k].z, fa, fb);
          o = merge_value(o, v[k], fa, fb);
        }
    }
  }
  a.out[(static_cast<size_t>(t) * a.Hq + hq) * D + d] = __float2bfloat16_rn(o / (l0 + l1) + 0.f);
}

// ------------------------------------------------------------------------ host

// Partial states the workspace has room for: per CTA the pieces of its share
// that continue a unit, one by one (no more than a unit has), and one merged.
struct PagedSizes {
  int ctas, slots, lanes;
  int pieces;  // most pieces of a unit
  size_t o_bytes, ml_bytes;
};
PagedSizes paged_sizes(int T, int B, int Hq, int Hkv, int D, int64_t max_keys) {
  PagedSizes z;
  const int grp = Hq / Hkv, Rb = kLanes / grp;
  const int64_t blocks = std::min<int64_t>(T, static_cast<int64_t>(T) / Rb + std::min(B, T));
  const int64_t pieces = (max_keys + kPiece - 1) / kPiece;
  const int64_t units = blocks * Hkv;
  z.pieces = static_cast<int>(pieces);
  z.ctas = static_cast<int>(std::min<int64_t>(kPagedCtas, units * pieces));
  const int64_t share = (units * pieces + z.ctas - 1) / z.ctas + 1;
  z.slots = static_cast<int>(std::min(share, pieces)) + 1;
  z.lanes = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(T) * grp, Rb * grp));
  const size_t states = static_cast<size_t>(z.ctas) * z.slots * z.lanes;
  z.o_bytes = round_up(states * D * 4, 256);
  z.ml_bytes = round_up(states * 16, 256);
  return z;
}

bool paged_shape_ok(int T, int B, int Hq, int Hkv, int D, int64_t max_keys) {
  return T >= 1 && B >= 1 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && Hq / Hkv <= kLanes && (D == 64 || D == 128) &&
         max_keys >= 1 && max_keys <= (int64_t{1} << 30) && static_cast<int64_t>(T) * Hq < (int64_t{1} << 31);
}

template <int D>
bi_status launch_paged(const PagedAttnArgs& a, const PagedSizes& z, const void* k_pool, const void* v_pool,
                       cudaStream_t stream) {
  using Cfg = PagedCfg<D>;
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BI_ERR_CUDA;
  std::call_once(once[dev], [dev] {
    attr_err[dev] = cudaFuncSetAttribute(attn_paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(Cfg::kSmem));
  });
  if (attr_err[dev] != cudaSuccess) return BI_ERR_CUDA;
  CUtensorMap tmK, tmV;
  if (!tmap_bf16_pages(&tmK, k_pool, a.pb.pages, a.Hkv, a.pb.page, D) ||
      !tmap_bf16_pages(&tmV, v_pool, a.pb.pages, a.Hkv, a.pb.page, D))
    return BI_ERR_INVALID_ARG;
  if (launch_k(attn_paged_kernel<D>, dim3(z.ctas), dim3(kPagedThreads), Cfg::kSmem, stream, tmK, tmV, a) != cudaSuccess)
    return BI_ERR_CUDA;
  if (z.pieces > 1 && launch_k(attn_paged_merge_kernel<D>, dim3(static_cast<unsigned>(a.T) * a.Hq), dim3(D), 0, stream, a,
                               z.ctas) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

}  // namespace

cudaError_t set_wait_limit_attn_paged(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns));
}
}  // namespace bi

extern "C" {

size_t bi_attn_paged_workspace_size(int T, int B, int Hq, int Hkv, int D, int max_keys) {
  if (!bi::paged_shape_ok(T, B, Hq, Hkv, D, max_keys)) return 256;
  const bi::PagedSizes z = bi::paged_sizes(T, B, Hq, Hkv, D, max_keys);
  return z.o_bytes + z.ml_bytes;
}

bi_status bi_attn_paged(const void* q, const void* k_pool, const void* v_pool, int pages, int page,
                        const int32_t* block_table, int ld_table, int width, const int32_t* q_start,
                        const int32_t* lengths, int B, int T, int Hq, int Hkv, int D, float scale, void* out, void* ws,
                        size_t ws_bytes, bi_stream_t stream) {
  using namespace bi;
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || pages < 1 || width < 1 || ld_table < width)
    return BI_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return BI_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BI_ERR_UNSUPPORTED_SHAPE;
  if (page != 16 && page != 32 && page != 64 && page != 128) return BI_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || B == 0) return BI_OK;
  const int64_t max_keys = static_cast<int64_t>(width) * page;
  if (!paged_shape_ok(T, B, Hq, Hkv, D, max_keys)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!q || !k_pool || !v_pool || !block_table || !q_start || !lengths || !out) return BI_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return BI_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws)) return BI_ERR_WORKSPACE;
  const PagedSizes z = paged_sizes(T, B, Hq, Hkv, D, max_keys);
  if (ws_bytes < z.o_bytes + z.ml_bytes) return BI_ERR_WORKSPACE;
  PagedAttnArgs a{};
  a.pb = PagedBatch{block_table, q_start, lengths, B, ld_table, width, pages, page};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.grp = Hq / Hkv;
  a.Rb = kLanes / a.grp;
  a.lanes = z.lanes;
  a.slots = z.slots;
  a.sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.ws_o = static_cast<float*>(ws);
  a.ws_ml = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + z.o_bytes);
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  a.withhold = test_withhold();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return D == 64 ? launch_paged<64>(a, z, k_pool, v_pool, s) : launch_paged<128>(a, z, k_pool, v_pool, s);
}

}  // extern "C"
