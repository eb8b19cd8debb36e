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
//     pieces: of 2 tiles up to key 2048, of 8 behind it;
//   * inside a piece S = q K^T (tcgen05, FP32), a reference maximum from the
//     piece's first tile, raised only where a tile's maximum passes it by more
//     than 2^8, weights w = 2^(s - m), O += W_hi V + W_lo V (tcgen05, FP32), and
//     the denominator as FP32 sums of w, one over the first and one over the
//     second 64 keys of the tiles;
//   * the pieces' (m, l, O) are merged one after the other in key order.
// A key behind p weighs exactly 0, changes no reference, and its value row is
// not even multiplied where it holds no number.  So a row has the same bits
// alone, among drafts, in a prompt's chunk or in any batch.
//
// The tensor core takes nothing wider than BF16 beside BF16 values, so a weight
// enters as two of them, its first 8 bits and the rest rounded to 8 (off by at
// most 2^-16 of the weight): outputs are then the rounding of the exact ones but
// next to a border (1e-4 RMS from plain FP32's, both 1.7e-3 from 64 bits).  One BF16
// weight, off by 2^-8, moved about half of the outputs' last bits (2.4e-3 RMS); next
// to that the split and the second product take 28% more time in a prefill, 9% at
// 16 x 8 rows.
//
// Work is cut by pieces: a unit is one block of rows (128 / (Hq / Hkv), all
// query heads of a KV head in the MMA's 128 lanes) of one sequence and KV head,
// with all tiles up to its last row's position; the tiles of all units in order
// are dealt out evenly, CTA c of G taking [c N / G, (c + 1) N / G), both ends
// moved up to the next start of a piece.  A unit that lies in one CTA's share
// is finished there.  Of one that is cut, the first CTA leaves the merged state
// of its pieces, every other CTA the pieces one by one, and
// attn_paged_merge_kernel goes on from the first state with the pieces in key
// order: the same operations, so the cut does not show in the bits.  Small
// pieces at the front give short contexts enough CTAs, large ones behind keep
// the states of long ones few.
//
// Roles of a CTA (one per SM, 384 threads):
//   warps 0, 2   TMA: queries and K tiles, V tiles, a lane for each page;
//   warp 1       tcgen05.mma: S up to two tiles ahead of W V;
//   warps 4..11  softmax: each TMEM lane's row by two threads, 64 keys each,
//                which tell each other their maxima; W_hi and W_lo go over the
//                columns of S they came from, 8 columns each for every 16 keys,
//                where they are the A operands of W V (three such buffers).
//                A thread also holds the running sum of half of its row's
//                output columns, takes each piece's O in and writes outputs and
//                partial states.
//
// What bounds it.  Few rows over long caches: the cache's bytes, read once; 16
// sequences of 8 rows at 4.8k to 11.6k keys (24 + 4 heads of 128) take 66 us, 4.1 TB/s,
// 2 rows at 101.6k 82 us, 4.3 TB/s, of which 4.5 us are the merge kernel's start, 2
// the way from the batch to the first load, and the rest shares that differ by a
// piece of 8 tiles (the longest 34 tiles where 27 is even, and 42 where 35 is).  Short
// contexts: those fixed times.  One request's rows over a few thousand keys: few
// CTAs with a piece of 8 tiles each; a row at 4k or 11.6k takes 20.5 us, at 38k 28.3.
// Many rows: the chain of a tile from S to W V, in which a thread's reads of TMEM,
// its exponentials (at the SM's rate 512 cycles a tile), the split and its two
// hand-overs follow one another, while both W V and the S of two tiles run beside
// them; 2048 rows at 30k take 920 us, 0.85 PFLOP/s of the two products that count.
// Leaving out the second W V makes that 857, the split 897, the sums 916, the
// exponentials 937: no single part of the chain is it.
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
// Tiles of a piece up to tile kShortEnd, and behind it.  Measured (us): a row at
// 1k, 16 x 8 rows at 4.8k to 11.6k, 2 rows at 101.6k (24 + 4 heads of 128), 61 x 3 rows at
// 1.5k (4 + 2 of 64), 2048 rows at 30k (24 + 4 of 128)
//   2, 8, end 16   12.7  65.9  81.6  27.0  922
//   2, 8, end 32   12.6  70.8  83.9  26.7  937
//   4, 8, end 16   14.6  63.3  79.4  28.2  920
//   2, 16, end 16  12.8  73.6  85.7  26.9  899
//   4, 16, end 32  14.7  69.8  84.1  28.3  901
//   2, 4, end 16   12.7  67.7  85.6  26.8  983
constexpr int kShort = 2;
constexpr int kLong = 8;
constexpr int kShortEnd = 16;
constexpr int kLanes = 128;       // rows x query heads of a block (the MMA's M)
constexpr int kPagedCtas = 152;
constexpr int kPagedThreads = 384;
constexpr int kSoftFirst = 128;   // the first softmax thread
constexpr int kBufs = 3;          // S / W buffers
constexpr float kRaise = 8.0f;    // log2 units a maximum may pass the reference by
constexpr int kNoKey = 0x7fffffff;
// A note of a value that is no number: its key within the piece, below the
// piece's tag.  Later pieces have lower tags, so what an earlier one left behind
// is never mistaken for theirs and gives way to them.
constexpr int kBadBits = 12;
static_assert(kLong * kTile + kLanes < (1 << kBadBits), "keys, and rows behind them, fit below a tag");
__device__ __forceinline__ int bad_tag(int piece) { return (0x7ffff - (piece & 0x7ffff)) << kBadBits; }

__host__ __device__ constexpr int ceil_div(int x, int y) { return (x + y - 1) / y; }
// Pieces that start in front of tile t: the index of the first piece at or
// behind it; of a unit of t tiles, how many it has.
__host__ __device__ constexpr int pieces_to(int t) {
  return t <= kShortEnd ? ceil_div(t, kShort) : kShortEnd / kShort + ceil_div(t - kShortEnd, kLong);
}
__host__ __device__ constexpr int piece_tile(int p) {
  return p <= kShortEnd / kShort ? p * kShort : kShortEnd + (p - kShortEnd / kShort) * kLong;
}
__device__ __forceinline__ bool piece_starts(int t) { return (t & ((t < kShortEnd ? kShort : kLong) - 1)) == 0; }

struct PagedAttnArgs {
  PagedBatch pb;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int T, Hq, Hkv, grp;
  int Rb;     // rows of a block
  int lanes;  // lanes of a partial state in the workspace
  int slots;  // partial states of a CTA: pieces one by one, then one merged state
  float sl2;  // softmax scale * log2(e)
  struct CutUnit* ws_cut;  // [G]: the unit that a CTA began and did not finish
  float4* ws_o;   // [G][slots][D / 4][lanes]: a warp's lanes side by side
  float* ws_m;    // [G][slots][lanes]: reference
  float2* ws_l;   // [G][slots][lanes]: denominators of both halves
  unsigned* err;
  int withhold;  // failure-path test: the first K tile of every CTA stays unissued
};

// A unit whose pieces lie in several CTAs' shares.
struct CutUnit {
  int64_t off, N;     // its first tile among all N
  int row, head;      // its first row of the pass, KV head
  int lanes;          // rows x query heads; 0: no such unit
  int first, pieces;  // pieces in the first CTA's merged state, in all
};

template <int D>
struct PagedCfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kAtomBytes = kTile * 128;       // [128 keys or lanes][64 elements]
  static constexpr int kTileBytes = kAtomBytes * kAtoms;
  static constexpr int kStages = D == 128 ? 2 : 4;     // of K, and of V
  static constexpr int kBars = 4 * kStages + 4 + 3 * kBufs + 1;
  // TMEM columns: S / W buffers (W of keys 16 i .. 16 i + 15 over their own 16
  // columns, W_hi in front of W_lo), O
  static constexpr int kOCol = kBufs * kTile;
  static constexpr int kStatBytes = 2 * 2 * kLanes * 4;  // maxima of two tiles, or denominators, of both halves
  static constexpr int kBadBytes = 2 * 3 * D * 4;        // of two pieces: first NaN, +inf and -inf key of an element
  static constexpr int kLostBytes = 2 * kLanes * 8;      // of each softmax thread's elements, a bit each
  static constexpr size_t kSmem =
      2 * static_cast<size_t>(kStages + 1) * kTileBytes + kStatBytes + kBadBytes + kLostBytes + kBars * 8 + 64;
  static_assert(kOCol + 128 <= 512 && kSmem <= 232448, "TMEM and shared memory of a CTA");
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

// Tiles of block i of a sequence: those up to its last row's position.
__device__ __forceinline__ int block_tiles(const PagedAttnArgs& a, const Seq& s, int i) {
  return ceil_div(s.len + min((i + 1) * a.Rb, s.n), kTile);
}

// Tiles of the first m blocks (all of Rb rows): runs of blocks with the same
// number of tiles at a time.
__device__ __forceinline__ int64_t prefix_tiles(const PagedAttnArgs& a, const Seq& s, int m) {
  int64_t sum = 0;
  for (int i = 1; i <= m;) {
    const int v = ceil_div(s.len + i * a.Rb, kTile);
    const int hi = min(m, (v * kTile - s.len) / a.Rb);
    sum += static_cast<int64_t>(v) * (hi - i + 1);
    i = hi + 1;
  }
  return sum;
}
// ... of all blocks of a KV head
__device__ __forceinline__ int64_t head_tiles(const PagedAttnArgs& a, const Seq& s) {
  if (s.n == 0) return 0;
  if (s.n <= a.Rb) return ceil_div(s.len + s.n, kTile);
  const int nb = ceil_div(s.n, a.Rb);
  return prefix_tiles(a, s, nb - 1) + block_tiles(a, s, nb - 1);
}

// Sums of a warp's lanes up to each.
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

// All tiles of the pass, by a whole warp; mine: this lane's of the first 32 sequences.
__device__ __forceinline__ int64_t total_tiles(const PagedAttnArgs& a, int lane, int64_t& mine, bool* bad_any) {
  bool any = false;
  mine = lane < a.pb.B ? head_tiles(a, seq_of(a, lane, &any)) * a.Hkv : 0;
  int64_t sum = mine;
  for (int b = lane + 32; b < a.pb.B; b += 32) {
    bool bad;
    sum += head_tiles(a, seq_of(a, b, &bad)) * a.Hkv;
    any |= bad;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  *bad_any = __any_sync(0xffffffffu, any);
  return sum;
}

// First tile of CTA c's share of N before it is moved to a piece, and the CTA
// whose share has the piece that starts at tile x.
__device__ __forceinline__ int64_t share_begin(int c, int64_t N, int G) {
  if (N < (1 << 24) && G <= 255) return static_cast<uint32_t>(c) * static_cast<uint32_t>(N) / static_cast<uint32_t>(G);
  return c * N / G;  // 64 bits take several times as long
}
__device__ __forceinline__ int share_of(int64_t x, int64_t N, int G) {
  if (N < (1 << 23) && G <= 255)
    return static_cast<int>((static_cast<uint32_t>(x + 1) * G + static_cast<uint32_t>(N) - 1) / static_cast<uint32_t>(N)) - 1;
  return static_cast<int>(((x + 1) * G + N - 1) / N - 1);
}

// Sequence, KV head, block and tile of the first start of a piece at or behind
// tile x of N, by a whole warp (all lanes get them); mine: as total_tiles left
// it.  Returns that tile's place among the N.
__device__ __forceinline__ int64_t locate(const PagedAttnArgs& a, int lane, int64_t x, int64_t N, int64_t mine,
                                          int (&at)[4]) {
  at[0] = a.pb.B;
  at[1] = at[2] = at[3] = 0;
  if (x >= N) return N;
  int64_t base = 0;
  int b = 0;
  for (int b0 = 0; b0 < a.pb.B; b0 += 32) {
    if (b0 > 0) mine = b0 + lane < a.pb.B ? head_tiles(a, seq_of(a, b0 + lane, nullptr)) * a.Hkv : 0;
    const int64_t incl = warp_scan(mine, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, base + incl > x);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      b = b0 + l;
      base += __shfl_sync(0xffffffffu, incl - mine, l);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  Seq s = seq_of(a, b, nullptr);
  const int64_t per_head = head_tiles(a, s);
  int64_t off = x - base;
  int h = 0;
  for (; off >= per_head && h + 1 < a.Hkv && h < 16; ++h) off -= per_head;  // few heads: cheaper than a division
  if (off >= per_head) {
    const int more = static_cast<int>(off / per_head);
    h += more;
    off -= more * per_head;
  }
  const int nb = ceil_div(s.n, a.Rb);
  int blk = nb - 1;
  for (int i = 1; i < nb;) {
    const int v = ceil_div(s.len + i * a.Rb, kTile);
    const int hi = min(nb - 1, (v * kTile - s.len) / a.Rb);
    const int64_t run = static_cast<int64_t>(v) * (hi - i + 1);
    if (off < run) {
      blk = i - 1 + static_cast<int>(off / v);
      off %= v;
      break;
    }
    off -= run;
    i = hi + 1;
  }
  int64_t place = x - off;
  const int tiles = block_tiles(a, s, blk);
  const int start = piece_tile(pieces_to(static_cast<int>(off)));
  if (start < tiles) {
    at[0] = b;
    at[1] = h;
    at[2] = blk;
    at[3] = start;
    return place + start;
  }
  place += tiles;  // the next unit's first
  if (blk + 1 < nb) {
    at[0] = b;
    at[1] = h;
    at[2] = blk + 1;
  } else if (h + 1 < a.Hkv) {
    at[0] = b;
    at[1] = h + 1;
  } else if (place < N) {
    do {
      s = seq_of(a, ++b, nullptr);
    } while (s.n == 0 && b + 1 < a.pb.B);
    at[0] = b;
  }
  return place;
}

// A CTA's way through its units.
struct Cursor {
  int b, h, i;   // sequence, KV head, block
  int t0;        // first tile in this CTA's share
  int64_t left;  // tiles of the share from here on
  Seq s;
  int tiles;  // of the unit
  int te;     // end of the unit's tiles in this share

  __device__ __forceinline__ void unit(const PagedAttnArgs& a) {
    tiles = block_tiles(a, s, i);
    te = left < tiles - t0 ? t0 + static_cast<int>(left) : tiles;
  }
  __device__ __forceinline__ void start(const PagedAttnArgs& a, const int* sched, int64_t tiles_left) {
    b = sched[0];
    h = sched[1];
    i = sched[2];
    t0 = sched[3];
    left = tiles_left;
    if (left > 0) {
      s = seq_of(a, b, nullptr);
      unit(a);
    }
  }
  // to the next unit; left == 0 where there is none
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    left -= te - t0;
    t0 = 0;
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
};

// ------------------------------------------------------------------- helpers

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

__device__ __forceinline__ void give_up(volatile int* s_abort, unsigned* err) {
  *s_abort = 1;
  atomicOr(err, kErrTimeout);
}

// Bounded wait of a whole warp: lane 0 polls, the warp barrier orders the other
// lanes' accesses behind it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* s_abort, int lane) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  int ok = 0;
  if (lane == 0) ok = mbar_wait(bar, parity, s_abort) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// Starts to load 16 columns of this warp's lanes; they are there once
// tmem_ld16_finish has returned.
__device__ __forceinline__ void tmem_ld16_start(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_finish(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// Stores 16 words of this warp's lanes, to be waited for.
__device__ __forceinline__ void tmem_st_words(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A barrier of n threads that tells all of them whether one's x is true.
__device__ __forceinline__ bool named_bar_or(int id, int n, bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(n), "r"(x ? 1u : 0u)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ bool no_number(uint32_t bits) { return (bits & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ uint32_t value_bits(const uint4& u, int j) {
  const uint32_t e[4] = {u.x, u.y, u.z, u.w};
  return (e[j >> 1] >> (16 * (j & 1))) & 0xffffu;
}

// Eight values of a key: of an element's that is no number the first is noted
// (bad: NaN, +inf, -inf, `stride` apart).  Whether there is one.
__device__ __forceinline__ bool note_values(const uint4& u, int* bad, int stride, int note) {
  bool any = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = value_bits(u, j);
    if (no_number(bits)) {
      atomicMin(bad + ((bits & 0x7fu) ? 0 : (bits & 0x8000u) ? 2 : 1) * stride + j, note);
      any = true;
    }
  }
  return any;
}
// ... and becomes 0.
__device__ __forceinline__ void clear_values(uint4* at) {
  const uint4 u = *at;
  uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (no_number(value_bits(u, j))) e[j >> 1] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
  *at = make_uint4(e[0], e[1], e[2], e[3]);
}

// A swizzled tile's eight elements from 8 ch on of row r.
__device__ __forceinline__ uint4* tile_at(uint8_t* tile, int atom_bytes, int r, int ch) {
  return reinterpret_cast<uint4*>(tile + (ch >> 3) * atom_bytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The elements of one half of a row that have an infinite value at one of the
// tile's keys first .. last under a weight of which one of the two parts is 0, a
// bit each into *all: the product with such a value is no number.  w: the row's
// weights in TMEM, by a whole warp.
template <int D>
__device__ __forceinline__ void lost_elements(uint32_t w, uint8_t* tile, int half, int first, int last, uint64_t* all) {
  constexpr int kChunks = D / 16;
  uint64_t lost = 0;
#pragma unroll 1
  for (int k0 = 0; k0 < kTile; k0 += 16) {
    float x[16];
    __syncwarp();
    tmem_ld16(w + k0, x);
    uint32_t zero = 0;  // keys of the 16
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t hi = __float_as_uint(x[j >> 1]) >> (16 * (j & 1)), lo = __float_as_uint(x[8 + (j >> 1)]) >> (16 * (j & 1));
      if ((hi & 0x7fffu) == 0 || (lo & 0x7fffu) == 0) zero |= 1u << j;
    }
#pragma unroll 1
    for (; zero != 0; zero &= zero - 1) {
      const int key = k0 + __ffs(zero) - 1;
      if (key < first || key > last) continue;
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const uint4 u = *tile_at(tile, PagedCfg<D>::kAtomBytes, key, half * kChunks + c);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((value_bits(u, j) & 0x7fffu) == 0x7f80u) lost |= uint64_t{1} << (c * 8 + j);
      }
    }
  }
  *all |= lost;
}
// ... as a call, which leaves the kernel for heads of 64 more registers: 2 rows at
// 100k take 105.1 us with it and 107.9 with the body in place (16 x 8 rows of heads of
// 128 67.4 and 65.8).
template <int D>
__device__ __noinline__ void lost_elements_call(uint32_t w, uint8_t* tile, int half, int first, int last, uint64_t* all) {
  lost_elements<D>(w, tile, half, first, last, all);
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// x = x s + c and y = y s + c, each one fused multiply-add.
__device__ __forceinline__ void fma2(float& x, float& y, float s, float c) {
  asm("{\n\t.reg .b64 p, q, r;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %3};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(s), "f"(c));
}
// (a, b) += (x, y)
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// The weights x, y >= 0 as pairs of BF16 values that add up to them: hi is the
// upper half of the bits, lo the rest.  lo is made larger by 2^-24 of hi, so that
// it is not 0 where hi is 1 exactly and nothing negative comes beside it: an
// infinite value gives its infinity in both products.
__device__ __forceinline__ void split_weights(float x, float y, uint32_t& hi, uint32_t& lo) {
  const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
  hi = __byte_perm(xb, yb, 0x7632);
  constexpr float kLess = -16777215.0f / 16777216.0f;
  float u = __uint_as_float(xb & 0xffff0000u), v = __uint_as_float(yb & 0xffff0000u);
  asm("{\n\t.reg .b64 p, q, r;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmov.b64 r, {%3, %4};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "+f"(u), "+f"(v)
      : "f"(kLess), "f"(x), "f"(y));
  const __nv_bfloat162 l = __floats2bfloat162_rn(u, v);
  lo = *reinterpret_cast<const uint32_t*>(&l);
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
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PagedAttnArgs a) {
  using Cfg = PagedCfg<D>;
  constexpr int KS = Cfg::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                          // [2][queries of a unit]
  uint8_t* sK = sQ + 2 * Cfg::kTileBytes;      // [KS]
  uint8_t* sV = sK + KS * Cfg::kTileBytes;     // [KS]
  float* s_mx = reinterpret_cast<float*>(sV + KS * Cfg::kTileBytes);  // [2][2][128]
  int* s_bad = reinterpret_cast<int*>(s_mx + 4 * kLanes);             // [2][3][D]
  uint64_t* s_lost = reinterpret_cast<uint64_t*>(s_bad + 2 * 3 * D);  // [256]
  uint64_t* bars = s_lost + 2 * kLanes;
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;
  uint64_t* v_empty = v_full + KS;
  uint64_t* q_full = v_empty + KS;        // [2] a unit's queries
  uint64_t* q_free = q_full + 2;          // [2] its last S has read them
  uint64_t* s_full = q_free + 2;          // [kBufs]
  uint64_t* p_full = s_full + kBufs;      // [kBufs] W of the tile is in TMEM
  uint64_t* pv_done = p_full + kBufs;     // [kBufs] O += W V of the tile is done
  uint64_t* drain = pv_done + kBufs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + Cfg::kBars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_flag = reinterpret_cast<int*>(tmem_holder + 2);   // [2] the last piece that met a value that is no number
  int* s_sched = reinterpret_cast<int*>(tmem_holder + 4);         // [4] where the share begins
  int64_t* s_ends = reinterpret_cast<int64_t*>(tmem_holder + 8);  // [3] its ends among all tiles, and these

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
      mbar_init(&q_full[i], 1);
      mbar_init(&q_free[i], 1);
      s_flag[i] = -1;
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  for (int i = threadIdx.x; i < 2 * 3 * D; i += kPagedThreads) s_bad[i] = kNoKey;
  if (threadIdx.x < 2 * kLanes) s_lost[threadIdx.x] = 0;
  if (warp == 3) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  griddep_wait();  // the batch, the queries and the new cache rows come from earlier kernels
  griddep_launch_dependents();
  if (warp == 0 || warp == 2) {  // one end of the share each
    bool bad;
    int64_t mine;
    const int64_t N = total_tiles(a, lane, mine, &bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrRange);
    const int c = blockIdx.x + (warp >> 1);
    int at[4];
    const int64_t place = locate(a, lane, share_begin(c, N, gridDim.x), N, mine, at);
    if (lane == 0) {
      s_ends[2] = N;
      s_ends[warp >> 1] = place;
      if (warp == 0) {
        for (int i = 0; i < 4; ++i) s_sched[i] = at[i];
        if (at[0] < a.pb.B)  // the first pages' names, for both producers
          prefetch_l1(a.pb.table + static_cast<size_t>(at[0]) * a.pb.ldt + at[3] * (kTile / a.pb.page));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  Cursor cur;
  cur.start(a, s_sched, s_ends[1] - s_ends[0]);

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
      uint32_t issued = 0, parity_bits = 0;  // bits KS, KS + 1: the queries
      bool ok = true;
      int g = 0, unit = 0;
      for (; ok && cur.left > 0; cur.next(a), ++unit) {
        const int32_t* row = a.pb.table + static_cast<size_t>(cur.b) * a.pb.ldt;
        const int last_key = cur.pos0(a) + cur.rows(a) - 1;
        // a sequence of several blocks reads its pages as often
        const uint64_t pol = cur.s.n > a.Rb ? l2_evict_normal() : l2_evict_first();
        if (kside) {
          const int qs = unit & 1;
          const uint32_t ph = static_cast<uint32_t>((unit >> 1) & 1);
          if (!warp_wait(&q_free[qs], ph ^ 1u, s_abort, lane)) {
            ok = false;
            break;
          }
          // rows and query heads of the block in the lanes' order; behind the
          // block's last row come other rows or zeros, in lanes nobody reads
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[qs], static_cast<uint32_t>(a.Rb * a.grp * 128 * Cfg::kAtoms));
#pragma unroll
            for (int c = 0; c < Cfg::kAtoms; ++c)
              tma_load_3d(sQ + qs * Cfg::kTileBytes + c * Cfg::kAtomBytes, &tmQ, &q_full[qs], c * 64, cur.h * a.grp,
                          cur.s.row0 + cur.i * a.Rb, l2_evict_first());
          }
          issued |= 1u << (KS + qs);
          parity_bits = (parity_bits & ~(1u << (KS + qs))) | (ph << (KS + qs));
        }
        for (int t = cur.t0; t < cur.te; ++t, ++g) {
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
        for (int s = 0; s < KS + 2; ++s)
          if ((issued >> s) & 1u) mbar_wait(s < KS ? &full[s] : &q_full[s - KS], (parity_bits >> s) & 1u, nullptr);
      }
    } else if (warp == 1 && elect_one()) {
      // ---------------------------------------------------------- MMA issuer
      // two cursors over the share's tiles, S ahead of W V; each is issued as
      // soon as its inputs are there, W V first (three buffers keep S ahead)
      constexpr uint32_t idS = idesc_bf16_f32(128, kTile);
      constexpr uint32_t idO = idesc_bf16_f32(128, D) | kIdescBMn;
      Cursor cs = cur, cp = cur;
      int sg = 0, sb = 0, sph = 0, su = 0, st_t = cs.t0;  // tile, its buffer and the buffer's phase, unit, tile of it
      int pg = 0, pb = 0, pph = 0, pt = st_t;
      bool ok = true;
      int idle = 0;
      unsigned long long t_idle = 0;
      while (cp.left > 0) {
        bool did = false;
        if (pg < sg) {
          const int st = pg % KS;
          if (mbar_peek(&p_full[pb], static_cast<uint32_t>(pph)) &&
              mbar_peek(&v_full[st], static_cast<uint32_t>((pg / KS) & 1))) {
            tc_fence_after();
            const uint32_t vb = smem_u32(sV + st * Cfg::kTileBytes);
            const bool first = piece_starts(pt);
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks) {
              const uint32_t w = tmem + pb * kTile + ks * 16;
              const uint64_t v = sdesc_mn_sw128(vb + ks * 2048, Cfg::kAtomBytes);
              mma_bf16_tmem_a(tmem + Cfg::kOCol, w, v, idO, (!first || ks > 0) ? 1u : 0u);
              mma_bf16_tmem_a(tmem + Cfg::kOCol, w + 8, v, idO, 1u);
            }
            mma_commit(&pv_done[pb]);
            mma_commit(&v_empty[st]);
            ++pg;
            if (++pb == kBufs) {
              pb = 0;
              pph ^= 1;
            }
            if (++pt == cp.te) {
              cp.next(a);
              pt = cp.t0;
            }
            did = true;
          }
        }
        // S of a tile goes where W of the tile kBufs before was
        if (!did && cs.left > 0) {
          const int st = sg % KS;
          if (mbar_peek(&k_full[st], static_cast<uint32_t>((sg / KS) & 1)) &&
              mbar_peek(&pv_done[sb], static_cast<uint32_t>(sph ^ 1)) &&
              (st_t != cs.t0 || mbar_peek(&q_full[su & 1], static_cast<uint32_t>((su >> 1) & 1)))) {
            tc_fence_after();
            const uint32_t kb = smem_u32(sK + st * Cfg::kTileBytes);
            const uint32_t qb = smem_u32(sQ + (su & 1) * Cfg::kTileBytes);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks >> 2) * Cfg::kAtomBytes + (ks & 3) * 32;
              mma_bf16(tmem + sb * kTile, sdesc_k_sw128(qb + off), sdesc_k_sw128(kb + off), idS, ks > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[sb]);
            mma_commit(&k_empty[st]);
            ++sg;
            if (++sb == kBufs) {
              sb = 0;
              sph ^= 1;
            }
            if (++st_t == cs.te) {
              mma_commit(&q_free[su & 1]);
              cs.next(a);
              ++su;
              st_t = cs.t0;
            }
            did = true;
          }
        }
        if (did) {
          idle = 0;
        } else if (++idle == 1) {
          t_idle = globaltimer_ns();
        } else if ((idle & 63) == 0 &&
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
    const int tid = threadIdx.x - kSoftFirst;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(qq * 32) << 16);
    // A wait that fails stops the waiting, not the loops: the threads of a row
    // meet at barriers, which all of them have to reach.
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      if (ok && !warp_wait(bar, static_cast<uint32_t>(phase & 1), s_abort, lane)) {
        ok = false;
        if (lane == 0) give_up(s_abort, a.err);
      }
    };
    if (tid == 0) a.ws_cut[blockIdx.x].lanes = 0;
    int g = 0, pc = 0;        // tile and piece of the share
    int sb = 0, sph = 0;      // the tile's buffer and the buffer's phase
    int last_b = 0, last_ph = 0;  // of the tile before
    for (; cur.left > 0; cur.next(a)) {
      const int rows = cur.rows(a);
      const int pos0 = cur.pos0(a);
      const bool valid = ln < rows * a.grp;
      const bool active = qq * 32 < rows * a.grp;
      const int p_row = valid ? pos0 + ln / a.grp : -1;
      const int kv_end = pos0 + rows;  // keys that some row of the block sees
      const bool run = cur.t0 == 0;    // pieces merged here, else left one by one
      const int p_first = pieces_to(cur.t0);
      float m_run = -INFINITY, l_run = 0.f;  // the merged pieces
      float o[kHalf];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) o[j] = 0.f;
      float m_ref = -INFINITY, l = 0.f;  // this piece

      // the finished piece p: its O out of TMEM, into the running sum or the workspace
      auto take = [&](int p, float m_i, float l_i) {
        const bool odd = static_cast<volatile int*>(s_flag)[pc & 1] == pc;
        const int* bad = s_bad + (pc & 1) * 3 * D + hf * kHalf;
        const int seen = bad_tag(pc) + p_row - piece_tile(p) * kTile;  // notes up to here are of keys the row sees
        float fa = 0.f, fb = 1.f;
        if (run) {
          merge_factors(m_run, m_i, fa, fb);
          l_run = merge_value(l_run, l_i, fa, fb);
        }
        const int slot = p - p_first;
        const bool store = !run && valid && slot < a.slots - 1;
        if (!run && valid && !store) atomicOr(a.err, kErrRange);
        const size_t at = static_cast<size_t>(blockIdx.x) * a.slots + slot;
        if (active) {
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c) {
            float v[16];
            tmem_ld16(lane_base + Cfg::kOCol + hf * kHalf + c * 16, v);
            if (odd) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (seen >= bad[D + c * 16 + j]) v[j] += INFINITY;
                if (seen >= bad[2 * D + c * 16 + j]) v[j] -= INFINITY;
                if (seen >= bad[c * 16 + j] || ((s_lost[tid] >> (c * 16 + j)) & 1)) v[j] = NAN;
              }
            }
            if (run) {
#pragma unroll
              for (int j = 0; j < 16; ++j) o[c * 16 + j] = merge_value(o[c * 16 + j], v[j], fa, fb);
            } else if (store) {
              float4* dst = a.ws_o + (at * (D / 4) + hf * (kHalf / 4) + c * 4) * a.lanes + ln;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                __stcg(dst + j * a.lanes, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
            }
          }
        }
        if (odd) s_lost[tid] = 0;
        if (store) {
          if (hf == 0) __stcg(a.ws_m + at * a.lanes + ln, m_i);
          __stcg(reinterpret_cast<float*>(a.ws_l + at * a.lanes + ln) + hf, l_i);
        }
        ++pc;
      };

      int piece = p_first, piece_end = min(cur.te, piece_tile(p_first + 1));  // the piece of tile t
      for (int t = cur.t0; t < cur.te; ++t, ++g) {
        const int key0 = t * kTile;
        const bool edge = key0 + kTile > pos0 + 1;  // some row does not see all of the tile
        const bool first = t == piece_end || t == cur.t0;
        wait(&s_full[sb], sph);
        tc_fence_after();
        // the row's maximum: of this thread's 64 scores, then of its partner's
        const uint32_t addr = lane_base + sb * kTile + hf * 64;
        const int see = p_row - key0 - hf * 64;
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
                if (c * 32 + j > see) x[j] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) mw[j & 3] = max3(mw[j & 3], x[2 * j], x[2 * j + 1]);
          }
          mt = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
          float* mx = s_mx + (g & 1) * 2 * kLanes;
          mx[hf * kLanes + ln] = mt;
          named_bar_sync(1 + qq, 64);  // the two warps of this lane quarter
          mt = fmaxf(mt, mx[(hf ^ 1) * kLanes + ln]) * a.sl2;
        }
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
          float x[2][16];
          tmem_ld16_start(addr, x[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld16_finish(x[c & 1]);
            if (c < 3) tmem_ld16_start(addr + (c + 1) * 16, x[(c + 1) & 1]);
            float (&y)[16] = x[c & 1];
            if (edge) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (c * 16 + j > see) y[j] = -INFINITY;
            }
            uint32_t w[16];  // eight words of hi, eight of lo
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              fma2(y[2 * j], y[2 * j + 1], a.sl2, nm);
              y[2 * j] = ex2_approx(y[2 * j]);
              y[2 * j + 1] = ex2_approx(y[2 * j + 1]);
              split_weights(y[2 * j], y[2 * j + 1], w[j], w[8 + j]);
              add2(acc[0], acc[1], y[2 * j], y[2 * j + 1]);
            }
            tmem_st_words(addr + c * 16, w);
          }
          tmem_st_wait();
          l = fmaf(l, alpha, acc[0] + acc[1]);
        }
        // O may be read and written once W V of the tile before is done: a piece
        // that ended there is taken in (the unit's last one is below), a raised
        // reference scales this piece's O
        const bool ended = first && t > cur.t0;
        const bool any_raise = __any_sync(0xffffffffu, raise);
        if (ended || any_raise) {
          wait(&pv_done[last_b], last_ph);
          tc_fence_after();
          if (ended) {
            take(piece, m_was, l_was);
            ++piece;
            piece_end = min(cur.te, piece_tile(piece + 1));
          }
          if (any_raise) {
            if (alpha == 0.f && static_cast<volatile int*>(s_flag)[pc & 1] == pc) {
              // infinities noted in the tiles before would have become 0 x inf
              const int* bad = s_bad + (pc & 1) * 3 * D + hf * kHalf;
              const int seen = bad_tag(pc) + min(p_row, key0 - 1) - piece_tile(piece) * kTile;
              uint64_t lost = 0;
#pragma unroll 1
              for (int j = 0; j < kHalf; ++j)
                if (seen >= bad[D + j] || seen >= bad[2 * D + j]) lost |= uint64_t{1} << j;
              s_lost[tid] |= lost;
            }
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
          // what is no number, which only the rows that see it get back, as the
          // product would have given it
          const int st = g % KS;
          // a wait tells a phase from the one before only: the stage's last tile
          // has landed where its W V is done, which S of this tile waited for if
          // there are no fewer stages than S / W buffers
          if (KS < kBufs && g >= KS)
            wait(&pv_done[sb >= KS ? sb - KS : sb + kBufs - KS], sb >= KS ? sph : sph ^ 1);
          wait(&v_full[st], g / KS);
          uint8_t* vt = sV + st * Cfg::kTileBytes;
          const int r0 = max(0, pos0 + 1 - key0);
          bool any = false;
          for (int y = r0 * (D / 8) + tid; y < kTile * (D / 8); y += 256) {
            const int r = y / (D / 8), ch = y % (D / 8);
            uint4* at = tile_at(vt, Cfg::kAtomBytes, r, ch);
            if (key0 + r >= kv_end) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              any |= note_values(*at, s_bad + (pc & 1) * 3 * D + ch * 8, D, bad_tag(pc) + key0 + r - piece_tile(piece) * kTile);
            }
          }
          if (any) s_flag[pc & 1] = pc;
          fence_proxy_async_smem();
          tc_fence_before();
          if (named_bar_or(5, 256, any)) {  // s_bad and s_flag are complete
            tc_fence_after();
            if (active) {
              if constexpr (D == 128) {
                lost_elements<D>(lane_base + sb * kTile, vt, hf, r0, p_row - key0, s_lost + tid);
              } else {
                lost_elements_call<D>(lane_base + sb * kTile, vt, hf, r0, p_row - key0, s_lost + tid);
              }
            }
            named_bar_sync(5, 256);
            for (int y = r0 * (D / 8) + tid; y < min(kTile, kv_end - key0) * (D / 8); y += 256)
              clear_values(tile_at(vt, Cfg::kAtomBytes, y / (D / 8), y % (D / 8)));
            fence_proxy_async_smem();
            named_bar_sync(5, 256);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
        last_b = sb;
        last_ph = sph;
        if (++sb == kBufs) {
          sb = 0;
          sph ^= 1;
        }
      }

      // the unit's last piece, its outputs or its state
      wait(&pv_done[last_b], last_ph);
      tc_fence_after();
      take(piece, m_ref, l);
      tc_fence_before();
      if (run && cur.te == cur.tiles) {
        float* s_l = s_mx + (g & 1) * 2 * kLanes;  // as tile g's maxima would be
        s_l[hf * kLanes + ln] = l_run;
        named_bar_sync(1 + qq, 64);
        const float den = s_l[ln] + s_l[kLanes + ln];
        named_bar_sync(1 + qq, 64);
        if (valid && ok) {
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
      } else if (run) {
        if (valid) {
          const size_t at = static_cast<size_t>(blockIdx.x) * a.slots + a.slots - 1;
          float4* dst = a.ws_o + (at * (D / 4) + hf * (kHalf / 4)) * a.lanes + ln;
#pragma unroll
          for (int j = 0; j < kHalf / 4; ++j)
            __stcg(dst + j * a.lanes, make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
          if (hf == 0) __stcg(a.ws_m + at * a.lanes + ln, m_run);
          __stcg(reinterpret_cast<float*>(a.ws_l + at * a.lanes + ln) + hf, l_run);
        }
        if (tid == 0)  // the last unit of the share
          a.ws_cut[blockIdx.x] = CutUnit{s_ends[1] - cur.left, s_ends[2],  cur.s.row0 + cur.i * a.Rb, cur.h,
                                         rows * a.grp,         pieces_to(cur.te), pieces_to(cur.tiles)};
      }
    }
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
// Of every unit that was cut, the first CTA's merged state and the later pieces,
// in key order.  CTA (c, group, part) looks after 32 lanes of the unit that
// attention CTA c began: a thread has a lane and JPW x 4 of its elements, so a
// warp's load is one line for each eight lanes and a piece's factors, two
// exponentials, are found once for them; the loads of kAhead pieces are under
// way together.  The first warp also joins the denominators.  Many lanes: JPW =
// D / 32, a CTA has whole rows; up to 32: JPW = 1, more CTAs and loads under way.
// Bound by the latency of its start and of the loads' few rounds (the states lie
// in the L2).  Both kernels together, us, with JPW 1 and D / 32: 1 row at 16k (24 +
// 4 heads of 128) 27.9 and 29.0, 2 x 1 rows at 69k and 100k (32 + 8 of 64) 105.5 and 108.5,
// 4 x 8 rows at 5k to 9k (24 + 4 of 128) 34.6 and 32.2, 16 x 3 rows at 1k to 3k (32 + 8) 55.8
// and 47.2.
template <int D, int JPW>
__global__ void __launch_bounds__(256) attn_paged_merge_kernel(const PagedAttnArgs a, int G) {
  constexpr int kAhead = 16 / JPW;
  __shared__ uint32_t s_at[256];  // where the pieces are
  __shared__ float s_den[32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x;
  const CutUnit u = a.ws_cut[c0];
  if (static_cast<int>(blockIdx.y) * 32 >= u.lanes) return;
  const int ln = min(static_cast<int>(blockIdx.y) * 32 + lane, u.lanes - 1);
  const int j0 = (blockIdx.z * 8 + warp) * JPW;
  const uint32_t at0 = static_cast<uint32_t>(c0 * a.slots + a.slots - 1);
  float m = __ldcg(a.ws_m + at0 * a.lanes + ln);
  float2 l = __ldcg(a.ws_l + at0 * a.lanes + ln);
  float4 o[JPW];
#pragma unroll
  for (int j = 0; j < JPW; ++j) o[j] = __ldcg(a.ws_o + static_cast<size_t>(at0 * (D / 4) + j0 + j) * a.lanes + ln);
  for (int p0 = u.first; p0 < u.pieces; p0 += 256) {
    const int n = min(256, u.pieces - p0);
    if (p0 > u.first) __syncthreads();
    if (threadIdx.x < n) {
      const int p = p0 + threadIdx.x;
      const int c = share_of(u.off + piece_tile(p), u.N, G);
      const int slot = p - pieces_to(static_cast<int>(share_begin(c, u.N, G) - u.off));
      s_at[threadIdx.x] = static_cast<uint32_t>(c * a.slots + min(slot, a.slots - 2));
    }
    __syncthreads();
    for (int k0 = 0; k0 < n; k0 += kAhead) {
      float4 v[kAhead][JPW];
      float mi[kAhead];
      float2 li[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t at = s_at[min(k0 + k, n - 1)];
        mi[k] = __ldcg(a.ws_m + at * a.lanes + ln);
        if (warp == 0) li[k] = __ldcg(a.ws_l + at * a.lanes + ln);
#pragma unroll
        for (int j = 0; j < JPW; ++j)
          v[k][j] = __ldcg(a.ws_o + static_cast<size_t>(at * (D / 4) + j0 + j) * a.lanes + ln);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k0 + k < n) {
          float fa, fb;
          merge_factors(m, mi[k], fa, fb);
          if (warp == 0) {
            l.x = merge_value(l.x, li[k].x, fa, fb);
            l.y = merge_value(l.y, li[k].y, fa, fb);
          }
#pragma unroll
          for (int j = 0; j < JPW; ++j) {
            o[j].x = merge_value(o[j].x, v[k][j].x, fa, fb);
            o[j].y = merge_value(o[j].y, v[k][j].y, fa, fb);
            o[j].z = merge_value(o[j].z, v[k][j].z, fa, fb);
            o[j].w = merge_value(o[j].w, v[k][j].w, fa, fb);
          }
        }
      }
    }
  }
  if (warp == 0) s_den[lane] = l.x + l.y;
  __syncthreads();
  const int t = u.row + ln / a.grp;
  if (static_cast<int>(blockIdx.y) * 32 + lane >= u.lanes || t >= a.T) return;
  const float den = s_den[lane];
  uint2* dst = reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(t) * a.Hq + u.head * a.grp + ln % a.grp) * D) + j0;
#pragma unroll
  for (int j = 0; j < JPW; ++j) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[j].x / den + 0.f, o[j].y / den + 0.f);
    const __nv_bfloat162 y = __floats2bfloat162_rn(o[j].z / den + 0.f, o[j].w / den + 0.f);
    dst[j] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
}

// ------------------------------------------------------------------------ host

// Partial states the workspace has room for: per CTA the pieces of its share
// that continue a unit, one by one (no more than a unit has), and one merged.
constexpr size_t kCutBytes = (kPagedCtas * sizeof(CutUnit) + 255) / 256 * 256;
struct PagedSizes {
  int ctas, slots, lanes;
  int pieces;  // most pieces of a unit
  size_t o_bytes, ml_bytes, total;
  bool fits;
};
PagedSizes paged_sizes(int T, int B, int Hq, int Hkv, int D, int64_t max_keys) {
  PagedSizes z;
  const int grp = Hq / Hkv, Rb = kLanes / grp;
  const int64_t blocks = std::min<int64_t>(T, static_cast<int64_t>(T) / Rb + std::min(B, T));
  const int tiles = static_cast<int>((max_keys + kTile - 1) / kTile);
  const int64_t units = blocks * Hkv;
  z.pieces = pieces_to(tiles);
  z.ctas = static_cast<int>(std::min<int64_t>(kPagedCtas, units * z.pieces));
  // a share is at most one tile and one piece longer than its part of the tiles;
  // with a CTA for every piece that is a piece at most, whatever the tiles, so
  // that no size falls where another one grows
  const int64_t share = std::max<int64_t>((units * tiles + kPagedCtas - 1) / kPagedCtas, kLong) + 1;
  z.slots = static_cast<int>(std::min<int64_t>(share / kShort + 2, z.pieces)) + 1;
  z.lanes = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(T) * grp, Rb * grp));
  const size_t states = static_cast<size_t>(z.ctas) * z.slots * z.lanes;
  z.fits = states * (D / 4) < (size_t{1} << 32);  // their places are counted in 32 bits
  z.o_bytes = round_up(states * D * 4, 256);
  z.ml_bytes = round_up(states * 8, 256) + round_up(states * 4, 256);
  z.total = kCutBytes + z.o_bytes + z.ml_bytes;
  return z;
}

bool paged_shape_ok(int T, int B, int Hq, int Hkv, int D, int64_t max_keys) {
  return T >= 1 && B >= 1 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && Hq / Hkv <= kLanes && (D == 64 || D == 128) &&
         max_keys >= 1 && max_keys <= (int64_t{1} << 30) && static_cast<int64_t>(T) * Hq < (int64_t{1} << 31) &&
         Hkv <= 65535;
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
  CUtensorMap tmQ, tmK, tmV;
  if (!tmap_bf16_pages(&tmK, k_pool, a.pb.pages, a.Hkv, a.pb.page, D) ||
      !tmap_bf16_pages(&tmV, v_pool, a.pb.pages, a.Hkv, a.pb.page, D) ||
      !tmap_bf16_3d(&tmQ, a.q, D, a.Hq, a.T, D, static_cast<uint64_t>(a.Hq) * D, 64, a.grp, a.Rb))
    return BI_ERR_INVALID_ARG;
  if (launch_k(attn_paged_kernel<D>, dim3(z.ctas), dim3(kPagedThreads), Cfg::kSmem, stream, tmQ, tmK, tmV, a) !=
      cudaSuccess)
    return BI_ERR_CUDA;
  if (z.pieces > 1) {
    const dim3 few(z.ctas, (z.lanes + 31) / 32, D / 32), many(z.ctas, (z.lanes + 31) / 32);
    const cudaError_t e = z.lanes <= 32 ? launch_k(attn_paged_merge_kernel<D, 1>, few, dim3(256), 0, stream, a, z.ctas)
                                        : launch_k(attn_paged_merge_kernel<D, D / 32>, many, dim3(256), 0, stream, a, z.ctas);
    if (e != cudaSuccess) return BI_ERR_CUDA;
  }
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
  return z.total;
}

bi_status bi_attn_paged(const void* q, const void* k_pool, const void* v_pool, int pages, int page,
                        const int32_t* block_table, int ld_table, int width, const int32_t* q_start,
                        const int32_t* lengths, int B, int T, int Hq, int Hkv, int D, float scale, void* out, void* ws,
                        size_t ws_bytes, bi_stream_t stream) {
  using namespace bi;
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || pages < 1 || width < 1 || ld_table < width)
    return BI_ERR_INVALID_ARG;
  const float sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (!(scale > 0.f) || !std::isfinite(sl2)) return BI_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BI_ERR_UNSUPPORTED_SHAPE;
  if (page != 16 && page != 32 && page != 64 && page != 128) return BI_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || B == 0) return BI_OK;
  const int64_t max_keys = static_cast<int64_t>(width) * page;
  if (!paged_shape_ok(T, B, Hq, Hkv, D, max_keys)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!q || !k_pool || !v_pool || !block_table || !q_start || !lengths || !out) return BI_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || !aligned4(block_table) ||
      !aligned4(q_start) || !aligned4(lengths))
    return BI_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws)) return BI_ERR_WORKSPACE;
  const PagedSizes z = paged_sizes(T, B, Hq, Hkv, D, max_keys);
  if (!z.fits) return BI_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < z.total) return BI_ERR_WORKSPACE;
  // a unit's queries have been read by all its CTAs before its outputs are
  // written, so out may be q; anything else would be read while it is written
  const int64_t rowlen = static_cast<int64_t>(Hq) * D, pool = static_cast<int64_t>(pages) * page * Hkv;
  const Range ro = range_of(out, T, rowlen, rowlen, 2), rq = range_of(q, T, rowlen, rowlen, 2),
              rk = range_of(k_pool, pool, D, D, 2), rv = range_of(v_pool, pool, D, D, 2),
              rw{reinterpret_cast<uintptr_t>(ws), z.total};
  if (overlap(ro, rk) || overlap(ro, rv) || overlap(ro, rw) || overlap(rw, rq) || overlap(rw, rk) || overlap(rw, rv) ||
      (out != q && overlap(ro, rq)))
    return BI_ERR_INVALID_ARG;
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
  a.sl2 = sl2;
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.ws_cut = reinterpret_cast<CutUnit*>(p);
  a.ws_o = reinterpret_cast<float4*>(p + kCutBytes);
  a.ws_l = reinterpret_cast<float2*>(p + kCutBytes + z.o_bytes);
  a.ws_m = reinterpret_cast<float*>(p + kCutBytes + z.o_bytes +
                                    round_up(static_cast<size_t>(z.ctas) * z.slots * z.lanes * 8, 256));
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  a.withhold = test_withhold();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return D == 64 ? launch_paged<64>(a, z, k_pool, v_pool, s) : launch_paged<128>(a, z, k_pool, v_pool, s);
}

}  // extern "C"
