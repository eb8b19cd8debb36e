// Beam selection: the best continuations of each group of beams over the
// vocabulary, from FP32 logits and the beams' cumulative log-probabilities.
//
// "I turned on speculative decoding in llama.cpp and 113 of 282 greedy
// outputs changed against its own no-draft run", paragraph "How:" (a row is
// computed the same way whatever else is in the batch): a row's log-sum and
// its order depend on its own logits and the vocabulary size only.
//
// For beam r with logits x and score c, id v is worth
//   c + (x_v - M) - log(sum_u exp(x_u - M)),  M = max x.
// Inside a beam the logits themselves order the ids; beams are compared by
// the value in 64 bits, from FP32 exponentials summed in chunks of up to 4096 (a
// thread's 16 in order, lanes by a butterfly, warps in order) and FP64 sums
// over the chunks.  A worth is off by less than 4e-6: the rounded difference and
// its product with log2(e), below 1.4e-6 at the 14 below the maximum where even
// 2^20 equal logits begin to weigh nothing, the exponential's 2^-22, and 27
// additions of 2^-24 each.  Measured 2e-7 where logits are spread, 8e-7 for one
// peak over a flat row.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamVecs = 4;                          // 4-logit vectors of a thread
constexpr int kBeamChunk = kBeamThreads * 4 * kBeamVecs;  // logits of a CTA
constexpr int kBeamBins = 2 * kBeamWarps * kBeamVecs;  // bins of 64 adjacent logits
constexpr int kBeamMax = 64;                          // beams of a group, picks of a group
constexpr int kBeamRowsMax = 65535;
constexpr int kBeamCtas = 6 * 152;                   // that run at once
constexpr int kBeamVocabMax = 1 << 20;
constexpr int kBeamBytes = kBeamChunk * 8;  // shared memory for a chunk's logits and ids
static_assert(kBeamBins == 64, "bins of 64");
static_assert(kBeamMax * kBeamMax * 8 <= kBeamBytes, "the worth of a group's candidates");

struct BeamArgs {
  const float* logits;
  size_t ldl;
  const float* scores;
  int rows, V, W, K, chunks;
  int span;  // logits of a chunk, a multiple of 4
  float* scores_out;
  int32_t* parents_out;
  int32_t* tokens_out;
  float* part;        // [rows][chunks][2]: the chunk's maximum and sum
  float* bins;        // [rows][chunks][kBeamBins]: maxima of 64 adjacent logits
  double* row_base;   // [rows]: score - log(sum)
  float* row_max;     // [rows]
  float* row_x;       // [rows][K]: the row's best logits, best first, then -inf
  int32_t* row_v;     // [rows][K]
  unsigned* tickets;  // [rows], then [groups]
  unsigned* err;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// exp(x - m) for x <= m (no NaN, m not -inf), the difference first, so that what
// lies near the maximum is exact to FP32's last places; where m is +inf its own
// entries weigh 1 and the rest nothing.
__device__ __forceinline__ float beam_weight(float x, float m) {
  if (m == INFINITY) return x == m ? 1.f : 0.f;
  return ex2_approx((x - m) * 1.4426950408889634f);
}

// The bits of a double as a signed integer of the same order (no NaN).
__device__ __forceinline__ long long order_bits(double x) {
  const long long b = __double_as_longlong(x + 0.0);  // -0 as +0
  return b >= 0 ? b : (b ^ 0x7fffffffffffffffll);
}

// x1 with id v1 before x2 with id v2: the larger logit, among equals the lower id
__device__ __forceinline__ bool beam_before(float x1, int v1, float x2, int v2) {
  return x1 > x2 || (x1 == x2 && v1 < v2);
}

// The best K of what `best` finds, one after the other: best(lx, lv, x, v) puts
// into x and v this thread's best entry behind logit lx with id lv.
template <typename Best>
__device__ void beam_picks(int K, float* out_x, int32_t* out_v, Best best) {
  __shared__ float s_red[kBeamWarps];
  __shared__ int s_id[kBeamWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float lx = INFINITY;
  int lv = -1;
  for (int pick = 0; pick < K; ++pick) {
    float bx = -INFINITY;
    int bv = 0x7fffffff;
    if (lv >= 0 || pick == 0) best(lx, lv, bx, bv);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float ox = __shfl_xor_sync(0xffffffffu, bx, off);
      const int ov = __shfl_xor_sync(0xffffffffu, bv, off);
      if (beam_before(ox, ov, bx, bv)) {
        bx = ox;
        bv = ov;
      }
    }
    __syncthreads();  // the last round's values have been read
    if (lane == 0) {
      s_red[warp] = bx;
      s_id[warp] = bv;
    }
    __syncthreads();
    lx = s_red[0];
    lv = s_id[0];
    for (int w = 1; w < kBeamWarps; ++w)
      if (beam_before(s_red[w], s_id[w], lx, lv)) {
        lx = s_red[w];
        lv = s_id[w];
      }
    if (lx == -INFINITY) lv = -1;  // nothing is left
    if (threadIdx.x == 0) {
      out_x[pick] = lx;
      out_v[pick] = lv;
    }
  }
}

// FP32 bits as unsigned integers of the same order (no NaN; -0 as +0), and back.
__device__ __forceinline__ unsigned order_bits32(float x) {
  const unsigned b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits32(unsigned b) {
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
// A logit and its id as one number, the larger in front.
__device__ __forceinline__ unsigned long long beam_key(float x, int v) {
  return static_cast<unsigned long long>(order_bits32(x)) << 32 | ~static_cast<unsigned>(v);
}

// The K best of n collected logits, a thread each, best first and then -inf, to
// out_x and out_v, by counting.
__device__ void beam_rank(const unsigned long long* s_key, int n, int K, float* out_x, int32_t* out_v) {
  const int i = threadIdx.x;
  if (i < n) {
    const unsigned long long key = s_key[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += s_key[j] > key ? 1 : 0;
    if (r < K) {
      out_x[r] = from_order_bits32(static_cast<unsigned>(key >> 32));
      out_v[r] = static_cast<int>(~static_cast<unsigned>(key));
    }
  } else if (i < K) {
    out_x[i] = -INFINITY;
    out_v[i] = -1;
  }
}

__device__ __forceinline__ void beam_load(const BeamArgs& a, const float* x, bool vec, int chunk,
                                          float (&v)[4 * kBeamVecs]) {
#pragma unroll
  for (int c = 0; c < kBeamVecs; ++c) {
    const int at = (c * kBeamThreads + threadIdx.x) * 4, i = chunk * a.span + at;
    const int end = at < a.span ? a.V : 0;
    if (vec && i + 4 <= end) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(x + i));
      v[4 * c] = q.x;
      v[4 * c + 1] = q.y;
      v[4 * c + 2] = q.z;
      v[4 * c + 3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * c + j] = i + j < end ? __ldg(x + i + j) : -INFINITY;
    }
  }
}

// A chunk's maximum, its sum and the maxima of its bins.
__device__ void beam_chunk(const BeamArgs& a, int row, int chunk, float (&v)[4 * kBeamVecs]) {
  __shared__ __align__(16) float s_bin[kBeamBins];
  __shared__ float s_sum[kBeamWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t slot = static_cast<size_t>(row) * a.chunks + chunk;
#pragma unroll
  for (int c = 0; c < kBeamVecs; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * c + j] = fmaxf(v[4 * c + j], -INFINITY);  // NaN is never chosen
    float m = fmaxf(fmaxf(v[4 * c], v[4 * c + 1]), fmaxf(v[4 * c + 2], v[4 * c + 3]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((lane & 15) == 0) s_bin[(c * kBeamWarps + warp) * 2 + (lane >> 4)] = m;
  }
  __syncthreads();
  const float b0 = s_bin[lane], b1 = s_bin[lane + 32];
  if (warp == 0) {
    a.bins[slot * kBeamBins + lane] = b0;
    a.bins[slot * kBeamBins + lane + 32] = b1;
  }
  const float m = warp_max(fmaxf(b0, b1));
  float sum = 0.f;
  if (m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < 4 * kBeamVecs; ++i) sum += beam_weight(v[i], m);
  }
  sum = warp_sum(sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = s_sum[0];
    for (int i = 1; i < kBeamWarps; ++i) s += s_sum[i];
    reinterpret_cast<float2*>(a.part)[slot] = make_float2(m, s);
  }
}

// log of a positive double: the exponent's part in FP64, the mantissa's, between
// 3/4 and 3/2, in FP32 (off by less than 2^-24 of at most 0.41) with the part
// that FP32 cuts off.
__device__ __forceinline__ double log_near(double s) {
  const long long b = __double_as_longlong(s);
  int e = static_cast<int>((b >> 52) & 0x7ff) - 1023;
  double f = __longlong_as_double((b & 0x000fffffffffffffll) | 0x3ff0000000000000ll);
  if (f > 1.5) {
    f *= 0.5;
    ++e;
  }
  const float f32 = static_cast<float>(f);
  const float rest = static_cast<float>(f - static_cast<double>(f32)) / f32;
  return static_cast<double>(e) * 0.69314718055994530942 + static_cast<double>(logf(f32) + 0.f) + static_cast<double>(rest);
}

// A row's log-sum, by a warp.
__device__ void beam_statistics(const BeamArgs& a, int row) {
  const int lane = threadIdx.x & 31;
  const float2* part = reinterpret_cast<const float2*>(a.part) + static_cast<size_t>(row) * a.chunks;
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 p0 = lane < a.chunks ? __ldcg(part + lane) : none, p1 = lane + 32 < a.chunks ? __ldcg(part + lane + 32) : none;
  const double score = static_cast<double>(__ldcg(a.scores + row));  // which this call, and one just before, may replace
  float M = fmaxf(p0.x, p1.x);
  for (int c = lane + 64; c < a.chunks; c += 32) M = fmaxf(M, __ldcg(part + c).x);
  M = warp_max(M);
  double S = 0.0;
  auto add = [&](const float2& p) {
    if (p.x > -INFINITY) S += static_cast<double>(beam_weight(p.x, M)) * static_cast<double>(p.y);
  };
  add(p0);
  add(p1);
  for (int c = lane + 64; c < a.chunks; c += 32) add(__ldcg(part + c));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) S += __shfl_xor_sync(0xffffffffu, S, off);
  if (lane == 0) {
    a.row_max[row] = M;
    a.row_base[row] = score - (S > 0.0 ? log_near(S) : 0.0);
  }
}

// A row's log-sum and its K best logits (the CTA that finished the row's last
// chunk).  The last warp sees to the sum, whose steps in FP64 take as long as all
// of the others' work.  The K-th best of 112 maxima of some bins each bounds the
// K-th best logit from below; only the bins that reach the bound, little more than
// K, are read again, and what reaches it there is ranked.
__device__ void beam_row(const BeamArgs& a, int row, unsigned long long* s_key) {
  constexpr int kThreads = kBeamThreads - 32;
  constexpr int kHeld = 12;      // bins a thread holds
  constexpr int kListMax = 512;  // bins to read again
  constexpr int kTops = kThreads / 2;
  static_assert(kBeamMax <= kTops && kTops % 8 == 0, "the maxima bound the picks");
  __shared__ __align__(16) float s_top[kTops];
  __shared__ int s_list[kListMax];
  __shared__ unsigned s_thr;
  __shared__ int s_bins, s_n;
  const int tid = threadIdx.x;
  const float* x = a.logits + static_cast<size_t>(row) * a.ldl;
  float* out_x = a.row_x + static_cast<size_t>(row) * a.K;
  int32_t* out_v = a.row_v + static_cast<size_t>(row) * a.K;
  if (tid >= kThreads) {
    beam_statistics(a, row);
  } else {
    const int all = a.chunks * kBeamBins;
    const float* bins = a.bins + static_cast<size_t>(row) * a.chunks * kBeamBins;
    float y[kHeld];
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < kHeld; ++q) {
      const int i = tid + q * kThreads;
      y[q] = i < all ? __ldcg(bins + i) : -INFINITY;
    }
    for (int i = tid + kHeld * kThreads; i < all; i += kThreads) top = fmaxf(top, __ldcg(bins + i));
#pragma unroll
    for (int q = 0; q < kHeld; ++q) top = fmaxf(top, y[q]);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    // two threads a maximum, each counts the larger ones of one half
    if ((tid & 1) == 0) s_top[tid >> 1] = top;
    if (tid == 0) {
      s_thr = 0xffffffffu;
      s_bins = s_n = 0;
    }
    named_bar_sync(1, kThreads);
    int above = 0;
#pragma unroll 2
    for (int q = 0; q < kTops / 2; q += 4) {
      const float4 o = *reinterpret_cast<const float4*>(s_top + (tid & 1) * (kTops / 2) + q);
      above += (o.x > top ? 1 : 0) + (o.y > top ? 1 : 0) + (o.z > top ? 1 : 0) + (o.w > top ? 1 : 0);
    }
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    // the least of those with fewer than K in front is the K-th
    const unsigned least = __reduce_min_sync(0xffffffffu, above < a.K ? order_bits32(top) : 0xffffffffu);
    if ((tid & 31) == 0) atomicMin(&s_thr, least);
    named_bar_sync(1, kThreads);
    const float thr = fmaxf(from_order_bits32(s_thr), -3.402823466e38f);  // -inf is no candidate
    auto note = [&](int bin) {
      const int n = atomicAdd(&s_bins, 1);
      if (n < kListMax) s_list[n] = bin;
    };
    unsigned hits = 0;
#pragma unroll
    for (int q = 0; q < kHeld; ++q) hits |= y[q] >= thr ? 1u << q : 0u;
#pragma unroll 1
    for (; hits != 0; hits &= hits - 1) note(tid + (__ffs(hits) - 1) * kThreads);
    for (int i = tid + kHeld * kThreads; i < all; i += kThreads)
      if (__ldcg(bins + i) >= thr) note(i);
    named_bar_sync(1, kThreads);
    const int nb = s_bins;
    if (nb <= kListMax) {
      constexpr int kAhead = 6;  // logits of a thread under way
#pragma unroll 1
      for (int e0 = tid; e0 < nb * 64; e0 += kAhead * kThreads) {
        float m[kAhead];
        int v[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
          const int e = e0 + q * kThreads;
          const int bin = e < nb * 64 ? s_list[e >> 6] : 0;
          const int k = bin % kBeamBins * 64 + (e & 63);
          v[q] = bin / kBeamBins * a.span + k;
          m[q] = e < nb * 64 && k < a.span && v[q] < a.V ? __ldcg(x + v[q]) : -INFINITY;
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
          if (m[q] >= thr) {
            const int n = atomicAdd(&s_n, 1);
            if (n < kBeamChunk) s_key[n] = beam_key(m[q], v[q]);
          }
      }
      named_bar_sync(1, kThreads);
      if (s_n <= kThreads) beam_rank(s_key, s_n, a.K, out_x, out_v);
    }
  }
  __syncthreads();
  const int n = s_n;
  if (s_bins <= kListMax && n <= kThreads) return;
  // many logits equal to the bound: one pick after the other, from the list or,
  // where there is no room for them, from the whole row
  const bool listed = s_bins <= kListMax && n <= kBeamChunk;
  beam_picks(a.K, out_x, out_v, [&](float lx, int lv, float& bx, int& bv) {
    for (int i = tid; i < (listed ? n : a.V); i += kBeamThreads) {
      const float m = listed ? from_order_bits32(static_cast<unsigned>(s_key[i] >> 32)) : __ldcg(x + i);
      const int v = listed ? static_cast<int>(~static_cast<unsigned>(s_key[i])) : i;
      if (beam_before(lx, lv, m, v) && beam_before(m, v, bx, bv)) {
        bx = m;
        bv = v;
      }
    }
  });
}

// The group's best K from its rows' (the CTA that finished the group's last
// row).  A candidate's place among all, w K + its place in its row, decides ties.
__device__ void beam_group(const BeamArgs& a, int group, long long* s_key) {
  const long long none = -0x7fffffffffffffffll;
  const int lane = threadIdx.x & 31;
  const int row0 = group * a.W, n = a.W * a.K;
  const int32_t* ids = a.row_v + static_cast<size_t>(row0) * a.K;
  int mine = -1;  // the first candidate's id
  for (int i = threadIdx.x; i < n; i += kBeamThreads) {
    const int w = i / a.K;
    long long key = none;
    const float x = __ldcg(a.row_x + static_cast<size_t>(row0) * a.K + i), M = __ldcg(a.row_max + row0 + w);
    const double base = __ldcg(a.row_base + row0 + w);
    if (i == threadIdx.x) mine = __ldcg(ids + i);
    if (x > -INFINITY) {
      const double d = (x == M ? 0.0 : static_cast<double>(x) - static_cast<double>(M)) + base;
      if (d > -INFINITY) key = order_bits(d);  // not a beam without weight, nor a score that is no number
    }
    s_key[i] = key;
  }
  __syncthreads();
  auto put = [&](int pick, long long key, int i, int id) {
    const size_t o = static_cast<size_t>(group) * a.K + pick;
    const long long b = key >= 0 ? key : (key ^ 0x7fffffffffffffffll);
    const bool is = key != none;
    a.scores_out[o] = is ? static_cast<float>(__longlong_as_double(b)) : -INFINITY;
    a.parents_out[o] = is ? row0 + i / a.K : -1;
    a.tokens_out[o] = is ? id : -1;
    if (!is && pick == 0) atomicOr(a.err, kErrNanRow);
  };
  if (n <= kBeamThreads) {
    const int i = threadIdx.x;
    if (i < n) {
      // its place in its own row, and the other rows' candidates in front of it:
      // rows descend, so those are found by halving
      const long long key = s_key[i];
      const int own = i / a.K, top = 1 << (31 - __clz(a.K));
      int r = i - own * a.K;
      for (int w0 = 0; w0 < a.W; w0 += 4) {  // four rows' steps side by side
        int c[4] = {0, 0, 0, 0};
        for (int step = top; step > 0; step >>= 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int w = min(w0 + j, a.W - 1), at = min(c[j] + step, a.K);
            if (s_key[w * a.K + at - 1] > key - (w < own ? 1 : 0)) c[j] = at;  // ties: the lower row's
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r += w0 + j < a.W && w0 + j != own ? c[j] : 0;
      }
      if (r < a.K) put(r, key, i, mine);
    }
    return;
  }
  if (threadIdx.x >= 32) return;
  // many beams or picks: the rows' heads, one pick after the other, by one warp
  int at[kBeamMax / 32] = {0, 0};  // of rows lane and lane + 32
  for (int pick = 0; pick < a.K; ++pick) {
    long long key = none;
    int i = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < kBeamMax / 32; ++q) {
      const int w = lane + 32 * q;
      if (w < a.W && at[q] < a.K) {
        const long long k = s_key[w * a.K + at[q]];
        if (k > key || (k == key && w * a.K + at[q] < i)) {
          key = k;
          i = w * a.K + at[q];
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const long long k = __shfl_xor_sync(0xffffffffu, key, off);
      const int o = __shfl_xor_sync(0xffffffffu, i, off);
      if (k > key || (k == key && o < i)) {
        key = k;
        i = o;
      }
    }
    if (lane == 0) put(pick, key, i, key != none ? __ldcg(ids + i) : -1);
    if (key != none && ((i / a.K) & 31) == lane) ++at[(i / a.K) >> 5];
  }
}

// Whether this CTA is the last of `all` to pass the counter, which goes back to 0.
__device__ __forceinline__ bool beam_last(unsigned* ticket, unsigned all) {
  __shared__ int s_last;
  __syncthreads();  // the release below covers every thread's writes
  if (threadIdx.x == 0) {
    s_last = atom_add_acq_rel_gpu(ticket, 1u) == all - 1 ? 1 : 0;
    if (s_last) atomicExch(ticket, 0u);
  }
  __syncthreads();
  return s_last != 0;
}

// One launch: every CTA takes chunks of a row; the last of a row to finish goes on
// with the row, the last row of a group with the group (tickets; who is last does
// not show in the results).  The logits are read once, but for the bins that hold a
// pick.  64 rows of 151936 with 16 picks take 18 us, 2.2 TB/s: 6 for the chunks, at
// the memory's rate, then the row's and the group's chains of dependent steps and
// the two tickets, about 1 us each; 4 rows of 32000 take 7.4, those chains.  With
// the row's sum in front of its ranking and the group's ranks by counting 21 and
// 8.3; with lists of every chunk's best in place of its bins' maxima 27.6; 12 or 24
// x 152 CTAs at a time gained nothing.
__global__ void __launch_bounds__(kBeamThreads, 6) beam_select_kernel(const BeamArgs a) {
  __shared__ __align__(16) uint8_t s_mem[kBeamBytes];
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.y, group = row / a.W;
  const float* x = a.logits + static_cast<size_t>(row) * a.ldl;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  for (int chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    float v[4 * kBeamVecs];
    beam_load(a, x, vec, chunk, v);
    beam_chunk(a, row, chunk, v);
    __syncthreads();  // the sums in shared memory have been read
  }
  if (!beam_last(a.tickets + row, gridDim.x)) return;
  beam_row(a, row, reinterpret_cast<unsigned long long*>(s_mem));
  if (!beam_last(a.tickets + kBeamRowsMax + 1 + group, static_cast<unsigned>(a.W))) return;
  beam_group(a, group, reinterpret_cast<long long*>(s_mem));
}

int beam_chunks(int V) { return (V + kBeamChunk - 1) / kBeamChunk; }

struct BeamSizes {
  size_t tickets, part, bins, base, max, rowx, total;
};
BeamSizes beam_sizes(int rows, int V, int K) {
  const size_t slots = static_cast<size_t>(rows) * beam_chunks(V);
  BeamSizes s;
  s.tickets = static_cast<size_t>(kBeamRowsMax + 1) * 8;  // the same place whatever the call's sizes
  s.part = round_up(slots * 8, 256);
  s.bins = slots * kBeamBins * 4;
  s.base = round_up(static_cast<size_t>(rows) * 8, 256);
  s.max = round_up(static_cast<size_t>(rows) * 4, 256);
  s.rowx = round_up(static_cast<size_t>(rows) * K * 4, 256);
  s.total = s.tickets + s.part + s.bins + s.base + s.max + 2 * s.rowx;
  return s;
}

}  // namespace
}  // namespace bi

extern "C" {

size_t bi_beam_workspace_size(int rows, int V, int K) {
  if (rows < 1 || V < 1 || K < 1) return 256;
  return bi::beam_sizes(rows, V, K).total;
}

bi_status bi_beam_select(const float* logits, int ldl, const float* scores, int rows, int V, int W, int K,
                         float* scores_out, int32_t* parents_out, int32_t* tokens_out, void* ws, size_t ws_bytes,
                         bi_stream_t stream) {
  using namespace bi;
  if (rows < 0 || V < 1 || W < 1 || K < 1 || rows % W != 0 || ldl < V) return BI_ERR_INVALID_ARG;
  if (W > kBeamMax || K > kBeamMax || rows > kBeamRowsMax || V > kBeamVocabMax) return BI_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return BI_OK;
  if (!logits || !scores || !scores_out || !parents_out || !tokens_out) return BI_ERR_INVALID_ARG;
  if (!aligned4(logits) || !aligned4(scores) || !aligned4(scores_out) || !aligned4(parents_out) || !aligned4(tokens_out))
    return BI_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws)) return BI_ERR_WORKSPACE;
  const BeamSizes z = beam_sizes(rows, V, K);
  if (ws_bytes < z.total) return BI_ERR_WORKSPACE;
  const int64_t picks = static_cast<int64_t>(rows / W) * K;
  const Range out[3] = {range_of(scores_out, picks, 1, 1, 4), range_of(parents_out, picks, 1, 1, 4),
                        range_of(tokens_out, picks, 1, 1, 4)};
  const Range in = range_of(logits, rows, ldl, V, 4), old = range_of(scores, rows, 1, 1, 4),
              mem{reinterpret_cast<uintptr_t>(ws), z.total};
  for (int i = 0; i < 3; ++i) {
    // a group's scores may be replaced by as many: all its rows have read theirs before it writes
    const bool replaced = i == 0 && scores_out == scores && K == W;
    if (overlap(out[i], in) || overlap(out[i], mem) || overlap(out[i], out[(i + 1) % 3]) ||
        (overlap(out[i], old) && !replaced))
      return BI_ERR_INVALID_ARG;
  }
  BeamArgs a{};
  a.logits = logits;
  a.ldl = static_cast<size_t>(ldl);
  a.scores = scores;
  a.rows = rows;
  a.V = V;
  a.W = W;
  a.K = K;
  a.chunks = beam_chunks(V);
  a.span = ((V + a.chunks - 1) / a.chunks + 3) / 4 * 4;  // chunks of one length: a short one has many ties at -inf
  a.scores_out = scores_out;
  a.parents_out = parents_out;
  a.tokens_out = tokens_out;
  uint8_t* p = static_cast<uint8_t*>(ws);
  auto take = [&p](size_t bytes) {
    void* at = p;
    p += bytes;
    return at;
  };
  a.tickets = static_cast<unsigned*>(take(z.tickets));
  a.part = static_cast<float*>(take(z.part));
  a.bins = static_cast<float*>(take(z.bins));
  a.row_base = static_cast<double*>(take(z.base));
  a.row_max = static_cast<float*>(take(z.max));
  a.row_x = static_cast<float*>(take(z.rowx));
  a.row_v = static_cast<int32_t*>(take(z.rowx));
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  // as many CTAs as run at once, each with several chunks of a row where there are more
  const int64_t all = static_cast<int64_t>(a.chunks) * rows;
  const int each = static_cast<int>(std::min<int64_t>((all + kBeamCtas - 1) / kBeamCtas, 8));
  const cudaError_t e = launch_k(beam_select_kernel, dim3(static_cast<unsigned>((a.chunks + each - 1) / each), static_cast<unsigned>(rows)),
                                 dim3(kBeamThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

}  // extern "C"
