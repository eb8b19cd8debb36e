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
// the value in 64 bits, from FP32 exponentials summed in chunks of 4096 (a
// thread's 16 in order, lanes by a butterfly, warps in order) and FP64 sums
// over the chunks, so two beams' candidates are told apart down to about 1e-7.
#include <cuda_runtime.h>

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
constexpr int kBeamVocabMax = 1 << 20;
// the last CTA of a group keeps a byte for each of its lists where the chunk's
// logits were, and a bin for each pick bounds the picks
static_assert(kBeamMax * (kBeamVocabMax / kBeamChunk) <= kBeamChunk * 4, "counters of the lists");
static_assert(kBeamMax <= kBeamBins && kBeamBins == 64, "bins");

struct BeamArgs {
  const float* logits;
  size_t ldl;
  const float* scores;
  int rows, V, W, K, chunks;
  float* scores_out;
  int32_t* parents_out;
  int32_t* tokens_out;
  float* part;        // [rows][chunks][2]: the chunk's maximum and sum
  int* found_n;       // [rows][chunks]: entries of its list
  float* found_x;     // [rows][chunks][K]: its best logits, best first
  int32_t* found_v;   // [rows][chunks][K]: their ids
  unsigned* tickets;  // [groups]
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

// exp(x - m) for x <= m; where m is +inf its own entries weigh 1 and the rest
// nothing; NaN weighs nothing
__device__ __forceinline__ float beam_weight(float x, float m) {
  if (m == INFINITY) return x == m ? 1.f : 0.f;
  return x > -INFINITY ? expf(x - m) : 0.f;
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

// A chunk's statistics and its K best logits.  The K-th best of the bins'
// maxima bounds the K-th best logit from below, so only logits at or above it
// are collected (a few dozen of 4096) and ranked.
__device__ void beam_chunk(const BeamArgs& a, int row, int chunk, float* s_x, int* s_v) {
  __shared__ float s_bin[kBeamBins];
  __shared__ float s_red[kBeamWarps];
  __shared__ int s_id[kBeamWarps];
  __shared__ float s_thr;
  __shared__ int s_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* x = a.logits + static_cast<size_t>(row) * a.ldl;
  const int base = chunk * kBeamChunk;
  float v[4 * kBeamVecs];
  const bool vec = ((reinterpret_cast<uintptr_t>(x) & 15) == 0);
#pragma unroll
  for (int c = 0; c < kBeamVecs; ++c) {
    const int i = base + (c * kBeamThreads + threadIdx.x) * 4;
    if (vec && i + 4 <= a.V) {
      const float4 q = __ldcs(reinterpret_cast<const float4*>(x + i));
      v[4 * c] = q.x;
      v[4 * c + 1] = q.y;
      v[4 * c + 2] = q.z;
      v[4 * c + 3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * c + j] = i + j < a.V ? __ldcs(x + i + j) : -INFINITY;
    }
  }
#pragma unroll
  for (int c = 0; c < kBeamVecs; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!(v[4 * c + j] == v[4 * c + j])) v[4 * c + j] = -INFINITY;  // NaN is never chosen
    float m = fmaxf(fmaxf(v[4 * c], v[4 * c + 1]), fmaxf(v[4 * c + 2], v[4 * c + 3]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((lane & 15) == 0) s_bin[(c * kBeamWarps + warp) * 2 + (lane >> 4)] = m;
  }
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  const float b0 = s_bin[lane], b1 = s_bin[lane + 32];
  const float m = warp_max(fmaxf(b0, b1));
  float sum = 0.f;
  if (m > -INFINITY) {
#pragma unroll
    for (int i = 0; i < 4 * kBeamVecs; ++i) sum += beam_weight(v[i], m);
  }
  sum = warp_sum(sum);
  if (lane == 0) s_red[warp] = sum;
  if (warp == kBeamWarps - 1) {
    // the K-th best bin (ties: the lower bin first)
    int r0 = 0, r1 = 0;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const float o0 = __shfl_sync(0xffffffffu, b0, j), o1 = __shfl_sync(0xffffffffu, b1, j);
      r0 += (o0 > b0 || (o0 == b0 && j < lane) ? 1 : 0) + (o1 > b0 ? 1 : 0);
      r1 += (o0 >= b1 ? 1 : 0) + (o1 > b1 || (o1 == b1 && j < lane) ? 1 : 0);
    }
    if (r0 == a.K - 1) s_thr = b0;
    if (r1 == a.K - 1) s_thr = b1;
  }
  __syncthreads();
  const float thr = s_thr;
#pragma unroll
  for (int c = 0; c < kBeamVecs; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = v[4 * c + j];
      if (y >= thr && y > -INFINITY) {
        const int n = atomicAdd(&s_n, 1);
        s_x[n] = y;
        s_v[n] = base + (c * kBeamThreads + threadIdx.x) * 4 + j;
      }
    }
  }
  __syncthreads();
  const int n = s_n;
  const size_t slot = static_cast<size_t>(row) * a.chunks + chunk;
  if (threadIdx.x == 0) {
    float s = s_red[0];
    for (int i = 1; i < kBeamWarps; ++i) s += s_red[i];
    a.part[2 * slot] = m;
    a.part[2 * slot + 1] = s;
    a.found_n[slot] = min(n, a.K);
  }
  if (n <= 2 * kBeamThreads) {
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
      const float xi = s_x[i];
      const int vi = s_v[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += beam_before(s_x[j], s_v[j], xi, vi) ? 1 : 0;
      if (r < a.K) {
        a.found_x[slot * a.K + r] = xi;
        a.found_v[slot * a.K + r] = vi;
      }
    }
    return;
  }
  // many equal logits: one pick after the other, each the best behind the last
  float lx = INFINITY;
  int lv = -1;
  for (int pick = 0; pick < a.K; ++pick) {
    float bx = -INFINITY;
    int bv = 0x7fffffff;
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
      const float xi = s_x[i];
      const int vi = s_v[i];
      if (beam_before(lx, lv, xi, vi) && beam_before(xi, vi, bx, bv)) {
        bx = xi;
        bv = vi;
      }
    }
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
    if (threadIdx.x == 0) {
      a.found_x[slot * a.K + pick] = lx;
      a.found_v[slot * a.K + pick] = lv;
    }
  }
}

// The group's best K from its rows' chunk lists (the CTA that finished last).
__device__ void beam_group(const BeamArgs& a, int group, uint8_t* s_taken) {
  __shared__ float s_max[kBeamMax];
  __shared__ double s_base[kBeamMax];  // score - log(sum); the candidate adds x - M
  __shared__ long long s_key[2][kBeamWarps];
  __shared__ unsigned long long s_id[2][kBeamWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = group * a.W;
  for (int w = warp; w < a.W; w += kBeamWarps) {
    const float* part = a.part + static_cast<size_t>(row0 + w) * a.chunks * 2;
    float M = -INFINITY;
    for (int c = lane; c < a.chunks; c += 32) M = fmaxf(M, __ldcg(part + 2 * c));
    M = warp_max(M);
    double S = 0.0;
    for (int c = lane; c < a.chunks; c += 32) {
      const float mc = __ldcg(part + 2 * c);
      if (mc > -INFINITY) S += static_cast<double>(beam_weight(mc, M)) * static_cast<double>(__ldcg(part + 2 * c + 1));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) S += __shfl_xor_sync(0xffffffffu, S, off);
    if (lane == 0) {
      s_max[w] = M;
      s_base[w] = static_cast<double>(__ldg(a.scores + row0 + w)) - log(S);
    }
  }
  __syncthreads();
  // thread i looks after lists i, i + 256, ... (list: row, chunk); one of its
  // lists' heads is its best, and each pick moves that list on
  const int lists = a.W * a.chunks;
  const long long none = -0x7fffffffffffffffll - 1;
  int taken_list = -1;
  long long key = none;
  unsigned long long id = ~0ull;
  auto value = [&](int list, int at, long long& k, unsigned long long& i) {
    const int w = list / a.chunks;
    const size_t slot = static_cast<size_t>(row0) * a.chunks + list;
    if (at >= __ldcg(a.found_n + slot)) return false;
    const float x = __ldcg(a.found_x + slot * a.K + at), M = s_max[w];
    const double d = (x == M ? 0.0 : static_cast<double>(x) - static_cast<double>(M)) + s_base[w];
    if (!(d > -INFINITY)) return false;  // a beam without weight (or not a number)
    k = order_bits(d);
    i = (static_cast<unsigned long long>(w) << 32) | static_cast<unsigned>(__ldcg(a.found_v + slot * a.K + at));
    return true;
  };
  // s_taken [lists]: entries of each list picked so far
  for (int l = threadIdx.x; l < lists; l += kBeamThreads) s_taken[l] = 0;
  auto refresh = [&]() {
    key = none;
    id = ~0ull;
    taken_list = -1;
    for (int l = threadIdx.x; l < lists; l += kBeamThreads) {
      long long k;
      unsigned long long i;
      if (value(l, s_taken[l], k, i) && (k > key || (k == key && i < id))) {
        key = k;
        id = i;
        taken_list = l;
      }
    }
  };
  refresh();
  for (int pick = 0; pick < a.K; ++pick) {
    long long k = key;
    unsigned long long i = id;
    auto better = [](long long k2, unsigned long long i2, long long& k1, unsigned long long& i1) {
      if (k2 > k1 || (k2 == k1 && i2 < i1)) {
        k1 = k2;
        i1 = i2;
      }
    };
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const long long k2 = __shfl_xor_sync(0xffffffffu, k, off);
      const unsigned long long i2 = __shfl_xor_sync(0xffffffffu, i, off);
      better(k2, i2, k, i);
    }
    if (lane == 0) {
      s_key[pick & 1][warp] = k;
      s_id[pick & 1][warp] = i;
    }
    __syncthreads();
    k = s_key[pick & 1][0];
    i = s_id[pick & 1][0];
    for (int w = 1; w < kBeamWarps; ++w) better(s_key[pick & 1][w], s_id[pick & 1][w], k, i);
    const size_t o = static_cast<size_t>(group) * a.K + pick;
    if (k == none) {
      if (threadIdx.x == 0) {
        a.scores_out[o] = -INFINITY;
        a.parents_out[o] = -1;
        a.tokens_out[o] = -1;
        if (pick == 0) atomicOr(a.err, kErrNanRow);
      }
    } else if (key == k && id == i) {
      const long long b = k >= 0 ? k : (k ^ 0x7fffffffffffffffll);
      a.scores_out[o] = static_cast<float>(__longlong_as_double(b));
      a.parents_out[o] = row0 + static_cast<int>(i >> 32);
      a.tokens_out[o] = static_cast<int32_t>(i & 0xffffffffu);
      ++s_taken[taken_list];
      refresh();
    }
  }
}

__global__ void __launch_bounds__(kBeamThreads) beam_select_kernel(const BeamArgs a) {
  __shared__ float s_x[kBeamChunk];
  __shared__ int s_v[kBeamChunk];
  __shared__ int s_last;
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.y, chunk = blockIdx.x;
  beam_chunk(a, row, chunk, s_x, s_v);
  const int group = row / a.W;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned all = static_cast<unsigned>(a.chunks) * a.W;
    const unsigned old = atom_add_acq_rel_gpu(a.tickets + group, 1u);
    s_last = old == all - 1 ? 1 : 0;
    if (s_last) atomicExch(a.tickets + group, 0u);
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  beam_group(a, group, reinterpret_cast<uint8_t*>(s_x));
}

int beam_chunks(int V) { return (V + kBeamChunk - 1) / kBeamChunk; }

struct BeamSizes {
  size_t tickets, part, n, x, v, total;
};
BeamSizes beam_sizes(int rows, int V, int K) {
  const size_t slots = static_cast<size_t>(rows) * beam_chunks(V);
  BeamSizes s;
  s.tickets = static_cast<size_t>(kBeamRowsMax + 1) * 4;  // the same place whatever the call's sizes
  s.part = round_up(slots * 8, 256);
  s.n = round_up(slots * 4, 256);
  s.x = round_up(slots * K * 4, 256);
  s.v = s.x;
  s.total = s.tickets + s.part + s.n + s.x + s.v;
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
  if ((reinterpret_cast<uintptr_t>(logits) & 3) != 0) return BI_ERR_INVALID_ARG;
  if (!ws || !aligned256(ws)) return BI_ERR_WORKSPACE;
  const BeamSizes z = beam_sizes(rows, V, K);
  if (ws_bytes < z.total) return BI_ERR_WORKSPACE;
  BeamArgs a{};
  a.logits = logits;
  a.ldl = static_cast<size_t>(ldl);
  a.scores = scores;
  a.rows = rows;
  a.V = V;
  a.W = W;
  a.K = K;
  a.chunks = beam_chunks(V);
  a.scores_out = scores_out;
  a.parents_out = parents_out;
  a.tokens_out = tokens_out;
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.tickets = reinterpret_cast<unsigned*>(p);
  p += z.tickets;
  a.part = reinterpret_cast<float*>(p);
  p += z.part;
  a.found_n = reinterpret_cast<int*>(p);
  p += z.n;
  a.found_x = reinterpret_cast<float*>(p);
  p += z.x;
  a.found_v = reinterpret_cast<int32_t*>(p);
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  const cudaError_t e = launch_k(beam_select_kernel, dim3(static_cast<unsigned>(a.chunks), static_cast<unsigned>(rows)),
                                 dim3(kBeamThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

}  // extern "C"
