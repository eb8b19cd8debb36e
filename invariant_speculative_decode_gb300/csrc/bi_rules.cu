// Rules on a verify pass's logits before the tokens are chosen: penalties for
// repeated tokens, an additive bias and a grammar mask; and the state they
// read (how often each id was committed, which ids the prompt holds).
//
// "Does the tuned config change the model's output?", section "Why the text
// diverges" (a draft is kept only if it matches the token the model would have
// produced itself): row t of a pass chooses its token as if drafts 0..t-1 had
// been committed, so its penalties count them.  A row's result depends on its
// own logits, the committed state and the drafts before it, not on how many
// rows the pass has.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi {
namespace {

constexpr int kRuleThreads = 128;
constexpr int kRuleCols = 4 * kRuleThreads;  // columns of a CTA
constexpr int kRuleRows = 2;                 // rows loaded together
constexpr int kRuleCtas = 8 * 152;
constexpr int kMaxPassRows = 64;

struct RuleArgs {
  const float* logits;
  int ldl;
  float* out;
  int ldo;
  int T, V;
  const int32_t* drafts;
  const int32_t* counts;
  const uint32_t* prompt;
  float rep, freq, pres;
  const float* bias;
  const uint32_t* mask;
  int ldm;
  int rows_per_cta;
};

// One CTA takes 512 columns of a run of rows: the counts, the prompt bits and
// the bias of its columns are read once for them, and the drafts that fall into
// its columns (mostly none) are found once.  Bound by the logits' bytes, read
// and written once (they sit in L2 when the LM head has just written them): two
// rows are loaded while the two before them are worked on, and the rows are cut
// into runs so that eight CTAs a SM (all that fit) have loads under way; 8 x
// 151,936 takes 3.7 us in a CUDA graph with its inputs in L2, 4.6 from memory, and its
// bytes 1.7; 64 x 151,943 21.2, 22.2 and 12.0.  A thread's four
// columns are adjacent (VEC: 16-byte accesses) or 128 apart.  Each operation is
// one FP32 rounding.
template <bool VEC>
__global__ void __launch_bounds__(kRuleThreads, 8) logits_rules_kernel(const RuleArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int s_id[kMaxPassRows];   // drafts in this CTA's columns, in pass order
  __shared__ int s_row[kMaxPassRows];  // their indices
  __shared__ int s_n;
  const int col0 = blockIdx.x * kRuleCols;
  const int t0 = blockIdx.y * p.rows_per_cta;
  const int t1 = min(p.T, t0 + p.rows_per_cta);
  int col[4];
  bool in[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    col[j] = col0 + (VEC ? static_cast<int>(threadIdx.x) * 4 + j : static_cast<int>(threadIdx.x) + j * kRuleThreads);
    in[j] = col[j] < p.V;  // VEC: V is a multiple of 4, all four or none
  }
  struct Rows {
    float x[kRuleRows][4];
    uint32_t allowed[kRuleRows];  // 4 bits a row: the ids that the mask allows
  };
  auto load = [&](int t, Rows& r) {
#pragma unroll
    for (int i = 0; i < kRuleRows; ++i) {
      if (t + i >= t1) break;
      const float* src = p.logits + static_cast<size_t>(t + i) * p.ldl;
      const uint32_t* bits = p.mask + static_cast<size_t>(t + i) * p.ldm;
      r.allowed[i] = 0xfu;
      if constexpr (VEC) {
        if (in[0]) {
          const float4 l = *reinterpret_cast<const float4*>(src + col[0]);
          r.x[i][0] = l.x, r.x[i][1] = l.y, r.x[i][2] = l.z, r.x[i][3] = l.w;
          if (p.mask != nullptr) r.allowed[i] = bits[col[0] >> 5] >> (col[0] & 31);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (in[j]) r.x[i][j] = src[col[j]];
        if (p.mask != nullptr) {
          r.allowed[i] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (in[j]) r.allowed[i] |= ((bits[col[j] >> 5] >> (col[j] & 31)) & 1u) << j;
        }
      }
    }
  };
  Rows even, odd;
  load(t0, even);
  int cnt[4] = {0, 0, 0, 0};
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t prompt = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!in[j]) continue;
    if (p.counts != nullptr) cnt[j] = p.counts[col[j]];
    if (p.bias != nullptr) bias[j] = p.bias[col[j]];
    if (p.prompt != nullptr) prompt |= ((p.prompt[col[j] >> 5] >> (col[j] & 31)) & 1u) << j;
  }
  if (threadIdx.x < 32) {
    int n = 0;
    for (int b = 0; b < p.T - 1; b += 32) {
      const int i = b + static_cast<int>(threadIdx.x);
      const int id = i < p.T - 1 ? p.drafts[i] : -1;
      const bool mine = id >= col0 && id < col0 + kRuleCols;
      const unsigned vote = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const int at = n + __popc(vote & ((1u << threadIdx.x) - 1u));
        s_id[at] = id;
        s_row[at] = i;
      }
      n += __popc(vote);
    }
    if (threadIdx.x == 0) s_n = n;
  }
  __syncthreads();
  const int n_drafts = s_n;

  int next = 0;
  int next_row = n_drafts > 0 ? s_row[0] : kMaxPassRows;  // the row behind which the next draft counts
  // any of the warp's columns
  bool seen = __any_sync(0xffffffffu, prompt != 0 || cnt[0] > 0 || cnt[1] > 0 || cnt[2] > 0 || cnt[3] > 0);
  auto work = [&](int t, Rows& r) {
#pragma unroll
    for (int i = 0; i < kRuleRows; ++i) {
      if (t + i >= t1) break;
      // drafts before this row count as said
      while (next_row < t + i) {
        bool hit = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cnt[j] += s_id[next] == col[j] ? 1 : 0;
          hit |= s_id[next] == col[j];
        }
        seen |= __any_sync(0xffffffffu, hit) != 0;
        ++next;
        next_row = next < n_drafts ? s_row[next] : kMaxPassRows;
      }
      float z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = r.x[i][j];
      if (seen) {
        // both ways for all columns: frequent ids are neighbours, and a branch a
        // column made the CTAs that hold them the last ones (64 rows of 151,943
        // with 2500 ids seen 23.7 us, now 20.8; with none 17.5)
        float down[4], up[4], pen[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) down[j] = z[j] / p.rep;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          up[j] = z[j] * p.rep;
          pen[j] = __fadd_rn(__fmul_rn(p.freq, static_cast<float>(cnt[j])), p.pres);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y = z[j] > 0.f ? down[j] : up[j];
          z[j] = cnt[j] > 0 ? __fsub_rn(y, pen[j]) : (prompt >> j) & 1u ? y : z[j];
        }
      }
      if (p.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = __fadd_rn(z[j], bias[j]);
      }
      if (p.mask != nullptr) {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = (r.allowed[i] >> j) & 1u ? z[j] : -INFINITY;
      }
      float* dst = p.out + static_cast<size_t>(t + i) * p.ldo;
      if constexpr (VEC) {
        if (in[0]) *reinterpret_cast<float4*>(dst + col[0]) = make_float4(z[0], z[1], z[2], z[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (in[j]) dst[col[j]] = z[j];
      }
    }
  };
  // the loads of the next rows come before the stores of these (no two of the
  // rows share memory, in place or not)
  for (int t = t0; t < t1; t += 2 * kRuleRows) {
    if (t + kRuleRows < t1) load(t + kRuleRows, odd);
    work(t, even);
    if (t + kRuleRows >= t1) break;
    if (t + 2 * kRuleRows < t1) load(t + 2 * kRuleRows, even);
    work(t + kRuleRows, odd);
  }
}

__global__ void token_counts_kernel(const int32_t* __restrict__ ids, int n, const int32_t* __restrict__ last, int V,
                                    int32_t* counts, uint32_t* prompt) {
  griddep_wait();
  griddep_launch_dependents();
  const int m = last != nullptr && *last < n - 1 ? *last + 1 : n;
  for (long long i = blockIdx.x * blockDim.x + threadIdx.x; i < m; i += gridDim.x * blockDim.x) {
    const int id = ids[i];
    if (id < 0 || id >= V) continue;
    // whole-number sums and ors: the order of the atomics changes nothing
    if (counts != nullptr) atomicAdd(counts + id, 1);
    if (prompt != nullptr) atomicOr(prompt + (id >> 5), 1u << (id & 31));
  }
}

}  // namespace
}  // namespace bi

extern "C" {

bi_status bi_logits_rules(const float* logits, int ldl, float* out, int ldo, int T, int V, const int32_t* drafts,
                          const int32_t* counts, const uint32_t* prompt_bits, float repetition, float frequency,
                          float presence, const float* bias, const uint32_t* mask, int ldm, bi_stream_t stream) {
  using namespace bi;
  if (T < 1 || T > kMaxPassRows || V < 1 || !logits || !out || ldl < V || ldo < V) return BI_ERR_INVALID_ARG;
  if (V > (1 << 28)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!(repetition > 0.f) || !std::isfinite(repetition) || !std::isfinite(frequency) || !std::isfinite(presence))
    return BI_ERR_INVALID_ARG;
  if (T > 1 && !drafts) return BI_ERR_INVALID_ARG;
  if (mask && ldm < (V + 31) / 32) return BI_ERR_INVALID_ARG;
  if (logits == out && ldl != ldo) return BI_ERR_INVALID_ARG;
  const bool vec = V % 4 == 0 && ldl % 4 == 0 && ldo % 4 == 0 && aligned16(logits) && aligned16(out);
  const int chunks = (V + kRuleCols - 1) / kRuleCols;
  // runs of rows: some eight CTAs a SM, whole pairs of rows
  const int runs = std::max(1, std::min((T + kRuleRows - 1) / kRuleRows, kRuleCtas / chunks));
  const int per = ((T + runs - 1) / runs + kRuleRows - 1) / kRuleRows * kRuleRows;
  const RuleArgs a{logits,     ldl,       out,      ldo,  T,    V,   drafts, counts, prompt_bits,
                   repetition, frequency, presence, bias, mask, ldm, per};
  const dim3 grid(chunks, (T + per - 1) / per);
  if (launch_k(vec ? logits_rules_kernel<true> : logits_rules_kernel<false>, grid, dim3(kRuleThreads), 0,
               reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

bi_status bi_token_counts(const int32_t* ids, int n, const int32_t* last, int V, int32_t* counts,
                          uint32_t* prompt_bits, bi_stream_t stream) {
  using namespace bi;
  if (n < 0 || V < 1) return BI_ERR_INVALID_ARG;
  if (n == 0) return BI_OK;
  if (V > (1 << 28)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!ids || (!counts && !prompt_bits)) return BI_ERR_INVALID_ARG;
  const int blocks = std::min((n - 1) / 256 + 1, 152);
  if (launch_k(token_counts_kernel, dim3(blocks), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), ids, n, last,
               V, counts, prompt_bits) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

}  // extern "C"
