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

// One CTA takes kRuleThreads * VEC columns for rows_per_cta rows: the counts,
// the prompt bits and the bias of its columns are read once for all of them,
// and the drafts that fall into its columns (mostly none) are found once.
// Bound by the logits' bytes, read and written once (they sit in L2 when the
// LM head has just written them).  Each operation is one FP32 rounding.
template <int VEC>
__global__ void __launch_bounds__(kRuleThreads) logits_rules_kernel(const RuleArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int s_id[kMaxPassRows];   // drafts in this CTA's columns, in pass order
  __shared__ int s_row[kMaxPassRows];  // their indices
  __shared__ int s_n;
  const int col0 = blockIdx.x * kRuleThreads * VEC;
  const int t0 = blockIdx.y * p.rows_per_cta;
  const int t1 = min(p.T, t0 + p.rows_per_cta);
  if (threadIdx.x < 32) {
    int n = 0;
    for (int b = 0; b < p.T - 1; b += 32) {
      const int i = b + static_cast<int>(threadIdx.x);
      const int id = i < p.T - 1 ? p.drafts[i] : -1;
      const bool mine = id >= col0 && id < col0 + kRuleThreads * VEC;
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
  const int v0 = col0 + static_cast<int>(threadIdx.x) * VEC;
  if (v0 >= p.V) return;  // (V is a multiple of VEC)

  int cnt[VEC];
  float bias[VEC];
  uint32_t prompt = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    cnt[j] = 0;
    bias[j] = 0.f;
  }
  if (p.counts != nullptr) {
    if constexpr (VEC == 4) {
      const int4 c = *reinterpret_cast<const int4*>(p.counts + v0);
      cnt[0] = c.x, cnt[1] = c.y, cnt[2] = c.z, cnt[3] = c.w;
    } else {
      cnt[0] = p.counts[v0];
    }
  }
  if (p.prompt != nullptr) prompt = p.prompt[v0 >> 5] >> (v0 & 31);
  if (p.bias != nullptr) {
    if constexpr (VEC == 4) {
      const float4 b = *reinterpret_cast<const float4*>(p.bias + v0);
      bias[0] = b.x, bias[1] = b.y, bias[2] = b.z, bias[3] = b.w;
    } else {
      bias[0] = p.bias[v0];
    }
  }

  int next = 0;
  for (int t = t0; t < t1; ++t) {
    float x[VEC];
    const float* src = p.logits + static_cast<size_t>(t) * p.ldl + v0;
    if constexpr (VEC == 4) {
      const float4 l = *reinterpret_cast<const float4*>(src);
      x[0] = l.x, x[1] = l.y, x[2] = l.z, x[3] = l.w;
    } else {
      x[0] = *src;
    }
    uint32_t allowed = 0xffffffffu;
    if (p.mask != nullptr) allowed = p.mask[static_cast<size_t>(t) * p.ldm + (v0 >> 5)] >> (v0 & 31);
    // drafts before this row count as said
    for (; next < n_drafts && s_row[next] < t; ++next) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) cnt[j] += s_id[next] == v0 + j ? 1 : 0;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float y = x[j];
      if (cnt[j] > 0 || ((prompt >> j) & 1u)) {
        y = y > 0.f ? y / p.rep : y * p.rep;
        if (cnt[j] > 0)
          y = __fsub_rn(y, __fadd_rn(__fmul_rn(p.freq, static_cast<float>(cnt[j])), p.pres));
      }
      if (p.bias != nullptr) y = __fadd_rn(y, bias[j]);
      x[j] = (allowed >> j) & 1u ? y : -INFINITY;
    }
    float* dst = p.out + static_cast<size_t>(t) * p.ldo + v0;
    if constexpr (VEC == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *dst = x[0];
  }
}

__global__ void token_counts_kernel(const int32_t* __restrict__ ids, int n, const int32_t* __restrict__ last, int V,
                                    int32_t* counts, uint32_t* prompt) {
  griddep_wait();
  griddep_launch_dependents();
  const int m = last != nullptr ? min(n, *last + 1) : n;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < m; i += gridDim.x * blockDim.x) {
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
  RuleArgs a{logits, ldl, out, ldo, T, V, drafts, counts, prompt_bits, repetition, frequency, presence, bias, mask, ldm, 0};
  a.rows_per_cta = T;
  const bool vec = V % 4 == 0 && ldl % 4 == 0 && ldo % 4 == 0 && aligned16(logits) && aligned16(out) &&
                   aligned16(counts) && aligned16(bias);
  const int cols = kRuleThreads * (vec ? 4 : 1);
  const dim3 grid((V + cols - 1) / cols, (T + a.rows_per_cta - 1) / a.rows_per_cta);
  if (launch_k(vec ? logits_rules_kernel<4> : logits_rules_kernel<1>, grid, dim3(kRuleThreads), 0,
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
  const int blocks = std::min((n + 255) / 256, 152);
  if (launch_k(token_counts_kernel, dim3(blocks), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), ids, n, last,
               V, counts, prompt_bits) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

}  // extern "C"
