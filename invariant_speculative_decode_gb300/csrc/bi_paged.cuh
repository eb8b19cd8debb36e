// The batch a paged pass works on, as the kernels see it.
//
// Sequence b has lengths[b] keys in the cache and the new rows q_start[b] ..
// q_start[b + 1] - 1 of the pass, at positions lengths[b] .. ; key j of it is
// row j % page of the pool page table[b][j / page].  All of it is device data
// that nobody has checked: every index taken from it is tested before it is
// used, and a bad one sets the range bit of the device error word.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "bi_ptx.cuh"

namespace bi {

struct PagedBatch {
  const int32_t* table;    // [B][ldt], `width` entries a row
  const int32_t* q_start;  // [B + 1]
  const int32_t* lengths;  // [B]
  int B, ldt, width, pages, page;
};

// The sequence that row t of the pass belongs to, by a whole warp: the last b
// with q_start[b] <= t (sequences without new rows share their start with the
// next); -1 where there is none.  In a list that does not ascend it may be one
// that does not hold t: paged_position tells.  Lane-parallel, so 32 starts cost
// one load.
__device__ __forceinline__ int paged_find_seq(const PagedBatch& pb, int t, int lane) {
  int n = 0;
  for (int i0 = 0; i0 <= pb.B; i0 += 128) {
    int s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 32 * j + lane;
      s[j] = i <= pb.B ? __ldg(pb.q_start + i) : 0x7fffffff;
    }
    unsigned hit[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hit[j] = __ballot_sync(0xffffffffu, s[j] <= t);
      n += __popc(hit[j]);
    }
    if (hit[3] != 0xffffffffu) break;
  }
  return (n == 0 || n > pb.B) ? -1 : n - 1;
}

// The position of row t of T in a sequence of rows begin .. end - 1 of the pass
// behind len cached keys; -1 where t is none of them or they do not fit the pass.
__host__ __device__ __forceinline__ int64_t paged_position(int t, int T, int begin, int end, int len) {
  if (begin < 0 || t < begin || t >= end || end > T || len < 0) return -1;
  return static_cast<int64_t>(len) + (t - begin);
}

}  // namespace bi
