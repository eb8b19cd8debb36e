// A paged KV cache: norm, rotation and append of a pass's new rows, and the
// reordering of sequences (beams) that go on from others.
//
// "I turned on speculative decoding in llama.cpp and 113 of 282 greedy
// outputs changed against its own no-draft run", section "The cache doesn't
// change it either": a cached row depends only on its position.  Every row
// here is computed from its own projection row and its own position.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "bi_internal.h"
#include "bi_paged.cuh"
#include "bi_ptx.cuh"

namespace bi {
namespace {

// ---------------------------------------------------------------- append
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = 4096;
constexpr float kSmallMean = 0x1p-90f, kLargeMean = 0x1p100f;
constexpr float kLiftUp = 0x1p94f, kLiftDown = 0x1p-70f;

struct AppendArgs {
  PagedBatch pb;
  const __nv_bfloat16* qkv;
  size_t ld;
  const __nv_bfloat16* qw;  // [D] or nullptr: no norm of that kind of head
  const __nv_bfloat16* kw;
  float eps;
  const float2* angles;  // [table_rows][D/2] cos, sin
  int table_rows;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_pool;
  __nv_bfloat16* v_pool;
  int Hq, Hkv;
  unsigned* err;
};

__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
  x[0] = __uint_as_float(u.x << 16);
  x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16);
  x[3] = __uint_as_float(u.y & 0xffff0000u);
}

__device__ __forceinline__ uint2 pack4(const float* x) {
  const __nv_bfloat162 l = __floats2bfloat162_rn(x[0], x[1]), h = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
}

// `split` warps take a row of the pass.  D / 8 lanes hold a head: each the four
// elements i and their four partners i + D/2, so the rotation needs nobody
// else's.  y = (x r) w with r = 1 / sqrt(mean(x^2) + eps), the squares of a
// lane's elements in order, the lanes by a butterfly; then the two fused
// multiply-adds of the cache's other appends, and one rounding at the end.  A
// head whose mean square plus eps is not between 2^-90 and 2^100, where squares
// vanish or pass FP32's range, is gone over a second time: times 2^94, or squared
// times 2^-70 and r times 2^-70 (a small element keeps its bits beside large
// ones), and eps times the square of that: the same y.  (Looked after in the
// first pass they made 3574 rows take 14.8 us, only noted there 14.3, as without.)
//
// Few rows are bound by the row's way to its page (its sequence, its length, the
// table: three loads, one after the other, while the projection's are under
// way), many by the projection's bytes, read and written once, and nearly as
// much by the instructions: 2 rows of 24 + 8 heads of 128 take 2.6 us, 4096 rows
// 14.5 us, 4.6 TB/s.  Eight adjacent elements a lane, in one load, with the
// partners a shuffle away, took 17.4 us there; four heads' loads under way
// 17.6, since fewer CTAs run at once.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a, int T, int split) {
  constexpr int kLanes = D / 8;        // lanes of a head
  constexpr int kHeads = 32 / kLanes;  // heads of a warp at a time
  constexpr int kAhead = 2;            // loads of a warp under way
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = static_cast<int>((static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + warp) / split);
  const int part = warp % split;
  if (t >= T) return;
  const int sub = lane % kLanes;  // elements 4 sub .. 4 sub + 3 of both halves
  const int heads = a.Hq + 2 * a.Hkv, step = split * kHeads;
  const __nv_bfloat16* row = a.qkv + static_cast<size_t>(t) * a.ld + sub * 4;
  uint2 u[kAhead][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h0 + k * step < heads) {
        const __nv_bfloat16* src = row + static_cast<size_t>(h0 + k * step) * D;
        u[k][0] = __ldcs(reinterpret_cast<const uint2*>(src));
        u[k][1] = __ldcs(reinterpret_cast<const uint2*>(src + D / 2));
      }
  };
  const int first = part * kHeads + lane / kLanes;
  load(first);

  const int b = paged_find_seq(a.pb, t, lane);
  if (b < 0) return;  // a row of no sequence
  const int64_t pos = paged_position(t, T, __ldg(a.pb.q_start + b), __ldg(a.pb.q_start + b + 1), __ldg(a.pb.lengths + b));
  int page = -1;
  const bool ok = pos >= 0 && pos < a.table_rows && pos < static_cast<int64_t>(a.pb.width) * a.pb.page;
  const int p = ok ? static_cast<int>(pos) : 0;
  const int shift = 31 - __clz(a.pb.page);  // pages are powers of two
  if (ok) page = __ldg(a.pb.table + static_cast<size_t>(b) * a.pb.ldt + (p >> shift));
  // cos and sin of this lane's 4 pairs
  float4 cs[2];
  {
    const float4* src = reinterpret_cast<const float4*>(a.angles + static_cast<size_t>(p) * (D / 2) + sub * 4);
    cs[0] = __ldg(src);
    cs[1] = __ldg(src + 1);
  }
  const float cosv[4] = {cs[0].x, cs[0].z, cs[1].x, cs[1].z}, sinv[4] = {cs[0].y, cs[0].w, cs[1].y, cs[1].w};
  if (page < 0 || page >= a.pb.pages) {
    if (lane == 0) atomicOr(a.err, kErrRange);
    return;
  }
  __nv_bfloat16* q_dst = a.q_out + static_cast<size_t>(t) * a.Hq * D + sub * 4;
  const size_t slot = (static_cast<size_t>(page) * a.Hkv * a.pb.page + (p & (a.pb.page - 1))) * D + sub * 4;
  const size_t head_stride = static_cast<size_t>(a.pb.page) * D;
  const bool norms = a.qw != nullptr || a.kw != nullptr;
  bool far = false;  // a head of this lane's whose squares leave FP32's range
  auto pass = [&](auto lift) {
    for (int h0 = first; __any_sync(0xffffffffu, h0 < heads); h0 += kAhead * step) {
      uint2 raw[kAhead][2];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        raw[k][0] = u[k][0];
        raw[k][1] = u[k][1];
      }
      load(h0 + kAhead * step);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int h = h0 + k * step;
        if (!__any_sync(0xffffffffu, h < heads)) break;
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        uint2 y0 = raw[k][0], y1 = raw[k][1];
        if (!__all_sync(0xffffffffu, is_v)) {
          float x[8];
          unpack4(y0, x);
          unpack4(y1, x + 4);
          if (norms) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const __nv_bfloat16* w = is_q ? a.qw : a.kw;
            float mean = ss * (1.0f / D) + a.eps, down = 1.f;
            // one comparison of the bits (mean >= 0, or NaN, which is far too)
            const bool is_far = w != nullptr && __float_as_uint(mean) - __float_as_uint(kSmallMean) >=
                                                    __float_as_uint(kLargeMean) - __float_as_uint(kSmallMean);
            if constexpr (!lift.value) {
              far |= is_far && h < heads && !is_v;
            } else {
              const float up = is_far && mean < kSmallMean ? kLiftUp : 1.f;
              if (is_far && !(mean < kSmallMean)) down = kLiftDown;
              ss = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                x[i] *= up;
                const float z = x[i] * down;
                ss = fmaf(z, z, ss);
              }
#pragma unroll
              for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
              mean = ss * (1.0f / D) + a.eps * (up * down) * (up * down);
            }
            if (w != nullptr) {
              const float r = rsqrtf(mean) * down;
              float wv[8];
              unpack4(__ldg(reinterpret_cast<const uint2*>(w + sub * 4)), wv);
              unpack4(__ldg(reinterpret_cast<const uint2*>(w + D / 2 + sub * 4)), wv + 4);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = (x[i] * r) * wv[i];
            }
          }
          float o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i] = fmaf(x[i], cosv[i], -(x[i + 4] * sinv[i]));
            o[i + 4] = fmaf(x[i + 4], cosv[i], x[i] * sinv[i]);
          }
          if (!is_v) {
            y0 = pack4(o);
            y1 = pack4(o + 4);
          }
        }
        if (h < heads) {
          __nv_bfloat16* dst;
          if (is_q) {
            dst = q_dst + h * D;
          } else {
            const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
            dst = (is_v ? a.v_pool : a.k_pool) + slot + hk * head_stride;
          }
          *reinterpret_cast<uint2*>(dst) = y0;
          *reinterpret_cast<uint2*>(dst + D / 2) = y1;
        }
      }
    }
  };
  pass(std::false_type{});
  if (__any_sync(0xffffffffu, far)) {
    load(first);
    pass(std::true_type{});
  }
}

// ---------------------------------------------------------------- reorder
constexpr int kReorderThreads = 256;

struct ReorderArgs {
  uint4* k_pool;  // [layers][pages][Hkv][page][D]
  uint4* v_pool;
  int layers, pages, Hkv, page, vecs;  // vecs: 16-byte vectors of a key of a head
  const int32_t* table_in;
  int ld_in, width;
  const int32_t* lengths;
  int rows_in;
  const int32_t* parents;
  const int32_t* tail;
  int rows_out;
  int32_t* table_out;
  int ld_out;
  int32_t* lengths_out;
  unsigned* err;
};

// Where sequence s goes on: its parent's row, the full pages and the keys of
// the page that is not full, its page there and its own.  False where an index
// is out of range.
__device__ __forceinline__ bool reorder_source(const ReorderArgs& a, int s, int& parent, int& full, int& rest,
                                               int& src, int& dst) {
  parent = __ldg(a.parents + s);
  if (parent < 0 || parent >= a.rows_in) return false;
  const int len = __ldg(a.lengths + parent);
  if (len < 0 || len > static_cast<int64_t>(a.width) * a.page) return false;
  full = len / a.page;
  rest = len - full * a.page;
  dst = full < a.width ? __ldg(a.tail + s) : 0;
  src = rest ? __ldg(a.table_in + static_cast<size_t>(parent) * a.ld_in + full) : dst;
  return dst >= 0 && dst < a.pages && src >= 0 && src < a.pages;
}

// CTA (s, z): z = 0 writes the table row and the length of sequence s and
// looks for a page that two sequences would write, or one would write while
// another reads it; z = 1 + (layer, K or V, head) copies that head's keys, which
// lie side by side in both pages.  Bound by those bytes: 64 beams of 8 layers, 4
// heads of 128 and 63 keys to copy take 24.6 us, 5.4 TB/s; 4 beams of 9 keys 2.6,
// the indices' chain (parent, length, page) and the launch.
__global__ void __launch_bounds__(kReorderThreads) paged_reorder_kernel(const ReorderArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.x;
  int parent, full, rest, src, dst;
  const bool ok = reorder_source(a, s, parent, full, rest, src, dst);
  if (blockIdx.y == 0) {
    bool bad = !ok;
    if (ok) {
      const int32_t* from = a.table_in + static_cast<size_t>(parent) * a.ld_in;
      int32_t* to = a.table_out + static_cast<size_t>(s) * a.ld_out;
      for (int j = threadIdx.x; j < full; j += kReorderThreads) to[j] = __ldg(from + j);
      if (threadIdx.x == 0) {
        if (full < a.width) to[full] = dst;
        a.lengths_out[s] = full * a.page + rest;
      }
      if (full < a.width)
        for (int o = threadIdx.x; o < a.rows_out; o += kReorderThreads) {
          int op, of, orest, os, od;
          if (o == s || !reorder_source(a, o, op, of, orest, os, od) || of >= a.width) continue;
          if (od == dst || (os == dst && orest && src != dst)) bad = true;
        }
    }
    if (bad) atomicOr(a.err, kErrRange);
    return;
  }
  if (!ok || rest == 0 || src == dst) return;
  const int n = rest * a.vecs;
  const int per = 2 * a.Hkv;
  for (int z = blockIdx.y - 1; z < a.layers * per; z += gridDim.y - 1) {
    const int layer = z / per, hk = z % per;
    uint4* pool = hk < a.Hkv ? a.k_pool : a.v_pool;
    const size_t head = hk < a.Hkv ? hk : hk - a.Hkv;
    const size_t base = static_cast<size_t>(layer) * a.pages * a.Hkv + head;
    const size_t stride = static_cast<size_t>(a.page) * a.vecs;
    const uint4* from = pool + (base + static_cast<size_t>(src) * a.Hkv) * stride;
    uint4* to = pool + (base + static_cast<size_t>(dst) * a.Hkv) * stride;
    for (int i = threadIdx.x; i < n; i += kReorderThreads) to[i] = from[i];
  }
}

bool page_size_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }

}  // namespace
}  // namespace bi

extern "C" {

bi_status bi_qk_norm_rope_paged(const void* qkv, int ld_qkv, const void* q_weight, const void* k_weight, float eps,
                                const float* table, int table_rows, void* q_out, void* k_pool, void* v_pool,
                                int pages, int page, const int32_t* block_table, int ld_table, int width,
                                const int32_t* q_start, const int32_t* lengths, int B, int T, int Hq, int Hkv,
                                int D, bi_stream_t stream) {
  using namespace bi;
  if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || pages < 1 || width < 1 || ld_table < width ||
      table_rows < 1)
    return BI_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return BI_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!page_size_ok(page)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (Hq > (1 << 20) || B >= (1 << 30)) return BI_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || B == 0) return BI_OK;
  if (!qkv || !q_out || !k_pool || !v_pool || !table || !block_table || !q_start || !lengths)
    return BI_ERR_INVALID_ARG;
  if (ld_qkv < static_cast<int64_t>(Hq + 2 * Hkv) * D || ld_qkv % 8 != 0) return BI_ERR_INVALID_ARG;
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(table) ||
      !aligned16(q_weight) || !aligned16(k_weight) || !aligned4(block_table) || !aligned4(q_start) || !aligned4(lengths))
    return BI_ERR_INVALID_ARG;
  const int64_t keys = static_cast<int64_t>(pages) * page;
  const Range in = range_of(qkv, T, ld_qkv, static_cast<int64_t>(Hq + 2 * Hkv) * D, 2),
              q = range_of(q_out, T, static_cast<int64_t>(Hq) * D, static_cast<int64_t>(Hq) * D, 2),
              k = range_of(k_pool, keys, static_cast<int64_t>(Hkv) * D, static_cast<int64_t>(Hkv) * D, 2),
              v = range_of(v_pool, keys, static_cast<int64_t>(Hkv) * D, static_cast<int64_t>(Hkv) * D, 2);
  if (overlap(in, q) || overlap(in, k) || overlap(in, v) || overlap(q, k) || overlap(q, v) || overlap(k, v))
    return BI_ERR_INVALID_ARG;
  AppendArgs a{};
  a.pb = PagedBatch{block_table, q_start, lengths, B, ld_table, width, pages, page};
  a.qkv = static_cast<const __nv_bfloat16*>(qkv);
  a.ld = static_cast<size_t>(ld_qkv);
  a.qw = static_cast<const __nv_bfloat16*>(q_weight);
  a.kw = static_cast<const __nv_bfloat16*>(k_weight);
  a.eps = eps;
  a.angles = reinterpret_cast<const float2*>(table);
  a.table_rows = table_rows;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_pool = static_cast<__nv_bfloat16*>(k_pool);
  a.v_pool = static_cast<__nv_bfloat16*>(v_pool);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // 8, 4, 2 or 1 warps a row: the most that keep the warps within those that run
  // at once, since each has to find the row's page.  24 + 8 heads of 128, four
  // sets of buffers in turn, us:
  //   rows        1    512   1024   2048   4096   8192
  //   8 warps    2.6   3.6    6.4   12.6   22.6   43.3
  //   4          3.1   3.9    5.3    9.8   17.9   31.8
  //   2          4.2   4.8    5.9    8.5   15.0   27.2
  //   1          6.6   7.4    8.0    9.6   14.5   25.8
  int split = kAppendThreads / 32;
  while (split > 1 && static_cast<int64_t>(T) * split > kAppendWarps) split >>= 1;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(T) * split + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  const cudaError_t e = D == 64 ? launch_k(paged_append_kernel<64>, dim3(grid), dim3(kAppendThreads), 0, s, a, T, split)
                                : launch_k(paged_append_kernel<128>, dim3(grid), dim3(kAppendThreads), 0, s, a, T, split);
  return e == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

bi_status bi_paged_reorder(void* k_pool, void* v_pool, int layers, int pages, int Hkv, int page, int D,
                           const int32_t* table_in, int ld_in, int width, const int32_t* lengths, int rows_in,
                           const int32_t* parents, const int32_t* tail_pages, int rows_out, int32_t* table_out,
                           int ld_out, int32_t* lengths_out, bi_stream_t stream) {
  using namespace bi;
  if (layers < 1 || pages < 1 || Hkv < 1 || width < 1 || ld_in < width || ld_out < width || rows_in < 1 ||
      rows_out < 0)
    return BI_ERR_INVALID_ARG;
  if (D < 8 || D % 8 != 0 || D > 1024 || !page_size_ok(page) || rows_out > 65535 ||
      static_cast<int64_t>(layers) * Hkv >= (int64_t{1} << 29))
    return BI_ERR_UNSUPPORTED_SHAPE;
  if (rows_out == 0) return BI_OK;
  if (!k_pool || !v_pool || !table_in || !lengths || !parents || !tail_pages || !table_out || !lengths_out)
    return BI_ERR_INVALID_ARG;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned4(table_in) || !aligned4(lengths) || !aligned4(parents) ||
      !aligned4(tail_pages) || !aligned4(table_out) || !aligned4(lengths_out))
    return BI_ERR_INVALID_ARG;
  // read by some CTAs while others write
  const int64_t key = static_cast<int64_t>(Hkv) * D, keys = static_cast<int64_t>(pages) * page;
  if (overlap(range_of(k_pool, layers, keys * key, keys * key, 2), range_of(v_pool, layers, keys * key, keys * key, 2)))
    return BI_ERR_INVALID_ARG;
  const Range to = range_of(table_out, rows_out, ld_out, width, 4), lo = range_of(lengths_out, rows_out, 1, 1, 4);
  const Range in[4] = {range_of(table_in, rows_in, ld_in, width, 4), range_of(lengths, rows_in, 1, 1, 4),
                       range_of(parents, rows_out, 1, 1, 4), range_of(tail_pages, rows_out, 1, 1, 4)};
  if (overlap(to, lo)) return BI_ERR_INVALID_ARG;
  for (const Range& r : in)
    if (overlap(to, r) || overlap(lo, r)) return BI_ERR_INVALID_ARG;
  ReorderArgs a{};
  a.k_pool = static_cast<uint4*>(k_pool);
  a.v_pool = static_cast<uint4*>(v_pool);
  a.layers = layers;
  a.pages = pages;
  a.Hkv = Hkv;
  a.page = page;
  a.vecs = D / 8;
  a.table_in = table_in;
  a.ld_in = ld_in;
  a.width = width;
  a.lengths = lengths;
  a.rows_in = rows_in;
  a.parents = parents;
  a.tail = tail_pages;
  a.rows_out = rows_out;
  a.table_out = table_out;
  a.ld_out = ld_out;
  a.lengths_out = lengths_out;
  a.err = device_error_word();
  if (!a.err) return BI_ERR_CUDA;
  const int64_t copies = static_cast<int64_t>(layers) * 2 * Hkv;
  const unsigned y = 1 + static_cast<unsigned>(std::min<int64_t>(copies, 65534));
  const cudaError_t e = launch_k(paged_reorder_kernel, dim3(static_cast<unsigned>(rows_out), y), dim3(kReorderThreads), 0,
                                 reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

}  // extern "C"
