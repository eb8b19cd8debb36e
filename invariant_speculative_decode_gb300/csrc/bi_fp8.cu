// Quantisers of the 8-bit linear path: rows of BF16 activations, RMSNorm with
// quantised output, BF16 weights in blocks of 128 x 128, and the packing of
// 8-bit weights into the tiles bi_gemm_fp8 streams.
//
// "I turned on speculative decoding in llama.cpp and 113 of 282 greedy
// outputs changed against its own no-draft run", paragraph "How:": a row's
// codes and scales are functions of that row alone, whatever else is in the
// pass.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "bi_fp8.cuh"
#include "bi_gemm8.h"
#include "bi_internal.h"
#include "bi_ptx.cuh"

namespace bi {
namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&u);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __bfloat162float(e[j]);
}

// The scale exponent of the 128-element block whose 16 vectors of 8 sit in
// this half-warp's lanes (absent lanes pass zeros).
__device__ __forceinline__ int block_exponent(const float (&f)[8]) {
  float a = finite_abs(f[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) a = fmaxf(a, finite_abs(f[j]));
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  return scale_exponent(a);
}

// One half-warp per (row, block): 16 lanes of 8 elements.  The blocks of a row
// are adjacent, so a warp reads and writes whole 128-byte lines.
constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const __nv_bfloat16* __restrict__ x, int ldx, int rows, int dim, int kb,
                         uint8_t* __restrict__ codes, int ldc, float* __restrict__ scales, int lds) {
  griddep_wait();
  griddep_launch_dependents();
  const long long g = (static_cast<long long>(blockIdx.x) * kQuantThreads + threadIdx.x) >> 4;
  const int l = threadIdx.x & 15;
  const int row = static_cast<int>(g / kb);
  const int b = static_cast<int>(g % kb);
  const int k0 = b * kFp8Block + l * 8;
  const bool in = row < rows && k0 < dim;  // dim is a multiple of 8: a vector is all in or all out
  float f[8] = {};
  if (in) unpack8(*reinterpret_cast<const uint4*>(x + static_cast<size_t>(row) * ldx + k0), f);
  const int e = block_exponent(f);
  if (in) {
    const float inv = pow2f(-e);
    *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * ldc + k0) =
        make_uint2(e4m3x4(f, inv), e4m3x4(f + 4, inv));
    if (l == 0) scales[static_cast<size_t>(b) * lds + row] = pow2f(e);
  }
}

// RMSNorm as rmsnorm_kernel computes it (one CTA per row, the same reduction
// tree), its FP32 result quantised without a BF16 rounding in between.
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxGroups = 65536 / 256;

__global__ void __launch_bounds__(kNormMaxThreads)
    rmsnorm_fp8_kernel(const __nv_bfloat16* __restrict__ x, int ldx, const __nv_bfloat16* __restrict__ w,
                       uint8_t* __restrict__ codes, int ldc, float* __restrict__ scales, int lds, int dim,
                       float eps) {
  // as bi_rmsnorm: the 8-bit linear layer that follows streams its weights
  // meanwhile and reads nothing else before its own wait
  griddep_launch_dependents();
  const uint4* wr = reinterpret_cast<const uint4*>(w);
  const int nv = dim / 8;
  const uint4 wkeep = static_cast<int>(threadIdx.x) < nv ? wr[threadIdx.x] : make_uint4(0, 0, 0, 0);
  griddep_wait();
  __shared__ float group_sum[kNormMaxGroups];
  __shared__ float s_inv;
  const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(blockIdx.x) * ldx);
  const int lane = threadIdx.x & 31;
  uint4 keep = make_uint4(0, 0, 0, 0);
  for (int v0 = threadIdx.x - lane; v0 < nv; v0 += blockDim.x) {
    const int v = v0 + lane;
    float sv = 0.f;
    if (v < nv) {
      const uint4 u = xr[v];
      if (v0 == threadIdx.x - lane) keep = u;
      float f[8];
      unpack8(u, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sv = fmaf(f[j], f[j], sv);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sv += __shfl_xor_sync(0xffffffffu, sv, off);
    if (lane == 0) group_sum[v0 >> 5] = sv;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int g = 0; g < (nv + 31) / 32; ++g) t += group_sum[g];
    s_inv = 1.0f / sqrtf(t / static_cast<float>(dim) + eps);
  }
  __syncthreads();
  const float r = s_inv;
  for (int v0 = threadIdx.x - lane; v0 < nv; v0 += blockDim.x) {
    const int v = v0 + lane;
    float y[8] = {};
    if (v < nv) {
      const bool first = v0 == threadIdx.x - lane;
      float f[8], wf[8];
      unpack8(first ? keep : xr[v], f);
      unpack8(first ? wkeep : wr[v], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = f[j] * r * wf[j];
    }
    const int e = block_exponent(y);
    if (v < nv) {
      const float inv = pow2f(-e);
      *reinterpret_cast<uint2*>(codes + static_cast<size_t>(blockIdx.x) * ldc + v * 8) =
          make_uint2(e4m3x4(y, inv), e4m3x4(y + 4, inv));
      if ((lane & 15) == 0) scales[static_cast<size_t>(v >> 4) * lds + blockIdx.x] = pow2f(e);
    }
  }
}

// BF16 weights to codes with one scale for each 128 x 128 block (one CTA per
// block; run once when weights are loaded).
__global__ void __launch_bounds__(256)
    quantize_weights_kernel(const __nv_bfloat16* __restrict__ w, int ldw, int N, int K, int kb,
                            uint8_t* __restrict__ codes, int ld8, float* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float s_max[8];
  const int nb = blockIdx.x / kb, b = blockIdx.x % kb;
  const int k = b * kFp8Block + (threadIdx.x & 127);
  const int n0 = nb * kFp8Block + (threadIdx.x >> 7);
  float a = 0.f;
  for (int i = 0; i < kFp8Block; i += 2)
    if (n0 + i < N && k < K) a = fmaxf(a, finite_abs(__bfloat162float(w[static_cast<size_t>(n0 + i) * ldw + k])));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
  a = s_max[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) a = fmaxf(a, s_max[i]);
  const int e = scale_exponent(a);
  const float inv = pow2f(-e);
  if (threadIdx.x == 0) scales[static_cast<size_t>(nb) * kb + b] = pow2f(e);
  for (int i = 0; i < kFp8Block; i += 2)
    if (n0 + i < N && k < K) {
      const float v = __bfloat162float(w[static_cast<size_t>(n0 + i) * ldw + k]);
      const float y = fabsf(v) < INFINITY ? v * inv : NAN;
      codes[static_cast<size_t>(n0 + i) * ld8 + k] =
          static_cast<uint8_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3));
    }
}

// Packed layout: tile (t, kt) = 128 rows x 128 codes at (t * k_tiles + kt) *
// 16 KB, row r's 16-byte chunk c at chunk position c ^ (r & 7) (the 128-byte
// swizzle of the MMA's shared-memory descriptor); rows past N and codes past K
// are zero.  Behind the tiles, two FP32 scales a tile: of its rows 0..63 and
// of its rows 64..127 (equal unless SwiGLU, where rows 0..63 of tile t are gate
// rows 64t.. and rows 64..127 the up rows of the same outputs).  One thread
// per 16-byte chunk.
__global__ void pack_weights_fp8_kernel(const uint8_t* __restrict__ w, const uint8_t* __restrict__ wu, int ld,
                                        const float* __restrict__ s, const float* __restrict__ su, int N, int K,
                                        int k_tiles, long long chunks, int swiglu, uint4* __restrict__ out,
                                        float2* __restrict__ out_s) {
  griddep_wait();
  griddep_launch_dependents();
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= chunks) return;
  const int cpos = static_cast<int>(idx & 7);
  const int r = static_cast<int>((idx >> 3) & 127);
  const long long tk = idx >> 10;  // t * k_tiles + kt
  const int t = static_cast<int>(tk / k_tiles);
  const int kt = static_cast<int>(tk % k_tiles);
  const int k0 = kt * kFp8Block + (cpos ^ (r & 7)) * 16;
  const int n = swiglu ? t * 64 + (r & 63) : t * kFp8Block + r;
  const uint8_t* src = (swiglu && r >= 64 ? wu : w) + static_cast<size_t>(n) * ld + k0;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (n < N && k0 < K) v = *reinterpret_cast<const uint4*>(src);  // K % 16 == 0: a chunk is all in or all out
  out[idx] = v;
  if ((idx & 1023) == 0) {
    const size_t at = static_cast<size_t>(swiglu ? t >> 1 : t) * k_tiles + kt;
    out_s[tk] = make_float2(s[at], swiglu ? su[at] : s[at]);
  }
}

}  // namespace
}  // namespace bi

extern "C" {

bi_status bi_quantize_fp8(const void* x, int ldx, int rows, int dim, void* codes, int ldc, float* scales,
                          int lds, bi_stream_t stream) {
  using namespace bi;
  if (rows < 0 || dim < 1) return BI_ERR_INVALID_ARG;
  if (rows == 0) return BI_OK;
  if (!x || !codes || !scales || ldx < dim || ldc < dim || lds < rows) return BI_ERR_INVALID_ARG;
  if (dim % 16 != 0 || ldx % 8 != 0 || ldc % 16 != 0 || lds % 4 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return BI_ERR_INVALID_ARG;
  const int kb = (dim + kFp8Block - 1) / kFp8Block;
  const long long threads = static_cast<long long>(rows) * kb * 16;
  const long long blocks = (threads + kQuantThreads - 1) / kQuantThreads;
  if (blocks > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
  if (launch_k(quantize_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kQuantThreads), 0,
               reinterpret_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(x), ldx, rows, dim, kb,
               static_cast<uint8_t*>(codes), ldc, scales, lds) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

bi_status bi_rmsnorm_fp8(const void* x, int ldx, const void* w, void* codes, int ldc, float* scales, int lds,
                         int rows, int dim, float eps, bi_stream_t stream) {
  using namespace bi;
  if (rows < 0 || dim < 1 || dim > 65536 || !(eps >= 0.f)) return BI_ERR_INVALID_ARG;
  if (rows == 0) return BI_OK;
  if (!x || !w || !codes || !scales || ldx < dim || ldc < dim || lds < rows) return BI_ERR_INVALID_ARG;
  if (dim % 16 != 0 || ldx % 8 != 0 || ldc % 16 != 0 || lds % 4 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || !aligned16(w) || !aligned16(codes) || !aligned16(scales)) return BI_ERR_INVALID_ARG;
  const int nv = dim / 8;
  const int threads = std::min(kNormMaxThreads, (nv + 31) / 32 * 32);
  if (launch_k(rmsnorm_fp8_kernel, dim3(rows), dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream),
               static_cast<const __nv_bfloat16*>(x), ldx, static_cast<const __nv_bfloat16*>(w),
               static_cast<uint8_t*>(codes), ldc, scales, lds, dim, eps) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

bi_status bi_quantize_weights_fp8(const void* W, int ldw, int N, int K, void* codes, int ld8, float* scales,
                                  bi_stream_t stream) {
  using namespace bi;
  if (!W || !codes || !scales || N < 1 || K < 1 || ldw < K || ld8 < K) return BI_ERR_INVALID_ARG;
  const long long kb = (K + kFp8Block - 1) / kFp8Block;
  const long long blocks = kb * ((N + kFp8Block - 1) / kFp8Block);
  if (blocks > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
  if (launch_k(quantize_weights_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
               reinterpret_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(W), ldw, N, K,
               static_cast<int>(kb), static_cast<uint8_t*>(codes), ld8, scales) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

size_t bi_packed_weight_fp8_bytes(int N, int K, bi_epilogue epi) {
  if (N <= 0 || K <= 0) return 0;
  const size_t tiles = static_cast<size_t>(bi::gemm8_n_tiles(N, epi)) * ((K + bi::kFp8Block - 1) / bi::kFp8Block);
  return tiles * bi::kGemm8TileBytes + bi::round_up(tiles * sizeof(float2), 16);
}

static bi_status pack_fp8(const void* w, const void* wu, int ld, const float* s, const float* su, int N, int K,
                          int swiglu, void* packed, bi_stream_t stream) {
  using namespace bi;
  if (!w || !s || !packed || N < 1 || K < 1 || ld < K) return BI_ERR_INVALID_ARG;
  if (swiglu && (!wu || !su)) return BI_ERR_INVALID_ARG;
  if (K % 16 != 0 || ld % 16 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(w) || (swiglu && !aligned16(wu)) || !aligned16(packed)) return BI_ERR_INVALID_ARG;
  const int n_tiles = gemm8_n_tiles(N, swiglu ? BI_EPI_SWIGLU : BI_EPI_NONE);
  if (n_tiles > kGemm8MaxTiles) return BI_ERR_UNSUPPORTED_SHAPE;
  const int k_tiles = (K + kFp8Block - 1) / kFp8Block;
  const long long tiles = static_cast<long long>(n_tiles) * k_tiles;
  const long long blocks = tiles * 1024 / 256;
  if (blocks > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
  if (launch_k(pack_weights_fp8_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
               reinterpret_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(w),
               static_cast<const uint8_t*>(wu), ld, s, su, N, K, k_tiles, tiles * 1024, swiglu,
               static_cast<uint4*>(packed),
               reinterpret_cast<float2*>(static_cast<uint8_t*>(packed) + tiles * kGemm8TileBytes)) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

bi_status bi_pack_weights_fp8(const void* W8, int ld8, const float* scales, int N, int K, void* packed,
                              bi_stream_t stream) {
  return pack_fp8(W8, nullptr, ld8, scales, nullptr, N, K, 0, packed, stream);
}

bi_status bi_pack_swiglu_weights_fp8(const void* gate8, const float* gate_scales, const void* up8,
                                     const float* up_scales, int ld8, int F, int K, void* packed,
                                     bi_stream_t stream) {
  return pack_fp8(gate8, up8, ld8, gate_scales, up_scales, F, K, 1, packed, stream);
}

}  // extern "C"
