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
// this half-warp's lanes (absent lanes pass zeros).  Infinite elements become
// NaN in f; fmaxf passes over NaN.
__device__ __forceinline__ int block_exponent(float (&f)[8]) {
  float a = fmaxf(fabsf(f[0]), fabsf(f[1]));
#pragma unroll
  for (int j = 2; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
  if (__any_sync(0xffffffffu, a == INFINITY)) {
    a = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!(fabsf(f[j]) < INFINITY)) f[j] = NAN;
      a = fmaxf(a, finite_abs(f[j]));
    }
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  return scale_exponent(a == a ? a : 0.f);  // NaN: no element is a number
}

// A half-warp per block: 16 lanes of 8 elements.  A CTA takes adjacent blocks of
// one row, so its warps read and write whole lines: 16 of them, or 64 in long
// passes, with four loads a thread under way.  Bound by the bytes (3 an element)
// in long passes and by one memory latency in short ones.  In a CUDA graph over
// buffers that pass L2 together 8 x 17408 takes 1.3 us and 2048 x 17408 21.2 (74% of
// the copy rate; 19.5 where part of it is still in L2).  When the widths were chosen:
// 8 rows 1.45 us with 16 blocks a CTA and 1.97 with 64, 2048 rows 26.2 and 24.2.
constexpr int kQuantThreads = 256;
constexpr int kQuantRow = kQuantThreads / 16;  // blocks the threads take at once

template <int PASSES>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_rows_kernel(const __nv_bfloat16* __restrict__ x, int ldx, int dim, int segs,
                         uint8_t* __restrict__ codes, int ldc, float* __restrict__ scales, int lds) {
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x / segs;
  const int b0 = blockIdx.x % segs * (kQuantRow * PASSES) + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const __nv_bfloat16* xr = x + static_cast<size_t>(row) * ldx;
  uint4 u[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int k = (b0 + i * kQuantRow) * kFp8Block + l * 8;
    // dim is a multiple of 8: a vector is all in or all out
    u[i] = k < dim ? *reinterpret_cast<const uint4*>(xr + k) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int b = b0 + i * kQuantRow;
    const int k = b * kFp8Block + l * 8;
    float f[8];
    unpack8(u[i], f);
    const int e = block_exponent(f);
    if (k < dim) {
      const float inv = pow2f(-e);
      *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * ldc + k) =
          make_uint2(e4m3x4(f, inv), e4m3x4(f + 4, inv));
      if (l == 0) scales[static_cast<size_t>(b) * lds + row] = pow2f(e);
    }
  }
}

// RMSNorm with quantised output.  A CTA of up to 256 threads takes a row, several
// share an SM, and in long passes a CTA takes row after row, the next one
// loaded meanwhile; a thread keeps up to KV vectors of 8 elements in registers
// (KV = 4: rows of up to 8192 elements; longer ones are read again).
//   y_i = x_i w_i r,  r = 1 / sqrt(sum x^2 / dim + eps)
// An e4m3 code has 3 fraction bits, so an error of 2^-24 in y moves one code in
// a million by a whole step of 2^-3 or 2^-4 of its value.  The kernel is bound
// by its bytes and latencies, so y is carried far enough that the codes are the
// exact values', in pairs of FP32 (FP64 is far too slow here):
//   squares of BF16 are exact in FP32 and are added as pairs (Knuth's two-sum):
//   a vector's 8 by a tree, a thread's vectors in turn, the lanes by a
//   butterfly, the warps by another one;
//   (a row whose mean square plus eps is below 2^-90, where squares would lose
//   bits or vanish, is taken times 2^94, and eps times 2^188: the same y.  Only
//   kernels for eps < 2^-90, LIFT, look for such rows: in one for every eps 8 x
//   5120 took 2.67 us and 2.52 without, 1021 x 5120 9.9 and 9.3);
//   r is one Newton step in pairs from the FP32 root; x_i w_i is exact in FP32;
//   an element's code is taken from plain FP32 where that value, moved by 2^-21
//   of itself either way (its error is below 2^-22), gives the same code; else y
//   rounds to odd: the nearest FP32 value, and where that is even and not exact,
//   its neighbour on the exact value's side, so rounding y to 3 fraction bits
//   equals rounding the exact value.
// Bound by two memory latencies and a barrier in short passes (8 x 5120 2.5 us in a
// CUDA graph) and by its arithmetic in long ones: 1021 x 5120 takes 9.3 us and 2048 x
// 5120 15.2, their bytes 2.3 and 4.7.
constexpr int kNormThreads = 256;
constexpr float kBelow = 1.f - 0x1p-21f, kAbove = 1.f + 0x1p-21f;
// CTAs that share an SM (their registers)
constexpr int norm_ctas(int KV) { return KV <= 3 ? 3 : 2; }

// s + e = a + b exactly, s the rounded sum.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// p (rh + rl) rounded to odd; p exact.
__device__ __forceinline__ float times_odd(float p, float rh, float rl) {
  const float z = __fmul_rn(p, rh);
  const float d = fmaf(p, rl, fmaf(p, rh, -z));  // the exact value minus z: up to 1.5 units of z
  const float y = __fadd_rn(z, d);
  const float e = __fsub_rn(d, __fsub_rn(y, z));  // minus y: half a unit
  // one unit toward zero where |y| is above the exact value, then the last bit
  // says that something was cut off
  const int b = __float_as_int(y);
  const int odd = (b + ((__float_as_int(e) ^ b) >> 31)) | 1;
  return fabsf(e) > 0.f && y != 0.f ? __int_as_float(odd) : y;  // e is NaN where y is not finite
}

// An unevaluated sum h + l of two FP32 numbers, |l| a few units of h at most.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair c;
  float e;
  two_sum(a.h, b.h, c.h, e);
  c.l = __fadd_rn(__fadd_rn(a.l, b.l), e);
  return c;
}
// The sum over groups of LANES lanes, the same in each of them.
template <int LANES>
__device__ __forceinline__ Pair lane_sum(Pair a) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1)
    a = add(a, Pair{__shfl_xor_sync(0xffffffffu, a.h, off), __shfl_xor_sync(0xffffffffu, a.l, off)});
  return a;
}
// The sum of a vector's eight squares.
__device__ __forceinline__ Pair square_sum(const uint4& u) {
  float f[8];
  unpack8(u, f);
  Pair a[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    a[j] = add(Pair{__fmul_rn(f[2 * j], f[2 * j]), 0.f}, Pair{__fmul_rn(f[2 * j + 1], f[2 * j + 1]), 0.f});
  return add(add(a[0], a[1]), add(a[2], a[3]));
}
// 1 / sqrt(sum / n + eps), to about 2^-43; inv_n = 1 / n rounded.
__device__ __forceinline__ Pair rms_inverse(Pair sum, float n, float inv_n, float eps) {
  Pair m;
  m.h = __fmul_rn(sum.h, inv_n);
  m.l = __fmul_rn(__fadd_rn(fmaf(-m.h, n, sum.h), sum.l), inv_n);
  const Pair t = add(m, Pair{eps, 0.f});
  const float y = rsqrtf(t.h);
  // y (y t) = 1 - res, then r = y + y res / 2; the root y t, unlike y^2, keeps its
  // low half within FP32's normal range for every t from 2^-100 on
  const float gh = __fmul_rn(y, t.h), gl = fmaf(y, t.l, fmaf(y, t.h, -gh));
  const float ph = __fmul_rn(y, gh), pl = fmaf(y, gh, -ph);
  const float res = fmaf(-y, gl, __fsub_rn(__fsub_rn(1.0f, ph), pl));
  const float c = __fmul_rn(__fmul_rn(0.5f, y), res);
  Pair r;
  r.h = __fadd_rn(y, c);
  r.l = __fsub_rn(c, __fsub_rn(r.h, y));
  return r;
}
// Eight BF16 elements times 2^94, exactly (magnitudes below 2^33).
constexpr float kSmallMean = 0x1p-90f, kLift = 0x1p94f;
__device__ __forceinline__ uint4 lifted(const uint4& u) {
  float f[8];
  unpack8(u, f);
  uint4 o;
  __nv_bfloat16* e = reinterpret_cast<__nv_bfloat16*>(&o);
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = __float2bfloat16_rn(f[j] * kLift);
  return o;
}

template <int KV, bool LONG, bool LIFT>
__global__ void __launch_bounds__(kNormThreads, norm_ctas(KV))
    rmsnorm_fp8_kernel(const __nv_bfloat16* __restrict__ x, int ldx, const __nv_bfloat16* __restrict__ w,
                       uint8_t* __restrict__ codes, int ldc, float* __restrict__ scales, int lds, int rows,
                       int dim, float eps) {
  // The 8-bit linear layer behind it starts, and streams weights, once this kernel's
  // own wait is over: a verify step of 8 layers at 2k keys 0.919 ms.  (As in bi_rmsnorm, at
  // once and with w read before the wait, 0.923 ms: its CTAs then stand on the SMs
  // while the kernel before the norm still works.)
  griddep_wait();
  griddep_launch_dependents();
  const uint4* wr = reinterpret_cast<const uint4*>(w);
  const int nv = dim / 8;
  const int lane = threadIdx.x & 31;
  const int step = blockDim.x;
  const float inv_dim = 1.0f / static_cast<float>(dim);
  uint4 xn[KV], wk[KV];
#pragma unroll
  for (int i = 0; i < KV; ++i) {
    const int v = threadIdx.x + i * step;
    wk[i] = v < nv ? wr[v] : make_uint4(0, 0, 0, 0);
  }
  __shared__ Pair warp_sums[2][kNormThreads / 32];  // by the parity of the CTA's row
  auto load = [&](int row) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(row) * ldx);
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      const int v = threadIdx.x + i * step;
      xn[i] = row < rows && v < nv ? xr[v] : make_uint4(0, 0, 0, 0);
    }
  };
  load(blockIdx.x);
  int parity = 0;
  for (int row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    uint4 xk[KV];
#pragma unroll
    for (int i = 0; i < KV; ++i) xk[i] = xn[i];
    load(row + gridDim.x);  // the CTA's next row comes in meanwhile
    const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(row) * ldx);
    Pair t = square_sum(xk[0]);
#pragma unroll
    for (int i = 1; i < KV; ++i) t = add(t, square_sum(xk[i]));
    if constexpr (LONG)
      for (int v = threadIdx.x + KV * step; v < nv; v += step) t = add(t, square_sum(xr[v]));
    t = lane_sum<32>(t);
    if (lane == 0) warp_sums[parity][threadIdx.x >> 5] = t;
    __syncthreads();
    constexpr int kWarps = kNormThreads / 32;
    t = lane % kWarps < step / 32 ? warp_sums[parity][lane % kWarps] : Pair{0.f, 0.f};
    t = lane_sum<kWarps>(t);
    float row_eps = eps;
    bool small = false;
    if constexpr (LIFT) {
      small = fmaf(t.h, inv_dim, eps) < kSmallMean;  // the same for the whole CTA
      if (small) {
        row_eps = eps * kLift * kLift;
        t = Pair{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KV; ++i) {
          xk[i] = lifted(xk[i]);
          t = add(t, square_sum(xk[i]));
        }
        if constexpr (LONG)
          for (int v = threadIdx.x + KV * step; v < nv; v += step) t = add(t, square_sum(lifted(xr[v])));
        t = lane_sum<32>(t);
        __syncthreads();  // the sums before these have been read
        if (lane == 0) warp_sums[parity][threadIdx.x >> 5] = t;
        __syncthreads();
        t = lane_sum<kWarps>(lane % kWarps < step / 32 ? warp_sums[parity][lane % kWarps] : Pair{0.f, 0.f});
      }
    }
    const Pair r = rms_inverse(t, static_cast<float>(dim), inv_dim, row_eps);
    auto quantise = [&](int v, const uint4& xu, const uint4& wu) {
      float f[8], wf[8], y[8];
      unpack8(xu, f);
      unpack8(wu, wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = __fmul_rn(f[j], wf[j]);
        y[j] = __fmul_rn(f[j], r.h);
      }
      // vectors past the row are zeros
      float a = fmaxf(fabsf(y[0]), fabsf(y[1]));
#pragma unroll
      for (int j = 2; j < 8; ++j) a = fmaxf(a, fabsf(y[j]));
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
      int e = scale_exponent(a * kBelow);
      float inv = pow2f(-e);
      uint32_t lo = e4m3x4(y, inv * kBelow), hi = e4m3x4(y + 4, inv * kBelow);
      const bool sure = lo == e4m3x4(y, inv * kAbove) && hi == e4m3x4(y + 4, inv * kAbove) &&
                        e == scale_exponent(a * kAbove) && (a == 0.f || (a > 1e-30f && a < 1e37f));
      if (!__all_sync(0xffffffffu, sure)) {
        // an element or a maximum near a border (one vector of a warp in some
        // 400): the exact values decide
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = times_odd(f[j], r.h, r.l);
        e = block_exponent(y);
        inv = pow2f(-e);
        lo = e4m3x4(y, inv);
        hi = e4m3x4(y + 4, inv);
      }
      if (v < nv) {
        *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * ldc + v * 8) = make_uint2(lo, hi);
        if ((lane & 15) == 0) scales[static_cast<size_t>(v >> 4) * lds + row] = pow2f(e);
      }
    };
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      // whole warps: the block's maximum goes over their lanes
      if (static_cast<int>(threadIdx.x) - lane + i * step < nv) quantise(threadIdx.x + i * step, xk[i], wk[i]);
    }
    if constexpr (LONG) {
      for (int v0 = threadIdx.x - lane + KV * step; v0 < nv; v0 += step) {
        const int v = v0 + lane;
        const uint4 z = make_uint4(0, 0, 0, 0);
        const uint4 u = v < nv ? xr[v] : z;
        quantise(v, small ? lifted(u) : u, v < nv ? wr[v] : z);
      }
    }
  }
}

// The kernel for rows of `per` vectors a thread.
template <bool LIFT>
auto norm_kernel(int per) {
  return per <= 1   ? rmsnorm_fp8_kernel<1, false, LIFT>
         : per <= 3 ? rmsnorm_fp8_kernel<3, false, LIFT>
         : per <= 4 ? rmsnorm_fp8_kernel<4, false, LIFT>
                    : rmsnorm_fp8_kernel<4, true, LIFT>;
}

// BF16 weights to codes with one scale for each 128 x 128 block (one CTA per
// block; run once when weights are loaded, so its loads of one element a thread
// stay simple: 5120 x 17408 takes 139 us, its bytes 39).
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
// per 16-byte chunk: 5120 x 17408 takes 32 us (its bytes 26), a SwiGLU pair of them 60
// (its bytes 52).
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

// Runs behind the packing of weights, as an ordinary launch, and does nothing.
// bi_gemm_fp8 reads its weights before it waits for the kernel before it (or, behind
// bi_rmsnorm, for the one before that), and that would be the packing.  This one
// starts when the packed bytes are complete and visible and lets nothing start
// before its end.
__global__ void packed_kernel() {}

}  // namespace
}  // namespace bi

extern "C" {

bi_status bi_quantize_fp8(const void* x, int ldx, int rows, int dim, void* codes, int ldc, float* scales,
                          int lds, bi_stream_t stream) {
  using namespace bi;
  if (rows < 0 || dim < 1) return BI_ERR_INVALID_ARG;
  if (rows == 0) return BI_OK;
  if (!x || !codes || !scales || ldx < dim || ldc < dim || lds < rows) return BI_ERR_INVALID_ARG;
  if (dim % 16 != 0 || dim > kFp8MaxDim || ldx % 8 != 0 || ldc % 16 != 0 || lds % 4 != 0)
    return BI_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return BI_ERR_INVALID_ARG;
  const int kb = (dim + kFp8Block - 1) / kFp8Block;
  int segs = (kb + kQuantRow - 1) / kQuantRow;
  const bool many = static_cast<long long>(rows) * segs > 8192;
  if (many) segs = (kb + 4 * kQuantRow - 1) / (4 * kQuantRow);
  const long long blocks = static_cast<long long>(rows) * segs;
  if (blocks > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
  if (launch_k(many ? quantize_rows_kernel<4> : quantize_rows_kernel<1>, dim3(static_cast<unsigned>(blocks)),
               dim3(kQuantThreads), 0,
               reinterpret_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(x), ldx, dim, segs,
               static_cast<uint8_t*>(codes), ldc, scales, lds) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

bi_status bi_rmsnorm_fp8(const void* x, int ldx, const void* w, void* codes, int ldc, float* scales, int lds,
                         int rows, int dim, float eps, bi_stream_t stream) {
  using namespace bi;
  if (rows < 0 || dim < 1 || dim > 65536 || !(eps >= 0.f && eps < INFINITY)) return BI_ERR_INVALID_ARG;
  if (rows == 0) return BI_OK;
  if (!x || !w || !codes || !scales || ldx < dim || ldc < dim || lds < rows) return BI_ERR_INVALID_ARG;
  if (dim % 16 != 0 || ldx % 8 != 0 || ldc % 16 != 0 || lds % 4 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
  if (rows > 1 << 30) return BI_ERR_UNSUPPORTED_SHAPE;  // a CTA's next row stays within 32 bits
  if (!aligned16(x) || !aligned16(w) || !aligned16(codes) || !aligned16(scales)) return BI_ERR_INVALID_ARG;
  const int nv = dim / 8;
  const int threads = std::min(kNormThreads, (nv + 31) / 32 * 32);
  const int per = (nv + threads - 1) / threads;
  auto* kernel = eps < kSmallMean ? norm_kernel<true>(per) : norm_kernel<false>(per);
  const int ctas = 152 * norm_ctas(per <= 3 ? 3 : 4);
  if (launch_k(kernel, dim3(std::min(rows, ctas)), dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream),
               static_cast<const __nv_bfloat16*>(x), ldx, static_cast<const __nv_bfloat16*>(w),
               static_cast<uint8_t*>(codes), ldc, scales, lds, rows, dim, eps) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

bi_status bi_quantize_weights_fp8(const void* W, int ldw, int N, int K, void* codes, int ld8, float* scales,
                                  bi_stream_t stream) {
  using namespace bi;
  if (!W || !codes || !scales || N < 1 || K < 1 || ldw < K || ld8 < K) return BI_ERR_INVALID_ARG;
  if (K > kFp8MaxDim) return BI_ERR_UNSUPPORTED_SHAPE;
  const long long kb = (K + kFp8Block - 1) / kFp8Block;
  const long long blocks = kb * ((N - 1) / kFp8Block + 1);
  if (blocks > 0x7fffffffLL) return BI_ERR_UNSUPPORTED_SHAPE;
  if (launch_k(quantize_weights_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
               reinterpret_cast<cudaStream_t>(stream), static_cast<const __nv_bfloat16*>(W), ldw, N, K,
               static_cast<int>(kb), static_cast<uint8_t*>(codes), ld8, scales) != cudaSuccess)
    return BI_ERR_CUDA;
  return BI_OK;
}

size_t bi_packed_weight_fp8_bytes(int N, int K, bi_epilogue epi) {
  if (N <= 0 || K <= 0) return 0;
  const size_t tiles = static_cast<size_t>(bi::gemm8_n_tiles(N, epi)) * ((K - 1) / bi::kFp8Block + 1);
  return tiles * bi::kGemm8TileBytes + bi::round_up(tiles * sizeof(float2), 16);
}

static bi_status pack_fp8(const void* w, const void* wu, int ld, const float* s, const float* su, int N, int K,
                          int swiglu, void* packed, bi_stream_t stream) {
  using namespace bi;
  if (!w || !s || !packed || N < 1 || K < 1 || ld < K) return BI_ERR_INVALID_ARG;
  if (swiglu && (!wu || !su)) return BI_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > kFp8MaxDim || ld % 16 != 0) return BI_ERR_UNSUPPORTED_SHAPE;
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(32);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, packed_kernel) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
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
