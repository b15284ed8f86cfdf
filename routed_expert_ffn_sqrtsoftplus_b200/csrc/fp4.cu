// Microscaled 4-bit floating point: quantisation and its inverse.
//
//   MXFP4  E2M1 elements, one E8M0 scale per 32: scale 2^(floor(log2 amax) - 2), clamped to
//          E8M0's range (OCP MX v1.0; an all-zero block has code 0)
//   NVFP4  E2M1 elements, one E4M3 scale per 16: sf = E4M3 nearest to amax / (6 ts), at most
//          448, with ts the tensor's own scale (1 where there is none); an element stands for
//          e2m1 * d, d = sf * ts rounded once to 32 bits. A block whose sf rounds to 0 is 0.
//   Elements are the nearest E2M1, ties to the even code, at most 6 in magnitude. A block that
//   holds NaN or infinity gets the scale format's NaN, so that it reads back as NaN.
//
// Every decision is the exact one: MXFP4 divides by a power of two; for NVFP4 a quotient that
// comes near a border of the grid is decided by the sign of |x| - border * d in one fused
// multiply-add, which rounds to zero only what is zero.
//
// Bound by HBM: 2 (or 4) bytes in and 0.5 + 1/16 (or 1/32) out per value. A thread takes 16
// consecutive values (an NVFP4 block, or half an MXFP4 block whose other half is the
// neighbouring lane's), so codes leave as 8-byte stores that adjoin across the warp.
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRun = 16;  // values per thread

template <typename T>
__device__ __forceinline__ void load16(const T* p, bool vec, float (&v)[kRun]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, bool vec, float (&v)[kRun]) {
  if (vec) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + q);
      v[4 * q] = f.x;
      v[4 * q + 1] = f.y;
      v[4 * q + 2] = f.z;
      v[4 * q + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = __ldg(p + i);
  }
}
template <typename T, typename T2>
__device__ __forceinline__ void load16_half(const T* p, bool vec, float (&v)[kRun], float2 (*to2)(T2),
                                            float (*to1)(T)) {
  if (vec) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + q);
      const T2* h = reinterpret_cast<const T2*>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = to2(h[i]);
        v[8 * q + 2 * i] = f.x;
        v[8 * q + 2 * i + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = to1(p[i]);
  }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, bool vec, float (&v)[kRun]) {
  load16_half<__nv_bfloat16, __nv_bfloat162>(
      p, vec, v, [](__nv_bfloat162 h) { return __bfloat1622float2(h); },
      [](__nv_bfloat16 h) { return __bfloat162float(h); });
}
template <>
__device__ __forceinline__ void load16<__half>(const __half* p, bool vec, float (&v)[kRun]) {
  load16_half<__half, __half2>(
      p, vec, v, [](__half2 h) { return __half22float2(h); }, [](__half h) { return __half2float(h); });
}

// E4M3 value of a non-negative code (0 .. 126).
__device__ __forceinline__ float e4m3_value(int code) {
  const int e = code >> 3, m = code & 7;
  return e == 0 ? static_cast<float>(m) * 0.001953125f
                : __uint_as_float(static_cast<uint32_t>(e + 120) << 23 | static_cast<uint32_t>(m) << 20);
}

// The E4M3 code nearest to amax / (6 ts), ties to even, at most 126 (448).
__device__ __forceinline__ int e4m3_scale(float amax, float ts) {
  int c = static_cast<int>(__nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f * ts), __NV_SATFINITE, __NV_E4M3)) & 0x7F;
  // the quotient was rounded: look at the borders on both sides, 6 * midpoint * ts, whose first
  // product is exact in 32 bits
  if (c < 126) {
    const float mid = 0.5f * (e4m3_value(c) + e4m3_value(c + 1));
    const float s = fmaf(-6.0f * mid, ts, amax);
    if (s > 0.f || (s == 0.f && (c & 1))) return c + 1;
  }
  if (c > 0) {
    const float mid = 0.5f * (e4m3_value(c) + e4m3_value(c - 1));
    const float s = fmaf(-6.0f * mid, ts, amax);
    if (s < 0.f || (s == 0.f && (c & 1))) return c - 1;
  }
  return c;
}

// E2M1 magnitude code of a against the element unit d, decided exactly.
__device__ __forceinline__ uint32_t e2m1_exact(float a, float d) {
  return (fmaf(-0.25f, d, a) > 0.f) + (fmaf(-0.75f, d, a) >= 0.f) + (fmaf(-1.25f, d, a) > 0.f) +
         (fmaf(-1.75f, d, a) >= 0.f) + (fmaf(-2.5f, d, a) > 0.f) + (fmaf(-3.5f, d, a) >= 0.f) +
         (fmaf(-5.0f, d, a) > 0.f);
}

// Whether q, rounded from an exact quotient, may sit on the other side of a border of the E2M1
// grid: every border has at most three significant bits, so the low 21 bits of its float are 0.
// (A quotient of 0 comes from a value of 0, or from one far below the first border.)
__device__ __forceinline__ bool near_border(float q) {
  return ((__float_as_uint(q) + 2u) & 0x1FFFFFu) <= 4u && q != 0.f;
}

template <typename T, bool kNv>
__global__ void __launch_bounds__(256)
    quantize_fp4_kernel(const T* __restrict__ src, int64_t runs, int runs_per_row, int64_t row_stride, int vec,
                        const float* __restrict__ tensor_scale, uint2* __restrict__ codes,
                        uint8_t* __restrict__ scales, int64_t scale_stride) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  // cols % 32 == 0: an even number of runs, so a lane and its neighbour are in range together
  if (i >= runs) return;
  const int64_t row = i / runs_per_row;
  const int run = static_cast<int>(i - row * runs_per_row);
  float v[kRun];
  load16<T>(src + row * row_stride + static_cast<int64_t>(run) * kRun, vec != 0, v);
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    const float a = fabsf(v[j]);
    finite = finite && a < INFINITY;
    amax = fmaxf(amax, a);
  }
  uint32_t w[2] = {0u, 0u};
  if constexpr (!kNv) {
    const unsigned pair = 3u << ((threadIdx.x & 31) & ~1);
    amax = fmaxf(amax, __shfl_xor_sync(pair, amax, 1));
    finite = __shfl_xor_sync(pair, finite ? 1 : 0, 1) != 0 && finite;
    int code;
    float inv;
    mx_scale(amax, 2, code, inv);
    if (!finite) {
      code = 0xFF;
      inv = 0.f;
    }
    // a power of two: the products are exact, and the conversion rounds them as the format asks
#pragma unroll
    for (int j = 0; j < kRun / 2; ++j) {
      const float2 f = finite ? make_float2(v[2 * j] * inv, v[2 * j + 1] * inv) : make_float2(0.f, 0.f);
      w[j / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * (j % 4));
    }
    if ((run & 1) == 0) scales[row * scale_stride + run / 2] = static_cast<uint8_t>(code);
  } else {
    const float ts = tensor_scale ? __ldg(tensor_scale) : 1.0f;
    const int code = finite ? e4m3_scale(amax, ts) : 0x7F;
    const float d = finite ? e4m3_value(code) * ts : 0.f;
    if (d > 0.f) {
      const float inv = __fdiv_rn(1.0f, d);
      bool near = false;
#pragma unroll
      for (int j = 0; j < kRun / 2; ++j) {
        const float2 f = make_float2(v[2 * j] * inv, v[2 * j + 1] * inv);
        near = near || near_border(f.x) || near_border(f.y);
        w[j / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * (j % 4));
      }
      // a unit that is a power of two leaves the quotients exact
      if (near && (__float_as_uint(d) & 0x7FFFFFu) != 0u) {
        w[0] = w[1] = 0u;
#pragma unroll
        for (int j = 0; j < kRun; ++j)
          w[j / 8] |= (e2m1_exact(fabsf(v[j]), d) | (signbit(v[j]) ? 8u : 0u)) << (4 * (j % 8));
      }
    }
    scales[row * scale_stride + run] = static_cast<uint8_t>(code);
  }
  codes[i] = make_uint2(w[0], w[1]);
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[kRun], bool vec);
template <>
__device__ __forceinline__ void store16<float>(float* p, const float (&v)[kRun], bool vec) {
  if (vec) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      reinterpret_cast<float4*>(p)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) p[i] = v[i];
  }
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[kRun], bool vec) {
  __nv_bfloat162 h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  if (vec) {
    reinterpret_cast<uint4*>(p)[0] = *reinterpret_cast<uint4*>(h);
    reinterpret_cast<uint4*>(p)[1] = *reinterpret_cast<uint4*>(h + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[2 * i] = h[i].x;
      p[2 * i + 1] = h[i].y;
    }
  }
}
template <>
__device__ __forceinline__ void store16<__half>(__half* p, const float (&v)[kRun], bool vec) {
  __half2 h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  if (vec) {
    reinterpret_cast<uint4*>(p)[0] = *reinterpret_cast<uint4*>(h);
    reinterpret_cast<uint4*>(p)[1] = *reinterpret_cast<uint4*>(h + 4);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[2 * i] = h[i].x;
      p[2 * i + 1] = h[i].y;
    }
  }
}

template <typename T, bool kNv>
__global__ void __launch_bounds__(256)
    dequantize_fp4_kernel(const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t runs,
                          int runs_per_row, int64_t scale_stride, const float* __restrict__ tensor_scale, int vec,
                          T* __restrict__ dst) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= runs) return;
  const int64_t row = i / runs_per_row;
  const int run = static_cast<int>(i - row * runs_per_row);
  const uint2 c = __ldg(codes + i);
  const uint32_t s = __ldg(scales + row * scale_stride + (kNv ? run : run / 2));
  float d;
  if constexpr (kNv) {
    // the sign bit of a scale is not used by the format
    d = (s & 0x7Fu) == 0x7Fu ? __int_as_float(0x7fc00000) : e4m3_value(static_cast<int>(s & 0x7Fu));
    if (tensor_scale) d *= __ldg(tensor_scale);
  } else {
    d = s == 0xFFu ? __int_as_float(0x7fc00000) : __uint_as_float(s == 0u ? 1u << 22 : s << 23);
  }
  float v[kRun];
#pragma unroll
  for (int j = 0; j < kRun / 2; ++j) {
    const uint32_t w = j < 4 ? c.x : c.y;
    const __half2_raw h =
        __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((w >> (8 * (j % 4))) & 0xFFu), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = f.x * d;
    v[2 * j + 1] = f.y * d;
  }
  store16<T>(dst + i * kRun, v, vec != 0);
}

// Scale rows into rows of another stride, 4 bytes of the destination per thread.
__global__ void __launch_bounds__(256)
    pad_scales_kernel(const uint8_t* __restrict__ src, int64_t words, int words_per_row, int cols,
                      uint32_t* __restrict__ dst) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= words) return;
  const int64_t row = i / words_per_row;
  const int c = static_cast<int>(i - row * words_per_row) * 4;
  const uint8_t* p = src + row * cols + c;
  uint32_t w = 0u;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (c + b < cols) w |= static_cast<uint32_t>(__ldg(p + b)) << (8 * b);
  dst[i] = w;
}

template <typename T, bool kNv>
cudaError_t quantize_t(const void* src, int64_t rows, int cols, int64_t row_stride, const float* ts, uint8_t* codes,
                       uint8_t* scales, int64_t scale_stride, cudaStream_t s) {
  const int rpr = cols / kRun;
  const int64_t runs = rows * rpr;
  const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && (row_stride * sizeof(T)) % 16 == 0;
  quantize_fp4_kernel<T, kNv><<<static_cast<unsigned>((runs + 255) / 256), 256, 0, s>>>(
      static_cast<const T*>(src), runs, rpr, row_stride, vec ? 1 : 0, ts, reinterpret_cast<uint2*>(codes), scales,
      scale_stride);
  return cudaGetLastError();
}

template <typename T, bool kNv>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, int64_t scale_stride,
                         const float* ts, void* dst, cudaStream_t s) {
  const int rpr = cols / kRun;
  const int64_t runs = rows * rpr;
  const bool vec = reinterpret_cast<uintptr_t>(dst) % 16 == 0;
  dequantize_fp4_kernel<T, kNv><<<static_cast<unsigned>((runs + 255) / 256), 256, 0, s>>>(
      reinterpret_cast<const uint2*>(codes), scales, runs, rpr, scale_stride, ts, vec ? 1 : 0, static_cast<T*>(dst));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_fp4(int format, const void* src, int dtype, int64_t rows, int cols, int64_t row_stride,
                                const float* tensor_scale, uint8_t* codes, uint8_t* scales, int64_t scale_stride,
                                cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
#define MOE_QUANT_CASE(V, T)                                                                                       \
  if (dtype == V)                                                                                                  \
    return format == kFp4Nv                                                                                        \
               ? quantize_t<T, true>(src, rows, cols, row_stride, tensor_scale, codes, scales, scale_stride, s)    \
               : quantize_t<T, false>(src, rows, cols, row_stride, tensor_scale, codes, scales, scale_stride, s);
  MOE_QUANT_CASE(kValBf16, __nv_bfloat16)
  MOE_QUANT_CASE(kValFp16, __half)
  MOE_QUANT_CASE(kValFp32, float)
#undef MOE_QUANT_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_pad_scales(const uint8_t* src, int64_t rows, int cols, uint8_t* dst, int64_t dst_stride,
                              cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int wpr = static_cast<int>(dst_stride / 4);
  const int64_t words = rows * wpr;
  pad_scales_kernel<<<static_cast<unsigned>((words + 255) / 256), 256, 0, s>>>(src, words, wpr, cols,
                                                                              reinterpret_cast<uint32_t*>(dst));
  return cudaGetLastError();
}

cudaError_t launch_dequantize_fp4(int format, const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols,
                                  int64_t scale_stride, const float* tensor_scale, void* dst, int dtype,
                                  cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
#define MOE_DEQUANT_CASE(V, T)                                                                                     \
  if (dtype == V)                                                                                                  \
    return format == kFp4Nv ? dequantize_t<T, true>(codes, scales, rows, cols, scale_stride, tensor_scale, dst, s) \
                            : dequantize_t<T, false>(codes, scales, rows, cols, scale_stride, tensor_scale, dst, s);
  MOE_DEQUANT_CASE(kValBf16, __nv_bfloat16)
  MOE_DEQUANT_CASE(kValFp16, __half)
  MOE_DEQUANT_CASE(kValFp32, float)
#undef MOE_DEQUANT_CASE
  return cudaErrorInvalidValue;
}

}  // namespace moe
