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
// Every decision is the exact one: MXFP4 divides by a power of two; for NVFP4 a block with a
// quotient near a border of the grid is decided by the signs of |x| - border * d in one fused
// multiply-add each, which rounds to zero only what is zero.
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

// n / d for n < 2^31 by a multiplication (the row of a run; a division costs as much as a value's
// whole conversion).
struct FastDiv {
  uint32_t mul, shift, d;
};
FastDiv fast_div(uint32_t d) {
  FastDiv f{0, 0, d};
  while ((uint64_t(1) << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.mul) + n) >> f.shift; }

__device__ __forceinline__ float value_f32(float v) { return v; }
__device__ __forceinline__ float value_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float value_f32(__half v) { return __half2float(v); }

// 16 consecutive values as they are in memory.
template <typename T>
struct Raw {
  static constexpr int kWords = kRun * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p, bool vec) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < kWords / 4; ++q) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + q);
        w[4 * q] = u.x;
        w[4 * q + 1] = u.y;
        w[4 * q + 2] = u.z;
        w[4 * q + 3] = u.w;
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = static_cast<uint32_t>(__ldg(h + 2 * i)) | static_cast<uint32_t>(__ldg(h + 2 * i + 1)) << 16;
    }
  }
};
// The values in 32 bits and the largest magnitude among them; not finite: false. Magnitudes are compared
// as integers, in which infinity and NaN come last, two 16-bit values at a time.
__device__ __forceinline__ bool unpack(const Raw<float>& r, float (&v)[kRun], float& amax) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    m = max(m, r.w[i] & 0x7FFFFFFFu);
    v[i] = __uint_as_float(r.w[i]);
  }
  amax = __uint_as_float(m);
  return m < 0x7F800000u;
}
__device__ __forceinline__ uint32_t largest16(const uint32_t (&w)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}
__device__ __forceinline__ bool unpack(const Raw<__nv_bfloat16>& r, float (&v)[kRun], float& amax) {
  const uint32_t m = largest16(r.w);
  amax = __uint_as_float(m << 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
  return m < 0x7F80u;
}
__device__ __forceinline__ bool unpack(const Raw<__half>& r, float (&v)[kRun], float& amax) {
  const uint32_t m = largest16(r.w);
  amax = __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
  return m < 0x7C00u;
}

// E4M3 value of a non-negative code (0 .. 126).
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// The E4M3 code nearest to amax / (6 ts), ties to even, at most 126 (448); 0 where amax is, also with the ts of 0 that a
// tensor of zeros calibrates to.
__device__ __forceinline__ uint32_t e4m3_scale(float amax, float ts) {
  // far out, both by one power of two, so that neither the reciprocal nor a difference leaves the normal range
  // (where amax does, the code is 0 or 126 with or without it)
  if (ts < 0x1p-60f || ts > 0x1p60f) {
    const float by = ts < 1.0f ? 0x1p60f : 0x1p-60f;
    ts *= by;
    amax *= by;
  }
  // off by less than 2^-22: where a little less and a little more give one code, it is the right one
  const float q = amax * __frcp_rn(6.0f * ts);
  const uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(q * (1.0f - 0x1p-21f), q * (1.0f + 0x1p-21f)),
                                                 __NV_SATFINITE, __NV_E4M3);
  uint32_t c = pair & 0x7Fu;
  const uint32_t up = pair >> 8 & 0x7Fu;
  if (c != up) {
    // the border between them, 6 * midpoint * ts: the first product is exact in 32 bits, and the fused
    // multiply-add keeps the difference's sign
    const float s = fmaf(-3.0f * (e4m3_value(c) + e4m3_value(up)), ts, amax);
    if (s > 0.f || (s == 0.f && (c & 1u))) c = up;
  }
  return amax == 0.f ? 0u : c;
}

// Eight scaled values to a word of E2M1 codes, the first in the lowest nibble: nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v, float scale) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b64 s, p, q, r, t;\n\t.reg .f32 x, y;\n\t"
      "mov.b64 s, {%9, %9};\n\tmov.b64 p, {%1, %2};\n\tmov.b64 q, {%3, %4};\n\t"
      "mov.b64 r, {%5, %6};\n\tmov.b64 t, {%7, %8};\n\t"
      "mul.rn.f32x2 p, p, s;\n\tmul.rn.f32x2 q, q, s;\n\tmul.rn.f32x2 r, r, s;\n\tmul.rn.f32x2 t, t, s;\n\t"
      "mov.b64 {x, y}, p;\n\tcvt.rn.satfinite.e2m1x2.f32 a, y, x;\n\t"
      "mov.b64 {x, y}, q;\n\tcvt.rn.satfinite.e2m1x2.f32 b, y, x;\n\t"
      "mov.b64 {x, y}, r;\n\tcvt.rn.satfinite.e2m1x2.f32 c, y, x;\n\t"
      "mov.b64 {x, y}, t;\n\tcvt.rn.satfinite.e2m1x2.f32 d, y, x;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(scale));
  return r;
}

// Decides the codes in which `lo` and `hi`, neighbours on the grid, differ: value j against the border
// between them, border * d, by the sign of one fused multiply-add. The few values are read again (an
// index into registers would put them all into local memory). A low unit is raised by a power of two, as
// differences of its size would not be normal numbers.
template <typename T>
__device__ __forceinline__ uint32_t settle(uint32_t lo, uint32_t hi, const T* p, float d) {
  const float by = d < 0x1p-60f ? 0x1p60f : 1.0f;
  for (uint32_t diff = lo ^ hi; diff != 0u;) {
    const int at = (__ffs(static_cast<int>(diff)) - 1) & ~3;
    const uint32_t c = (lo >> at) & 7u;
    // (grid[c] + grid[c + 1]) / 2: 1/4 + c/2 up to 7/4, then 5/2, 7/2, 5
    const float border = c < 4u ? 0.25f + 0.5f * static_cast<float>(c) : c < 6u ? static_cast<float>(c) - 1.5f : 5.0f;
    const float s = fmaf(-border, d * by, fabsf(value_f32(p[at / 4])) * by);
    if (s > 0.f || (s == 0.f && (c & 1u))) lo += 1u << at;
    diff &= ~(0xFu << at);
  }
  return lo;
}

// Runs a thread takes, a block's width apart and loaded together: two of 16-bit values to MXFP4, which
// HBM bounds (8192 x 5120: 18.3 us against 21.9 with one); one to NVFP4, whose arithmetic bounds it (23.1
// us against 22.5 with two, but 517 x 1312 2.0 against 2.2), and of 32-bit values, for their registers.
template <typename T, bool kNv>
constexpr int kRuns = sizeof(T) == 4 || kNv ? 1 : 2;

template <typename T, bool kNv>
__global__ void __launch_bounds__(256)
    quantize_fp4_kernel(const T* __restrict__ src, uint32_t runs, FastDiv per_row, int64_t row_stride, int vec,
                        const float* __restrict__ tensor_scale, uint2* __restrict__ codes,
                        uint8_t* __restrict__ scales, int64_t scale_stride) {
  // A product's prologue, which then waits for these codes. Not beside a grid of many rounds, whose blocks
  // would find the SMs taken by those that wait.
  if (gridDim.x <= 128) let_next_kernel_start();
  const uint32_t first = blockIdx.x * (256u * kRuns<T, kNv>) + threadIdx.x;
  Raw<T> raw[kRuns<T, kNv>];
#pragma unroll
  for (int u = 0; u < kRuns<T, kNv>; ++u) {
    const uint32_t i = first + 256u * u;
    if (i < runs) {
      const uint32_t row = divide(i, per_row);
      raw[u].load(src + row * row_stride + (i - row * per_row.d) * kRun, vec != 0);
    }
  }
  const float ts = kNv && tensor_scale ? __ldg(tensor_scale) : 1.0f;
#pragma unroll
  for (int u = 0; u < kRuns<T, kNv>; ++u) {
    const uint32_t i = first + 256u * u;
    // cols % 32 == 0: an even number of runs, so that a lane and its neighbour are in range together
    if (i >= runs) return;
    const uint32_t row = divide(i, per_row);
    const uint32_t run = i - row * per_row.d;
    float v[kRun], amax;
    bool finite = unpack(raw[u], v, amax);
    uint32_t w[2] = {0u, 0u};
    if constexpr (!kNv) {
      const unsigned pair = 3u << ((threadIdx.x & 31) & ~1);
      // a block that is not finite is one as a whole: the larger magnitude, compared as an integer
      const uint32_t m = max(__float_as_uint(amax), __shfl_xor_sync(pair, __float_as_uint(amax), 1));
      finite = m < 0x7F800000u;
      int code;
      float inv;
      mx_scale(__uint_as_float(m), 2, code, inv);
      // a power of two: the products are exact, and the conversion rounds them as the format asks
      w[0] = to_e2m1x8(v, inv);
      w[1] = to_e2m1x8(v + 8, inv);
      if (!finite) {
        code = 0xFF;
        w[0] = w[1] = 0u;
      }
      if ((run & 1) == 0) scales[row * scale_stride + run / 2] = static_cast<uint8_t>(code);
    } else {
      const uint32_t code = finite ? e4m3_scale(amax, ts) : 0x7Fu;
      const float d = finite ? e4m3_value(code) * ts : 0.f;
      const uint32_t db = __float_as_uint(d);
      if (db >= 0x00800000u && db < 0x7F800000u) {  // a unit below the normal range counts as 0
        // Quotients by two reciprocals, one a little low, one a little high: where both give the same
        // codes, so does the exact quotient. (A unit that is a power of two divides exactly.)
        const bool pow2 = (db & 0x7FFFFFu) == 0u && db >= 0x01000000u && db <= 0x7E000000u;
        const float inv = pow2 ? __uint_as_float(0x7F000000u - db) : __fdividef(1.0f, d);
        const float lo = pow2 ? inv : inv * (1.0f - 0x1p-20f), hi = pow2 ? inv : inv * (1.0f + 0x1p-20f);
        // Real tensors do come near borders: a tensor scale taken from a 16-bit maximum puts many blocks'
        // units at simple fractions of their values (1.5 % of the runs of normally distributed rows).
        const T* p = src + row * row_stride + run * kRun;
        w[0] = settle(to_e2m1x8(v, lo), to_e2m1x8(v, hi), p, d);
        w[1] = settle(to_e2m1x8(v + 8, lo), to_e2m1x8(v + 8, hi), p + 8, d);
      }
      scales[row * scale_stride + run] = static_cast<uint8_t>(code);
    }
    codes[i] = make_uint2(w[0], w[1]);
  }
}

// Eight consecutive values.
__device__ __forceinline__ void store8(float* p, const float (&v)[8], bool vec) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[i];
  }
}
template <typename T2, typename T>
__device__ __forceinline__ void store8_half(T* p, const T2 (&h)[4], bool vec) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[2 * i] = h[i].x;
      p[2 * i + 1] = h[i].y;
    }
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8], bool vec) {
  __align__(16) __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  store8_half(p, h, vec);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8], bool vec) {
  __align__(16) __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
  store8_half(p, h, vec);
}

// A thread takes eight values, so that a warp's 16-byte stores adjoin, and kSteps such pieces a
// block's width apart, loaded together.
constexpr int kSteps = 4;

template <typename T, bool kNv>
__global__ void __launch_bounds__(256)
    dequantize_fp4_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint32_t pieces,
                          FastDiv per_row, int64_t scale_stride, const float* __restrict__ tensor_scale, int vec,
                          T* __restrict__ dst) {
  constexpr uint32_t kPerScale = kNv ? 2 : 4;  // pieces of a block
  const uint32_t first = blockIdx.x * (256u * kSteps) + threadIdx.x;
  uint32_t c[kSteps], sc[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const uint32_t i = first + 256u * u;
    c[u] = sc[u] = 0u;
    if (i < pieces) {
      c[u] = __ldg(codes + i);
      const uint32_t row = divide(i, per_row);
      sc[u] = __ldg(scales + row * scale_stride + (i - row * per_row.d) / kPerScale);
    }
  }
  const float ts = kNv && tensor_scale ? __ldg(tensor_scale) : 1.0f;
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const uint32_t i = first + 256u * u;
    if (i >= pieces) break;
    const uint32_t s = sc[u];
    float d;
    if constexpr (kNv) {
      // the sign bit of a scale is not used by the format
      d = (s & 0x7Fu) == 0x7Fu ? __int_as_float(0x7fc00000) : e4m3_value(s & 0x7Fu) * ts;
    } else {
      d = s == 0xFFu ? __int_as_float(0x7fc00000) : __uint_as_float(s == 0u ? 1u << 22 : s << 23);
    }
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2_raw h =
          __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((c[u] >> (8 * j)) & 0xFFu), __NV_E2M1);
      const float2 f = __half22float2(__half2(h));
      v[2 * j] = f.x * d;
      v[2 * j + 1] = f.y * d;
    }
    store8(dst + static_cast<int64_t>(i) * 8, v, vec != 0);
  }
}

// Scale rows into rows of another stride, 4 bytes of the destination per thread.
__global__ void __launch_bounds__(256)
    pad_scales_kernel(const uint8_t* __restrict__ src, int64_t src_stride, int64_t words, int words_per_row, int cols,
                      uint32_t* __restrict__ dst) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= words) return;
  const int64_t row = i / words_per_row;
  const int c = static_cast<int>(i - row * words_per_row) * 4;
  const uint8_t* p = src + row * src_stride + c;
  uint32_t w = 0u;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (c + b < cols) w |= static_cast<uint32_t>(__ldg(p + b)) << (8 * b);
  dst[i] = w;
}

template <typename T, bool kNv>
cudaError_t quantize_t(const void* src, int64_t rows, int cols, int64_t row_stride, const float* ts, uint8_t* codes,
                       uint8_t* scales, int64_t scale_stride, cudaStream_t s) {
  const uint32_t rpr = cols / kRun, runs = static_cast<uint32_t>(rows * rpr);
  const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && (row_stride * sizeof(T)) % 16 == 0;
  quantize_fp4_kernel<T, kNv><<<(runs + 256 * kRuns<T, kNv> - 1) / (256 * kRuns<T, kNv>), 256, 0, s>>>(
      static_cast<const T*>(src), runs, fast_div(rpr), row_stride, vec ? 1 : 0, ts, reinterpret_cast<uint2*>(codes), scales,
      scale_stride);
  return cudaGetLastError();
}

template <typename T, bool kNv>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, int64_t scale_stride,
                         const float* ts, void* dst, cudaStream_t s) {
  const uint32_t ppr = cols / 8, pieces = static_cast<uint32_t>(rows * ppr);
  const bool vec = reinterpret_cast<uintptr_t>(dst) % 16 == 0;
  dequantize_fp4_kernel<T, kNv><<<(pieces + 256 * kSteps - 1) / (256 * kSteps), 256, 0, s>>>(
      reinterpret_cast<const uint32_t*>(codes), scales, pieces, fast_div(ppr), scale_stride, ts, vec ? 1 : 0,
      static_cast<T*>(dst));
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

cudaError_t launch_pad_scales(const uint8_t* src, int64_t src_stride, int64_t rows, int cols, uint8_t* dst,
                              int64_t dst_stride, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int wpr = static_cast<int>(dst_stride / 4);
  const int64_t words = rows * wpr;
  pad_scales_kernel<<<static_cast<unsigned>((words + 255) / 256), 256, 0, s>>>(src, src_stride, words, wpr, cols,
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
