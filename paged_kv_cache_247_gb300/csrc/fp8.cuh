// Rows of a cache held in 8 bits.
//
// A row (one token, one KV head, D elements) is held as D e4m3 codes and one
// scale, a power of two in bfloat16: element = code * scale.  With a = max |x|
// over the row, the scale is 2^e for the smallest e >= -126 with a <= 448 2^e
// (448 is the largest e4m3 value), so x * 2^-e is exact and each element is
// rounded once, to nearest even: the same 16-bit row gives the same bits
// wherever it is written.  Nothing is lost against a scale of a / 448: e4m3 is
// a floating-point type, and the codes keep their four significant bits down
// to 2^-14 of the row's largest element.  A row with a NaN or an infinity is
// held as NaN as a whole (scale NaN, codes 0), which the attention calls can
// leave out by its scale alone where it is masked.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace pkv {

constexpr uint16_t kNanScale = 0x7fc0;  // bfloat16

// e of the row scale from the bits of a, the row's largest magnitude (finite):
// a = 1.m 2^x gives x - 8, one more where 1.m > 1.75 (the addition carries).
__device__ __forceinline__ int row_exponent(float a) {
  return max((int)((__float_as_uint(a) + 0x1fffffu) >> 23) - 127 - 8, -126);
}

// bfloat16 bits of 2^e (-126 <= e <= 127).
__device__ __forceinline__ uint16_t scale_bits(int e) { return (uint16_t)((e + 127) << 7); }

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ float scale_value(uint16_t bits) {
  return __uint_as_float((uint32_t)bits << 16);
}

// Largest pattern of |x| over eight packed 16-bit values (fp16 or bf16: the
// patterns order like the magnitudes, infinities and NaN above all).
__device__ __forceinline__ uint32_t max_magnitude(uint4 w) {
  return __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                  __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}

template <typename T>
struct Magnitude;

template <>
struct Magnitude<__half> {
  static constexpr uint32_t kInf = 0x7c00;
  static __device__ __forceinline__ float value(uint32_t bits) {
    return __half2float(__ushort_as_half((unsigned short)bits));
  }
};

template <>
struct Magnitude<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7f80;
  static __device__ __forceinline__ float value(uint32_t bits) {
    return __uint_as_float(bits << 16);
  }
};

// Four codes of the two packed pairs a, b, each element times inv.
template <typename T>
__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, float inv) {
  float2 x = Cvt<T>::to_float2(a), y = Cvt<T>::to_float2(b);
  x.x *= inv;
  x.y *= inv;
  y.x *= inv;
  y.y *= inv;
  return (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) |
         ((uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << 16);
}

// The values of two codes.
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace pkv
