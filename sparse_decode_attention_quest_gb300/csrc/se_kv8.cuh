// Magnitudes and scales of bf16 values held as e4m3 codes.
#pragma once

#include "se_ptx.cuh"

namespace se {

// Larger of the magnitudes so far and a word's two; a NaN beside a number is dropped.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t x) {
  const __nv_bfloat162 a = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&m), a);
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_abs_bf16x8(uint32_t m, uint4 x) {
  return max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(m, x.x), x.y), x.z), x.w);
}

// The same with NaN above all numbers.
__device__ __forceinline__ uint32_t max_abs_nan_bf16x2(uint32_t m, uint32_t x) {
  const __nv_bfloat162 a = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&m), a);
  return *reinterpret_cast<uint32_t*>(&r) & 0x7fff7fffu;
}

// A word's infinities and NaN, by mask 0xffff each.
__device__ __forceinline__ uint32_t not_finite_bf16x2(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// The least power of two s >= 2^-100 with a <= 448 s, for the bits of a finite bf16 a >= 0: 448 is 1.75 * 2^8.
__device__ __forceinline__ float scale_for(uint32_t a) {
  const int e = (int)(a >> 7) - 127 - 8 + ((a & 0x7f) > 0x60 ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

// Four codes as numbers.
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  e4m3x4_to_f16(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

}  // namespace se
