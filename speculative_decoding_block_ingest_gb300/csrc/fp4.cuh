// fp4.cuh -- the element types of a packed cache: e2m1 codes (0, .5, 1, 1.5, 2,
// 3, 4, 6 and a sign; two a byte, the even element in the low half) and e4m3
// scales, one for 16 elements of a head row.
//
// A code times a scale has at most 6 significant bits and lies between 2^-10
// and 2688: the products below are exact in f16.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace dfl {

constexpr uint32_t kScaleNaN = 0x7F;

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return reinterpret_cast<const __half2&>(x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return reinterpret_cast<const uint32_t&>(x); }

// The nearest codes (ties to even, at most 6) of eight values, in order.
__device__ __forceinline__ uint32_t e2m1_of8(const float* v) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// Eight codes as f16 pairs, in order.
__device__ __forceinline__ void e2m1_to8(uint32_t w, uint32_t* h) {
  asm("{\n.reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// The nearest scales (ties to even, at most 448; NaN for NaN) of two values:
// a's in the low byte.
__device__ __forceinline__ uint32_t e4m3_of2(float a, float b) {
  uint16_t w;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(w) : "f"(a), "f"(b));
  return w;
}
// Two scales as f16, the low byte's first.
__device__ __forceinline__ __half2 e4m3_to2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return as_half2(h);
}
__device__ __forceinline__ float e4m3_to1(uint32_t w) { return __low2float(e4m3_to2(w & 0xFF)); }

}  // namespace dfl
