// Conversions into the cache records' element types, shared by the kernels that
// write records (internal header).
#pragma once
#include <stdint.h>

namespace csa2 {

// Eight floats -> four bytes of E2M1 pairs; byte i = code(v[2i+1]) << 4 | code(v[2i]).
__device__ __forceinline__ uint32_t cvt_e2m1x8(float v0, float v1, float v2, float v3, float v4, float v5,
                                               float v6, float v7) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "f"(v4), "f"(v5), "f"(v6), "f"(v7));
  return r;
}

__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return (uint32_t)r;
}

// fp64 -> bf16 bits, one rounding (nearest-even), for finite values of bf16 range.
__device__ __forceinline__ uint32_t bf16_from_f64(double v) {
  unsigned long long u = (unsigned long long)__double_as_longlong(v);
  uint32_t sign = (uint32_t)(u >> 63) << 15;
  unsigned long long a = u & 0x7FFFFFFFFFFFFFFFull;
  if (a == 0) return sign;
  int ex = (int)(a >> 52) - 1023;                 // unbiased exponent of a normal double
  uint32_t bits;
  if (ex >= -126) {
    // keep 7 of the 52 fraction bits: round away 45 bits, nearest-even
    unsigned long long r = a + ((1ull << 44) - 1) + ((a >> 45) & 1ull);
    r >>= 45;                                     // (exponent_d << 7) | frac7, may carry
    int e_bf = (int)(r >> 7) - 1023 + 127;
    bits = ((uint32_t)e_bf << 7) | (uint32_t)(r & 0x7F);
  } else {
    // bf16 subnormal: multiple of 2^-133; |v| < 2^-126 so the count is <= 128
    double m = fabs(v) * 0x1p133;                 // exact power-of-two scaling
    bits = (uint32_t)__double2ull_rn(m);          // nearest-even to an integer
  }
  return sign | bits;
}

// smallest e with lim * 2^e >= amax (amax > 0), for lim = 1.5 * 2^p, 1.75 * 2^p
__device__ __forceinline__ int pow2_exp_fp4(float amax) {   // lim = 6 = 1.5 * 2^2
  int ex;
  frexpf(amax, &ex);                     // amax in [2^(ex-1), 2^ex)
  int e0 = ex - 1;
  int e = (amax <= ldexpf(6.0f, e0 - 2)) ? e0 - 2 : e0 - 1;
  return max(-127, min(127, e));
}
__device__ __forceinline__ int pow2_exp_fp8(float amax) {   // lim = 448 = 1.75 * 2^8
  int ex;
  frexpf(amax, &ex);
  int e0 = ex - 1;
  int e = (amax <= ldexpf(448.0f, e0 - 8)) ? e0 - 8 : e0 - 7;
  return max(-127, min(127, e));
}

}  // namespace csa2
