// Operand helpers shared by the attention kernels (internal header).
#pragma once
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"

namespace csa2 {

// byte offset of 16-B chunk `ch` (0..7) in row r of a 128B-swizzled 1024-B atom
__device__ __forceinline__ uint32_t sw128(uint32_t r, uint32_t ch) { return r * 128u + ((ch ^ (r & 7u)) << 4); }

// kind::f16 instruction descriptor: bf16 x bf16 (or f16 x f16) -> f32, M=128,
// N = n (a multiple of 16), A K- or MN-major.
__host__ __device__ constexpr uint32_t idesc_m128(uint32_t a_mn_major, bool f16, uint32_t n) {
  return (1u << 4)                     // D format f32
         | ((f16 ? 0u : 1u) << 7)      // A: f16 0, bf16 1
         | ((f16 ? 0u : 1u) << 10)     // B: f16 0, bf16 1
         | (a_mn_major << 15)          // A major-ness
         | ((n >> 3) << 17)            // N / 8
         | ((128u >> 4) << 24);        // M / 16
}

// Eight E2M1 codes (channel i in nibble i of w) -> eight f16 values as four
// f16x2 words, by the hardware converter (exact: E2M1 is a subset of f16).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}

// Two E4M3 codes (low byte first) -> f16x2 bits (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return h;
}

// cos and sin of theta = pos * inv_freq (inv_freq = rope_base^(-2i/64), computed
// on the host in fp64): the product and its reduction modulo 2 pi are done in
// fp64 (pos reaches 2^20, so theta reaches ~1e6 rad), the sine and cosine of the
// reduced angle in fp32.
__device__ __forceinline__ void rope_cs(double inv_freq, int pos, float &c, float &s) {
  const double th = (double)pos * inv_freq;
  const double k = rint(th * 0.15915494309189535);            // 1 / (2 pi)
  const double r = fma(-k, 6.283185307179586, th);
  sincosf((float)r, &s, &c);
}

// Sums h + l of two fp64 numbers, |l| at most half an ulp of h (host; about 104 bits).
struct Double2 {
  double h, l;
};
inline Double2 sum2(double h, double l) {             // |l| below |h|
  const double s = h + l;
  return {s, l - (s - h)};
}
inline Double2 mul2(const Double2 &a, const Double2 &b) {
  volatile double p = a.h * b.h;                      // (rounded here, whatever the compiler contracts)
  return sum2(p, fma(a.h, b.h, -p) + (a.h * b.l + a.l * b.h));
}
inline Double2 sqrt2(const Double2 &a) {
  const double x = sqrt(a.h);
  return sum2(x, (fma(-x, x, a.h) + a.l) / (2.0 * x));
}
inline Double2 inverse2(const Double2 &a) {
  const double x = 1.0 / a.h;
  return sum2(x, (fma(-x, a.h, 1.0) - x * a.l) * x);
}

// The same angles in turns, as 64-bit fixed-point fractions: one position's
// turns modulo one in 2^-64ths, so that pos * turn (wrapping) drops whole turns
// exactly and is off by half a 2^-64th a position, 2^-31 rad at the farthest; the
// fraction (53 bits) goes to fp32 for the sine and cosine.  The powers
// rope_base^(-i/32) come from five square roots, an inverse and products, all in
// pairs of fp64 (pow's 53 bits left 2^-24 rad there, and the ulps differ between machines).
// (A host thread's last base is kept: 32 powers are a microsecond or two.)
inline void rope_turns(double rope_base, uint64_t (&turn)[kRopeDim / 2]) {
  static thread_local double base = 0.0;           // (not a base)
  static thread_local uint64_t last[kRopeDim / 2];
  if (base != rope_base) {
    Double2 step = {rope_base, 0.0};
    for (int i = 0; i < 5; i++) step = sqrt2(step);   // (kRopeDim / 2 is 2^5)
    step = inverse2(step);
    Double2 t = inverse2({6.283185307179586, 2.4492935982947064e-16});       // 1 / (2 pi)
    for (int i = 0; i < kRopeDim / 2; i++, t = mul2(t, step)) {
      // (beyond 2^53 turns a position, of a base near zero, nothing is left of the fraction)
      const bool some = fabs(t.h) < 0x1p53;
      const double h = some ? t.h - floor(t.h) : 0.0, a = floor(h * 0x1p32);
      const double rest = some ? ((h * 0x1p32 - a) + t.l * 0x1p32) * 0x1p32 : 0.0;
      last[i] = ((uint64_t)a << 32) + (uint64_t)(int64_t)rint(rest);
    }
    base = rope_base;
  }
  for (int i = 0; i < kRopeDim / 2; i++) turn[i] = last[i];
}
__device__ __forceinline__ void turn_cs(uint64_t u, float &c, float &s) {
  sincospif((float)(int64_t)u * 0x1p-63f, &s, &c);
}

}  // namespace csa2
