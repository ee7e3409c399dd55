// What the quantizers share: maxima that keep a NaN, quotients of many numbers by
// one divisor, each rounded as the division itself rounds it, and the nearest
// integer of such a quotient.
//
// With y = RN(1/b), q = RN(a y), the remainder r = a - q b is exact in one FMA
// and RN(q + r y) is the correctly rounded a / b, unless b's significand is all
// ones or a step leaves the normal range (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990):
// three operations a quotient instead of a division.  The quantizers need the
// exact quotient, because bf16 inputs put many of them on the border between two
// codes (a 4-bit group has a tie in one element of some dozens).
#pragma once
#include <cuda_runtime.h>

namespace gwb {

struct Divisor {
  float b, y;
  bool fast;     // the three steps give the nearest integer of the rounded quotient for |a| <= 2^8 |b|
};
__device__ __forceinline__ Divisor make_divisor(float b) {
  const unsigned u = __float_as_uint(b);
  Divisor d;
  d.b = b;
  // 2^-90 <= b <= 2^90: a quotient of at least 1/4 has a remainder of at least 2^-24 of a normal a, and
  // where a is too small for that its quotient's nearest integer is 0 whatever its last bits are
  d.fast = u >= 0x12800000u && u <= 0x6c800000u && (u & 0x7fffffu) != 0x7fffffu;
  d.y = d.fast ? __fdiv_rn(1.0f, b) : 0.0f;
  return d;
}
__device__ __forceinline__ float quotient_fast(float a, const Divisor &d) {
  const float q = __fmul_rn(a, d.y);
  return __fmaf_rn(__fmaf_rn(-q, d.b, a), d.y, q);
}

// a / N for a constant N (neither a power of two nor of an all-ones significand), correctly rounded.
template <int N>
__device__ __forceinline__ float quotient_const(float a) {
  constexpr float b = (float)N, y = 1.0f / (float)N;
  if (!(a >= 0x1p-90f && a <= 0x1p120f)) return __fdiv_rn(a, b);
  const float q = __fmul_rn(a, y);
  return __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
}

// Largest and smallest of two or three numbers; NaN where one is NaN (fmaxf and fminf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  asm("min.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(b), "f"(c));
  return a;
}

// Round half to even of |x| <= 2^22 as the low bits of a float (two's complement from bit 0).
constexpr float kRoundMagic = 12582912.0f;   // 1.5 * 2^23
__device__ __forceinline__ float round_bits(float x) { return __fadd_rn(x, kRoundMagic); }

}  // namespace gwb
