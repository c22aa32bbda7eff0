// e4m3.cuh -- e4m3 bytes of the quantised KV cache as bf16 values.
//
// An e4m3 number (sign, 4 exponent bits with bias 7, 3 fraction bits) whose
// bits are put at the sign, the low exponent and the high fraction bits of a
// bf16 number reads as its value times 2^(7 - 127), subnormal numbers
// included; one bf16 product with 2^120 times the row's scale then gives the
// stored value.  A scale byte c stands for 2^(c - 127) with c - 127 in
// -124 .. 7, so the factor's exponent field c + 120 is 123 .. 254 and the
// product (4 significant bits, no exponent outside bf16's range) is exact.
// Scale byte 135 marks a row with a non-finite element: its factor is
// infinity and its elements are stored as 0, so it reads as NaN.
#pragma once

#include <stdint.h>

namespace bi {

constexpr int kQ8MinExp = -124, kQ8MaxExp = 7;
constexpr int kQ8ScaleBias = 127, kQ8NonFinite = kQ8MaxExp + kQ8ScaleBias + 1;
constexpr uint32_t kQ8FactorBias = 0x3C003C00u;  // 120 in both exponent fields

// Bytes 0 and 2 (1 and 3) of x as the bf16 pair (low, high), times 2^-120.
__device__ __forceinline__ uint32_t e4m3_even(uint32_t x) {
  uint32_t y;  // each byte under eight copies of its sign
  asm("prmt.b32 %0, %1, 0, 0xA280;" : "=r"(y) : "r"(x));
  return (y << 4) & 0x87f087f0u;
}
__device__ __forceinline__ uint32_t e4m3_odd(uint32_t x) {
  return ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
}
// The factor of one scale byte in both halves; the factors of two.
__device__ __forceinline__ uint32_t q8_factor2(uint32_t c) { return c * 0x00800080u + kQ8FactorBias; }
__device__ __forceinline__ uint32_t q8_factors(uint32_t c0_c1) {
  return __byte_perm(c0_c1, 0, 0x4140) * 128u + kQ8FactorBias;
}
// The factor as fp32 (2^(c - 127 + 120), infinity for a non-finite row).
__device__ __forceinline__ float q8_factor_f32(uint32_t c) {
  return __uint_as_float((c + 120u) << 23);
}
// Product of bf16 pairs; exact here.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace bi
