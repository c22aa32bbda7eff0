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
  uint32_t y;
  asm("prmt.b32 %0, %1, 0, 0xB391;" : "=r"(y) : "r"(x));
  return (y << 4) & 0x87f087f0u;
}
// Bytes 0 and 1 (2 and 3) of x as the fp16 pair (low, high), exact.
__device__ __forceinline__ uint32_t e4m3_f16_lo(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(y)
      : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3_f16_hi(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(y)
      : "r"(x));
  return y;
}
// The fp16 pair (low, high) of two floats.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The factor of one scale byte in both halves.
__device__ __forceinline__ uint32_t q8_factor2(uint32_t c) { return c * 0x00800080u + kQ8FactorBias; }
// Product of bf16 pairs; exact here.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// e4m3_even and e4m3_odd times 2^3, so that an e4m3 subnormal is a normal bf16
// number too: an MMA aligns a product by its operands' exponent fields, and a
// subnormal operand, aligned above its own magnitude, can cost the sum its last
// bit (one fp32 element in some 10^8 came out a unit off without the product).
constexpr int kE4m3MmaShift = 117;  // the value times 2^-117
__device__ __forceinline__ uint32_t e4m3_even_mma(uint32_t x) {
  return mul_bf16x2(e4m3_even(x), 0x41004100u);
}
__device__ __forceinline__ uint32_t e4m3_odd_mma(uint32_t x) {
  return mul_bf16x2(e4m3_odd(x), 0x41004100u);
}

}  // namespace bi
