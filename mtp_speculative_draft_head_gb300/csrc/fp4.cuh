// Device helpers of the FP4 (E2M1) copies.
//
// Format. A row of k BF16 weights becomes
//   rs       = fp32( max |w| / 2688 )                       2688 = 6 * 448
//   s_j      = e4m3( max_{block j} |w| / (6 rs) )           one E4M3 scale per 16 columns
//   code     = e2m1( w / (s_j rs) )                         0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
// where e4m3 / e2m1 round the real quotient once, to nearest even, and saturate. The value a code
// stands for is code * s_j * rs; code * s_j needs 6 significant bits and is exact in f16.
#pragma once

#include <stdint.h>

#include "fp4.h"

namespace mtp {

// Eight E2M1 codes of one word -> four f16 pairs, exactly; pair i holds codes 2i (low half), 2i+1.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 codes (bits 0..15 of w) -> f16 pair, exactly (low half = lower byte).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float f16_lo(uint32_t h) {
  float r;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ float f16_hi(uint32_t h) {
  float r;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, u;\n\t}" : "=f"(r) : "r"(h));
  return r;
}

// One lane of a converged warp (as a predicate: what issues a warp's copies and MMAs).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Value of an E4M3 code 0..0x7E (non-negative), exactly.
__device__ __forceinline__ float e4m3_value(uint32_t code) { return f16_lo(e4m3x2_to_f16x2(code)); }

}  // namespace mtp
