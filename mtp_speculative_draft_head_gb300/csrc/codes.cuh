// Codes of the library's 8-bit and 4-bit copies (device helpers of every kernel that makes some).
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "fp4.cuh"

namespace mtp {

// Two E4M3 codes (round to nearest even, satfinite): byte 0 from lo, byte 1 from hi.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// max of the two 16-bit halves, lane by lane
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// ------------------------------------------------------------------------------------------ E4M3
// The codes without a division per element. The code of the quotient depends only on which
// pair of neighbouring E4M3 rounding boundaries the quotient lies between. With r = 1/s, the
// products y_up = f * r (1 + 2^-21) and y_dn = f * r (1 - 2^-21) (each factor and product
// rounded to nearest) bracket fp32(f / s) strictly: the four roundings move them by at most
// 3 * 2^-24 relative, fp32(f / s) is within 2^-24 of f / s, and 2^-21 - 3 * 2^-24 > 2^-24.
// The conversion to E4M3 (round to nearest even, saturating) is monotonic, so when y_up and
// y_dn give the same code, fp32(f / s) gives it too. Otherwise (a boundary inside the bracket:
// nearly always an exact tie, about 0.5 % of the elements of Gaussian rows) the code comes from
// the division itself. Quotients below the
// fp32 normal range convert to a signed zero on all three paths. Rows whose scale is not a
// normal fp32 number take the division for every element.
// Codes of one bf16 pair (32-bit word) through the bracket, the division when it is open.
__device__ __forceinline__ uint32_t pair_codes(uint32_t pair, float s, float r_up, float r_dn) {
  const float a = bf16_lo(pair), b = bf16_hi(pair);
  const uint32_t up = e4m3x2(__fmul_rn(a, r_up), __fmul_rn(b, r_up));
  const uint32_t dn = e4m3x2(__fmul_rn(a, r_dn), __fmul_rn(b, r_dn));
  if (up == dn) return up;
  return e4m3x2(__fdiv_rn(a, s), __fdiv_rn(b, s));
}

__device__ __forceinline__ uint32_t pair_codes_div(uint32_t pair, float s) {
  return e4m3x2(__fdiv_rn(bf16_lo(pair), s), __fdiv_rn(bf16_hi(pair), s));
}

// Eight codes e4m3( fp32( w / s ) ) of BF16 pairs, without a branch: with r = 1 / s rounded to nearest and q = w r, one
// step q + r (w - q s), both by fused multiply-adds, is the correctly rounded quotient (Markstein); the remainder is exact
// for s >= 2^-80 wherever the quotient reaches half of the smallest code. Smaller scales divide.
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint2 codes_e4m3x8(const uint32_t (&u)[4], float s) {
  if (s == 0.0f) return make_uint2(0u, 0u);
  uint32_t c[4];
  if (s >= 0x1p-80f) {
    const float r = __frcp_rn(s);
    const uint64_t r2 = f2_pack(r, r), ns = f2_pack(-s, -s);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint64_t w = bf16x2_to_f2(u[t]);
      const uint64_t q = f2_mul(w, r2);
      const uint64_t y = f2_fma(f2_fma(q, ns, w), r2, q);
      c[t] = e4m3x2(f2_lo(y), f2_hi(y));
    }
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) c[t] = pair_codes_div(u[t], s);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// ------------------------------------------------------------------------------------------ E2M1
// The same for a block of 16 E2M1 codes and its E4M3 scale (the format is in fp4.cuh): with
// r = 1 / (s_j rs), formed in fp32, the products |w| r (1 + 2^-21) and |w| r (1 - 2^-21) bracket
// the real quotient strictly (s_j rs, the factor and the product round by at most 2^-24 each, the
// approximate reciprocal errs by at most 2^-23: together less than 2^-21). The conversion is monotonic, so equal codes of both
// bracket ends are the code of the quotient. Otherwise one rounding boundary b lies inside the
// bracket and the sign of |w| - (b s_j) rs decides: b s_j has 7 significant bits and is exact, so
// one fused multiply-add gives that sign exactly (zero: a tie, to the even code). It comes up for
// a few of a thousand weights: BF16 weights and their row's maximum are 8-bit numbers, whose ratios
// often meet a boundary. (Deciding those in fp64 division made the whole copy 17 times slower.)
// The block scales go the same way, with 6 b in the place of b s_j. Rows whose scale is below
// 2^-100, where a product may leave the normal fp32 range, form the quotients in fp64 (w has 8
// significant bits, s_j rs 28 and a boundary 3, so a quotient off the boundary is off by 2^-40 of
// its size) and reach the conversion through round-to-odd.
constexpr float kUp = 1.0f + 0x1p-21f, kDn = 1.0f - 0x1p-21f;
constexpr float kSmallRs = 0x1p-100f;  // below: s_j rs or its reciprocal may leave the normal range

// Eight E2M1 codes (round to nearest even, satfinite), v[i] in bits 4i..4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}
// fp64 -> fp32 by round-to-odd: a following rounding to a few bits is the rounding of q itself.
__device__ __forceinline__ float to_odd(double q) {
  float f = __double2float_rz(q);
  if (static_cast<double>(f) != q) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// 1 / x within 2^-23 of it, x and the result normal numbers.
__device__ __forceinline__ float recip(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The quotients in fp64, for rows with a scale below kSmallRs. (Out of line, in block_codes_fp64: inlined,
// their conversions were executed for every block, on an fp64 pipe that was busy a third of the time.)
__device__ __forceinline__ uint32_t block_scale_code_fp64(float amax, float rs) {
  return e4m3x2(to_odd(static_cast<double>(amax) / (6.0 * static_cast<double>(rs))), 0.0f) & 0xFFu;
}
__device__ __forceinline__ uint32_t codes8_fp64(uint4 u, float s, float rs) {
  const double d = static_cast<double>(s) * static_cast<double>(rs);  // exact: 4 + 24 bits
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float a[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) a[t] = to_odd(static_cast<double>((t & 1) ? bf16_hi(w[t >> 1]) : bf16_lo(w[t >> 1])) / d);
  return e2m1x8(a);
}

// E4M3 code of amax / (6 rs), rs >= kSmallRs.
__device__ __forceinline__ uint32_t block_scale_code(float amax, float rs, float r6_up, float r6_dn) {
  const uint32_t two = e4m3x2(__fmul_rn(amax, r6_dn), __fmul_rn(amax, r6_up));
  const uint32_t c = two & 0xFFu;  // the lower end; the upper is c or c + 1
  if (c == two >> 8) return c;
  const float b6 = 3.0f * (e4m3_value(c) + e4m3_value(c + 1));  // 6 * the midpoint, exact
  const float d = __fmaf_rn(-b6, rs, amax);
  return c + ((d > 0.0f || (d == 0.0f && (c & 1u))) ? 1u : 0u);
}

// Eight codes of the BF16 pairs u[0..3] for the block scale value s (> 0) and row scale rs >= kSmallRs.
__device__ __forceinline__ uint32_t codes8(const uint32_t (&u)[4], float s, float rs, float r_up, float r_dn) {
  const uint64_t up2 = f2_pack(r_up, r_up), dn2 = f2_pack(r_dn, r_dn);
  float a[8];
  uint64_t f2[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    f2[t] = bf16x2_to_f2(u[t]);
    const uint64_t y = f2_mul(f2[t], up2);
    a[2 * t] = f2_lo(y);
    a[2 * t + 1] = f2_hi(y);
  }
  const uint32_t up = e2m1x8(a);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint64_t y = f2_mul(f2[t], dn2);
    a[2 * t] = f2_lo(y);
    a[2 * t + 1] = f2_hi(y);
  }
  uint32_t dn = e2m1x8(a);
  uint32_t diff = up ^ dn;
  while (diff != 0u) {  // the codes on either side of a boundary differ in their low three bits
    const int t = (__ffs(diff) - 1) >> 2;
    diff &= ~(0xFu << (4 * t));
    const uint32_t c = (dn >> (4 * t)) & 7u;
    // midpoint above code c: 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, as quarters in nibbles
    const float mid = 0.25f * static_cast<float>((0x14EA7531ull >> (4 * c)) & (c == 6u ? 0x1Fu : 0xFu));
    const uint32_t pair = t < 4 ? (t < 2 ? u[0] : u[1]) : (t < 6 ? u[2] : u[3]);
    const float f = fabsf((t & 1) ? bf16_hi(pair) : bf16_lo(pair));
    const float d = __fmaf_rn(-(mid * s), rs, f);
    if (d > 0.0f || (d == 0.0f && (c & 1u))) dn += 1u << (4 * t);
  }
  return dn;
}

__device__ __forceinline__ uint32_t mag_max(uint32_t m, const uint4& u) {
  m = max_u16x2(m, u.x & 0x7FFF7FFFu);
  m = max_u16x2(m, u.y & 0x7FFF7FFFu);
  m = max_u16x2(m, u.z & 0x7FFF7FFFu);
  return max_u16x2(m, u.w & 0x7FFF7FFFu);
}

// The scale and codes of one block of 16 columns.
struct BlockCodes {
  uint32_t c0, c1, sc;
};
static __device__ __noinline__ uint4 block_codes_fp64(uint4 u0, uint4 u1, float amax, float rs) {
  const uint32_t sc = block_scale_code_fp64(amax, rs);
  if (sc == 0u) return make_uint4(0u, 0u, 0u, 0u);
  const float s = e4m3_value(sc);
  return make_uint4(codes8_fp64(u0, s, rs), codes8_fp64(u1, s, rs), sc, 0u);
}
__device__ __forceinline__ BlockCodes block_codes(const uint4& u0, const uint4& u1, float rs, float r6_up, float r6_dn) {
  BlockCodes o{0u, 0u, 0u};
  const uint32_t bm = mag_max(mag_max(0u, u0), u1);
  const float amax = bf16_bits_to_f32(max(bm & 0xFFFFu, bm >> 16));
  if (rs < kSmallRs) {
    const uint4 v = block_codes_fp64(u0, u1, amax, rs);
    return BlockCodes{v.x, v.y, v.z};
  }
  o.sc = block_scale_code(amax, rs, r6_up, r6_dn);
  if (o.sc != 0u) {
    const float s = e4m3_value(o.sc);
    const float r = recip(__fmul_rn(s, rs));
    const float r_up = __fmul_rn(r, kUp), r_dn = __fmul_rn(r, kDn);
    o.c0 = codes8({u0.x, u0.y, u0.z, u0.w}, s, rs, r_up, r_dn);
    o.c1 = codes8({u1.x, u1.y, u1.z, u1.w}, s, rs, r_up, r_dn);
  }
  return o;
}

// The same with one conversion per code, for rows whose scale was rounded (rs != max|w| / 2688). A quotient
// w / (s_j rs) is R (1 - rho), R = 2688 w / (s_j max|w|) of numbers with 8, 4 and 8 significant bits and rho, below 2^-24,
// the scale's own rounding error relative to it. R is a rounding boundary b (3 bits) or off it by 2^-18 of it, so only R = b
// is decided by rho, and the same way in the whole row: downwards where the scale was rounded up, upwards where it was
// rounded down. The bracket's end on that side of the quotient gives it. The block scales, 448 max|w_j| / max|w| (1 - rho)
// against boundaries of 5 bits, go the same way. (About half the instructions of block_codes: 16384 rows of 8 heads into
// the cache took 26 us with that.)
__device__ __forceinline__ uint32_t codes8_biased(const uint32_t (&u)[4], float r) {
  const uint64_t r2 = f2_pack(r, r);
  float a[8];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint64_t y = f2_mul(bf16x2_to_f2(u[t]), r2);
    a[2 * t] = f2_lo(y);
    a[2 * t + 1] = f2_hi(y);
  }
  return e2m1x8(a);
}
// side: kUp or kDn; rs >= kSmallRs, r6 = recip(6 rs) * side.
__device__ __forceinline__ BlockCodes block_codes_biased(const uint4& u0, const uint4& u1, float rs, float r6, float side) {
  BlockCodes o{0u, 0u, 0u};
  const uint32_t bm = mag_max(mag_max(0u, u0), u1);
  const float amax = bf16_bits_to_f32(max(bm & 0xFFFFu, bm >> 16));
  o.sc = e4m3x2(__fmul_rn(amax, r6), 0.0f) & 0xFFu;
  if (o.sc != 0u) {
    const float r = __fmul_rn(recip(__fmul_rn(e4m3_value(o.sc), rs)), side);
    o.c0 = codes8_biased({u0.x, u0.y, u0.z, u0.w}, r);
    o.c1 = codes8_biased({u1.x, u1.y, u1.z, u1.w}, r);
  }
  return o;
}

}  // namespace mtp
