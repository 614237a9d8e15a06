// The FP4 (E2M1) copy of a BF16 matrix and back ("glm5next_mtp_head.rs", `head_fp8` doc: a
// low-precision copy of lm_head used for drafting only; here four bits a weight, with a scale per
// 16 weights and one per row -- the format is in fp4.cuh).
//
// The codes without a division per element, as in the FP8 quantiser (quantize.cu): with
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
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "tc.cuh"

namespace mtp {

namespace {

constexpr int kQThreads = 256;
constexpr int kWaves = 16;  // CTAs per one that runs, at most
constexpr float kUp = 1.0f + 0x1p-21f, kDn = 1.0f - 0x1p-21f;
constexpr float kSmallRs = 0x1p-100f;  // below: s_j rs or its reciprocal may leave the normal range

// Two E4M3 codes (round to nearest even, satfinite): byte 0 from lo, byte 1 from hi.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
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

// max of the two 16-bit halves, lane by lane
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mag_max(uint32_t m, const uint4& u) {
  m = max_u16x2(m, u.x & 0x7FFF7FFFu);
  m = max_u16x2(m, u.y & 0x7FFF7FFFu);
  m = max_u16x2(m, u.z & 0x7FFF7FFFu);
  return max_u16x2(m, u.w & 0x7FFF7FFFu);
}

// 16 columns starting at k0 of a row (zeros past k).
template <bool VEC>
__device__ __forceinline__ void load16(const uint16_t* row, int k0, int k, uint4& a, uint4& b) {
  a = b = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (VEC) {  // k % 8 == 0 and 16-byte aligned rows
    if (k0 < k) a = *reinterpret_cast<const uint4*>(row + k0);
    if (k0 + 8 < k) b = *reinterpret_cast<const uint4*>(row + k0 + 8);
  } else {
    uint32_t u[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t lo = k0 + 2 * t < k ? row[k0 + 2 * t] : 0u;
      const uint32_t hi = k0 + 2 * t + 1 < k ? row[k0 + 2 * t + 1] : 0u;
      u[t] = lo | (hi << 16);
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
    b = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

// The scale and codes of one block of 16 columns.
struct BlockCodes {
  uint32_t c0, c1, sc;
};
__device__ __noinline__ uint4 block_codes_fp64(uint4 u0, uint4 u1, float amax, float rs) {
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

// First scale byte of a row, and the distance of scale byte b from it (fp4.h).
__device__ __forceinline__ uint8_t* scale_row(uint8_t* bs, int64_t row, int kp, int tile) {
  if (tile == 0) return bs + row * (kp / kFp4Block);
  const int64_t tl = row / tile;
  const int lr = static_cast<int>(row - tl * tile);
  const int64_t chunk = tl * ((tile + 127) / 128) + lr / 128;
  return bs + chunk * (kp / 64) * 512 + (lr & 31) * 16 + ((lr & 127) >> 5) * 4;
}
__device__ __forceinline__ int scale_at(int b, int tile) { return tile > 0 ? (b >> 2) * 512 + (b & 3) : b; }

// TPR threads of a block (a warp, or the whole block) per row, two passes over it: the magnitude
// maximum, then 16 columns (one block scale) a thread at a time.
template <int TPR, bool VEC>
__global__ void __launch_bounds__(kQThreads) fp4_quantize_kernel(const uint16_t* __restrict__ w, uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ bs, float* __restrict__ rs_out,
                                                                 int32_t* __restrict__ status,
                                                                 const int32_t* __restrict__ valid, int rows, int k, int tile) {
  __shared__ uint32_t red[kQThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int kp = fp4_padded(k), nblk = kp / kFp4Block;
  pdl_wait_prior_grid();
  // The next kernel may launch at once (what it reads before its own wait, a linear's weights, was
  // written before this grid's wait ended).
  pdl_launch_dependents();
  for (int64_t row = (static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x) / TPR; row < rows;
       row += static_cast<int64_t>(gridDim.x) * kQThreads / TPR) {
    const uint16_t* wr = w + row * k;
    const bool ok = valid == nullptr || valid[row] != 0;
    uint32_t m = 0;
    if (ok)
      for (int b = t; b * kFp4Block < k; b += TPR) {
        uint4 u0, u1;
        load16<VEC>(wr, b * kFp4Block, k, u0, u1);
        m = mag_max(mag_max(m, u0), u1);
      }
    uint32_t mx = max(m & 0xFFFFu, m >> 16);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    if constexpr (TPR > 32) {
      if (lane == 0) red[warp] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kQThreads / 32; ++i) mx = max(mx, red[i]);
      __syncthreads();
    }
    float rs = __fdiv_rn(bf16_bits_to_f32(mx), 2688.0f);
    if (mx >= 0x7F80u) {  // a NaN or Inf in the row
      if (t == 0) store_status(status, MTP_ERR_NONFINITE);
      rs = 0.0f;
    }
    if (t == 0) rs_out[row] = rs;
    const float r6 = rs >= kSmallRs ? recip(__fmul_rn(6.0f, rs)) : 0.0f;
    const float r6_up = __fmul_rn(r6, kUp), r6_dn = __fmul_rn(r6, kDn);
    uint8_t* qr = q + row * (kp / 2);
    uint8_t* br = scale_row(bs, row, kp, tile);
    for (int b = t; b < nblk; b += TPR) {
      BlockCodes o{0u, 0u, 0u};
      if (rs > 0.0f && b * kFp4Block < k) {
        uint4 u0, u1;
        load16<VEC>(wr, b * kFp4Block, k, u0, u1);
        o = block_codes(u0, u1, rs, r6_up, r6_dn);
      }
      reinterpret_cast<uint2*>(qr)[b] = make_uint2(o.c0, o.c1);
      br[scale_at(b, tile)] = static_cast<uint8_t>(o.sc);
    }
  }
}

// A read-once load that stays in front of what follows.
__device__ __forceinline__ uint4 ld_now(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Rows that TPR threads hold in registers, kHeld blocks of 16 columns a thread: one read of the matrix.
// TPR = 32: a warp per row, eight rows a CTA; otherwise a CTA per row. Threads per SM over registers per
// thread: at H = 6144, V = 154880 768 threads (80 registers) took 516 us, 1,024 (64) 473, 1,280 (48, a few
// spilled) 458, and 415 with the grid in many waves (launch_held): 5.9 TB/s of bytes read and written.
constexpr int kHeld = 3;
constexpr int kHeldThreads = 1280;  // per SM
template <int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, kHeldThreads / (TPR == 32 ? 256 : TPR))
    fp4_quantize_held_kernel(const uint16_t* __restrict__ w, uint8_t* __restrict__ q, uint8_t* __restrict__ bs,
                             float* __restrict__ rs_out, int32_t* __restrict__ status, const int32_t* __restrict__ valid,
                             int rows, int k, int tile) {
  constexpr int kThreads = TPR == 32 ? 256 : TPR;
  __shared__ uint32_t red[2][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int kp = fp4_padded(k), nblk = kp / kFp4Block;
  pdl_wait_prior_grid();
  int turn = 0;
  bool first = true;
  for (int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / TPR; row < rows;
       row += static_cast<int64_t>(gridDim.x) * kThreads / TPR) {
    const uint4* wr = reinterpret_cast<const uint4*>(w + row * k);  // k % 8 == 0
    const bool ok = valid == nullptr || valid[row] != 0;
    uint4 u[kHeld][2];
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int p = 2 * (t + i * TPR);  // 8-column piece
      u[i][0] = u[i][1] = z;
      if (ok && 8 * p < k) u[i][0] = ld_now(wr + p);
      if (ok && 8 * p + 8 < k) u[i][1] = ld_now(wr + p + 1);
    }
    // The next kernel may launch once the first rows are asked for (so that a linear's weight stream does not
    // get in front of them); what it reads before its own wait was written before this grid's wait ended.
    if (first) pdl_launch_dependents();
    first = false;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) m = mag_max(mag_max(m, u[i][0]), u[i][1]);
    uint32_t mx = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if constexpr (TPR > 32) {
      if (lane == 0) red[turn][warp] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) mx = max(mx, red[turn][i]);
      turn ^= 1;  // the next row's maxima go elsewhere: one barrier a row is enough
    }
    float rs = __fdiv_rn(bf16_bits_to_f32(mx), 2688.0f);
    if (mx >= 0x7F80u) {  // a NaN or Inf in the row
      if (t == 0) store_status(status, MTP_ERR_NONFINITE);
      rs = 0.0f;
    }
    if (t == 0) rs_out[row] = rs;
    const float r6 = rs >= kSmallRs ? recip(__fmul_rn(6.0f, rs)) : 0.0f;
    const float r6_up = __fmul_rn(r6, kUp), r6_dn = __fmul_rn(r6, kDn);
    uint2* qr = reinterpret_cast<uint2*>(q + row * (kp / 2));
    uint8_t* br = scale_row(bs, row, kp, tile);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int b = t + i * TPR;
      if (b < nblk) {
        BlockCodes o{0u, 0u, 0u};
        if (rs > 0.0f) o = block_codes(u[i][0], u[i][1], rs, r6_up, r6_dn);
        qr[b] = make_uint2(o.c0, o.c1);
        br[scale_at(b, tile)] = static_cast<uint8_t>(o.sc);
      }
    }
  }
}

// bf16( fp32( code * s_j * rs ) ): eight columns (a 4-byte load, a 16-byte store) a thread, kUnits at a
// time, neighbouring lanes neighbouring columns. per_row: eights of a row; magic = floor(2^64 / per_row) + 1
// (its product with a 32-bit number has the quotient in the upper half). A chunk a block, as many blocks as that
// takes: lm_head 368 us (6.6 TB/s), by 1,216 blocks in a loop 410.
constexpr int kUnits = 4;
__global__ void __launch_bounds__(kQThreads) fp4_dequantize_vec_kernel(const Fp4Matrix m, uint16_t* __restrict__ w,
                                                                       uint32_t total, uint32_t per_row,
                                                                       unsigned long long magic, int kp) {
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const uint64_t i0 = (static_cast<uint64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5)) * 32 * kUnits + lane;
  uint32_t c[kUnits], s[kUnits];
  float rs[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint64_t i = i0 + 32 * j;
    if (i < total) {
      const uint32_t row = static_cast<uint32_t>(__umul64hi(i, magic)), b = static_cast<uint32_t>(i) - row * per_row;
      c[j] = __ldcs(reinterpret_cast<const uint32_t*>(m.q + static_cast<size_t>(row) * (kp / 2)) + b);
      s[j] = m.bs[static_cast<size_t>(row) * (kp / kFp4Block) + (b >> 1)];
      rs[j] = m.rs[row];
    }
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint64_t i = i0 + 32 * j;
    if (i < total) {
      const uint32_t s2 = e4m3x2_to_f16x2(s[j] * 0x0101u);
      uint32_t v[4], o[4];
      e2m1x8_to_f16x2x4(c[j], v);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t p = f16x2_mul(v[t], s2);  // exact
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
            : "=r"(o[t])
            : "f"(__fmul_rn(f16_hi(p), rs[j])), "f"(__fmul_rn(f16_lo(p), rs[j])));
      }
      __stcs(reinterpret_cast<uint4*>(w) + i, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
  // (no early launch: a sweep that follows may read w, as its lm_head, before its own wait)
}

// The same for rows that are not made of eights: 16 columns (one block scale) a thread.
__global__ void __launch_bounds__(kQThreads) fp4_dequantize_kernel(const Fp4Matrix m, uint16_t* __restrict__ w, int rows,
                                                                   int k) {
  const int kp = fp4_padded(k), nblk = (k + kFp4Block - 1) / kFp4Block;
  const int64_t total = static_cast<int64_t>(rows) * nblk;
  pdl_wait_prior_grid();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kQThreads) {
    const int64_t row = i / nblk;
    const int b = static_cast<int>(i - row * nblk);
    const uint2 c = reinterpret_cast<const uint2*>(m.q + row * (kp / 2))[b];
    const uint32_t s2 = e4m3x2_to_f16x2(m.bs[row * (kp / kFp4Block) + b] * 0x0101u);
    const float rs = m.rs[row];
    uint16_t* dst = w + row * k + b * kFp4Block;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[4];
      e2m1x8_to_f16x2x4(h == 0 ? c.x : c.y, v);
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const uint32_t p = f16x2_mul(v[t >> 1], s2);  // exact
        if (b * kFp4Block + 8 * h + t < k)
          dst[8 * h + t] = static_cast<uint16_t>(bf16_bits_rn(__fmul_rn((t & 1) ? f16_hi(p) : f16_lo(p), rs)));
      }
    }
  }
}

}  // namespace

namespace {

template <int TPR>
cudaError_t launch_held(const DeviceInfo& di, int rows, cudaStream_t stream, void** args) {
  constexpr int kThreads = TPR == 32 ? 256 : TPR;
  const int64_t blocks = (static_cast<int64_t>(rows) * TPR + kThreads - 1) / kThreads;
  // Many more CTAs than run at once, of a few rows each: rows that take longer (more boundaries inside their
  // brackets) and the last wave even out (lm_head 458 us with 1.6 waves of CTAs, 415 with 16; one row a CTA
  // is slower for short rows).
  const int64_t cap = static_cast<int64_t>(di.sm_count) * (kHeldThreads / kThreads) * kWaves;
  return launch_pdl(reinterpret_cast<const void*>(fp4_quantize_held_kernel<TPR>),
                    dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(kThreads), 0, stream, args);
}

}  // namespace

// Rows of up to 512 * kHeld blocks of 16 columns (24,576 columns) are held in the registers of as few
// threads as hold them; longer ones, and rows that are not made of 16-byte pieces, take two passes.
cudaError_t launch_fp4_quantize(const uint16_t* w, uint8_t* q, uint8_t* bs, float* rs, int32_t* status,
                                const int32_t* valid, int rows, int k, cudaStream_t stream, int tile) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const bool vec = k % 8 == 0;
  const int nblk = fp4_padded(k) / kFp4Block;
  void* args[] = {&w, &q, &bs, &rs, &status, &valid, &rows, &k, &tile};
  if (vec) {
    if (nblk <= 32 * kHeld) return launch_held<32>(di, rows, stream, args);
    if (nblk <= 128 * kHeld) return launch_held<128>(di, rows, stream, args);
    if (nblk <= 256 * kHeld) return launch_held<256>(di, rows, stream, args);
    if (nblk <= 512 * kHeld) return launch_held<512>(di, rows, stream, args);
  }
  const bool wide = rows < di.sm_count * 8;  // fewer rows than warps in flight: a block per row
  const void* kern = wide ? (vec ? reinterpret_cast<const void*>(fp4_quantize_kernel<kQThreads, true>)
                                 : reinterpret_cast<const void*>(fp4_quantize_kernel<kQThreads, false>))
                          : (vec ? reinterpret_cast<const void*>(fp4_quantize_kernel<32, true>)
                                 : reinterpret_cast<const void*>(fp4_quantize_kernel<32, false>));
  const int per_block = wide ? 1 : kQThreads / 32;
  int64_t blocks = (static_cast<int64_t>(rows) + per_block - 1) / per_block;
  if (blocks > 8 * kWaves * di.sm_count) blocks = 8 * kWaves * di.sm_count;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kQThreads), 0, stream, args);
}

cudaError_t launch_fp4_dequantize(const Fp4Matrix& m, uint16_t* w, int rows, int k, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  Fp4Matrix mm = m;
  const int64_t eights = static_cast<int64_t>(rows) * (k / 8);
  if (k % 8 == 0 && eights < (static_cast<int64_t>(1) << 32)) {
    uint32_t total = static_cast<uint32_t>(eights), per_row = static_cast<uint32_t>(k / 8);
    // (one eight a row: the quotient is the number itself, 2^64 does not fit)
    unsigned long long magic = per_row == 1 ? 0ull : ~0ull / per_row + 1;
    int kp = fp4_padded(k);
    if (per_row > 1) {
      const int64_t blocks = (eights + kQThreads * kUnits - 1) / (kQThreads * kUnits);
      void* args[] = {&mm, &w, &total, &per_row, &magic, &kp};
      return launch_pdl(reinterpret_cast<const void*>(fp4_dequantize_vec_kernel), dim3(static_cast<unsigned>(blocks)),
                        dim3(kQThreads), 0, stream, args);
    }
  }
  const int64_t total = static_cast<int64_t>(rows) * ((k + kFp4Block - 1) / kFp4Block);
  int64_t blocks = (total + kQThreads - 1) / kQThreads;
  if (blocks > 8 * kWaves * di.sm_count) blocks = 8 * kWaves * di.sm_count;
  void* args[] = {&mm, &w, &rows, &k};
  return launch_pdl(reinterpret_cast<const void*>(fp4_dequantize_kernel), dim3(static_cast<unsigned>(blocks)),
                    dim3(kQThreads), 0, stream, args);
}

}  // namespace mtp
