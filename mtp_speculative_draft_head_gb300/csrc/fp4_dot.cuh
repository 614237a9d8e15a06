// A warp's 16 weight rows x 8 activation rows of a product with an FP4 copy, straight from memory.
#pragma once

#include <stdint.h>

#include "fp4.cuh"
#include "tc.cuh"

namespace mtp {

// d[i] += sum_k code * s * x over a padded row of kp codes: rows r0 + g and r0 + g + 8 of the copy
// (clamped to the last row), activation rows xh (f16, row stride kp, 8 of them). Fragment layout of
// mma.m16n8k16: d[0], d[1] = row g, columns 2 t4, 2 t4 + 1; d[2], d[3] = row g + 8. Thread t4 takes
// the eight codes 8 t4 .. 8 t4 + 7 of every 32 of a row, in the activations as in the weights.
// The tensor cores' running sum is restarted every 256 columns and added in fp32.
__device__ __forceinline__ void fp4_dot_16x8(const uint8_t* q, const uint8_t* bs, int64_t r0, int64_t rows, int kp,
                                             const uint16_t* xh, float (&d)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int64_t ra = r0 + g < rows ? r0 + g : rows - 1, rb = r0 + g + 8 < rows ? r0 + g + 8 : rows - 1;
  const uint8_t *qa = q + ra * (kp / 2) + 4 * t4, *qb = q + rb * (kp / 2) + 4 * t4;
  const uint8_t *sa = bs + ra * (kp / 16) + (t4 >> 1), *sb = bs + rb * (kp / 16) + (t4 >> 1);
  const uint16_t* xr = xh + static_cast<int64_t>(g) * kp + 8 * t4;
  for (int k0 = 0; k0 < kp; k0 += 256) {
    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ch = k0 / 32 + j;
      uint32_t va[4], vb[4];
      e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(qa + 16 * ch), va);
      e2m1x8_to_f16x2x4(*reinterpret_cast<const uint32_t*>(qb + 16 * ch), vb);
      const uint32_t s2a = e4m3x2_to_f16x2(sa[2 * ch] * 0x0101u), s2b = e4m3x2_to_f16x2(sb[2 * ch] * 0x0101u);
      const uint4 x = *reinterpret_cast<const uint4*>(xr + 32 * ch);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a[4] = {f16x2_mul(va[2 * h], s2a), f16x2_mul(vb[2 * h], s2b), f16x2_mul(va[2 * h + 1], s2a),
                               f16x2_mul(vb[2 * h + 1], s2b)};
        mma_f16(c, a, h == 0 ? x.x : x.z, h == 0 ? x.y : x.w);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = __fadd_rn(d[i], c[i]);
  }
}

}  // namespace mtp
