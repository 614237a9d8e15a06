// The FP4 (E2M1) copy of a BF16 matrix and back ("glm5next_mtp_head.rs", `head_fp8` doc: a
// low-precision copy of lm_head used for drafting only; here four bits a weight, with a scale per
// 16 weights and one per row -- the format is in fp4.cuh).
//
// The codes of a block are made without a division per element (codes.cuh).
#include <cuda_runtime.h>
#include <stdint.h>

#include "codes.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "tc.cuh"

namespace mtp {

namespace {

constexpr int kQThreads = 256;
constexpr int kWaves = 16;  // CTAs per one that runs, at most

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
