// Rows of keys and values into the paged FP4 cache, and back to BF16.
//
// A row (one token, one head, key or value) is quantised by itself, in the format and with the
// roundings of the FP4 copies (codes.cuh): E2M1 codes, an E4M3 scale per 16 columns, an fp32 scale per
// row. D / 16 threads share a row, one block of 16 columns each (32 bytes in, 8 bytes of codes and
// one of scale out), so a row's maximum is a few shuffles and a warp's loads and stores are
// contiguous over whole heads. Bound by bytes: 4 D in and 2 (D/2 + D/16 + 4) out for a token's key and
// value of one head, or the other way round.
#include <cuda_runtime.h>
#include <stdint.h>

#include "codes.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "layer.h"
#include "tc.cuh"

namespace mtp {

namespace {

constexpr int kCThreads = 256;

// Where row t of the packed rows lives: its place in the cache's rows of one head and kind, as
// page * kind/head stride + offset. -1: the row belongs to no sequence; -2: its place does not exist.
struct Place {
  int page, off;
};
__device__ __forceinline__ int find_place(const CacheRowsArgs& a, int t, Place& p) {
  // the last sequence that starts at or before t
  int lo = 0, hi = a.B;  // row_start[lo] <= t < row_start[hi], if the starts ascend
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.row_start[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int s0 = a.row_start[lo], s1 = a.row_start[lo + 1];
  if (t < s0 || t >= s1) return -1;
  const int64_t pos = static_cast<int64_t>(a.position[lo]) + (t - s0);
  if (pos < 0 || pos >= static_cast<int64_t>(a.max_pages) * a.c.page) return -2;
  p.page = a.table[static_cast<int64_t>(lo) * a.max_pages + pos / a.c.page];
  p.off = static_cast<int>(pos % a.c.page);
  return p.page < 0 || p.page >= a.c.pages ? -2 : 0;
}

template <int D>
__global__ void __launch_bounds__(kCThreads) cache_write_kernel(const CacheRowsArgs a) {
  constexpr int kB = D / kFp4Block;  // blocks (and threads) of a row
  pdl_wait_prior_grid();
  const int per_token = 2 * a.c.heads * kB;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kCThreads + threadIdx.x;
  const int t = static_cast<int>(i / per_token), r = static_cast<int>(i % per_token);
  const int j = r % kB, h = (r / kB) % a.c.heads, kind = r / (kB * a.c.heads);
  Place p{0, 0};
  int found = -1;
  uint4 u0 = make_uint4(0u, 0u, 0u, 0u), u1 = u0;
  if (t < a.T) {
    const uint16_t* src = (kind == 0 ? a.k_in + t * a.ld_k : a.v_in + t * a.ld_v) + h * D + j * kFp4Block;
    u0 = __ldcs(reinterpret_cast<const uint4*>(src));
    u1 = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
    found = find_place(a, t, p);
  }
  uint32_t m = mag_max(mag_max(0u, u0), u1);
  uint32_t mx = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int k = kB / 2; k > 0; k >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  if (found != 0) {
    if (found == -2) store_status(a.status, MTP_ERR_ARG);
    return;
  }
  float rs = __fdiv_rn(bf16_bits_to_f32(mx), 2688.0f);
  if (mx >= 0x7F80u) {  // a NaN or Inf in the row
    if (j == 0) store_status(a.status, MTP_ERR_NONFINITE);
    rs = 0.0f;
  }
  BlockCodes o{0u, 0u, 0u};
  if (rs > 0.0f) {
    const float r6 = rs >= kSmallRs ? recip(__fmul_rn(6.0f, rs)) : 0.0f;
    o = block_codes(u0, u1, rs, __fmul_rn(r6, kUp), __fmul_rn(r6, kDn));
  }
  const int64_t dst = ((static_cast<int64_t>(p.page) * 2 + kind) * a.c.heads + h) * a.c.page + p.off;
  *reinterpret_cast<uint2*>(a.c.q + dst * (D / 2) + j * 8) = make_uint2(o.c0, o.c1);
  a.c.bs[dst * kB + j] = static_cast<uint8_t>(o.sc);
  if (j == 0) a.c.rs[dst] = rs;
}

template <int D>
__global__ void __launch_bounds__(kCThreads) cache_read_kernel(const CacheRowsArgs a) {
  constexpr int kB = D / kFp4Block;
  pdl_wait_prior_grid();
  const int per_token = 2 * a.c.heads * kB;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kCThreads + threadIdx.x;
  const int t = static_cast<int>(i / per_token), r = static_cast<int>(i % per_token);
  if (t >= a.T) return;
  const int j = r % kB, h = (r / kB) % a.c.heads, kind = r / (kB * a.c.heads);
  Place p{0, 0};
  const int found = find_place(a, t, p);
  if (found == -1) return;
  uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (found == 0) {
    const int64_t src = ((static_cast<int64_t>(p.page) * 2 + kind) * a.c.heads + h) * a.c.page + p.off;
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(a.c.q + src * (D / 2) + j * 8));
    const uint32_t s2 = e4m3x2_to_f16x2(a.c.bs[src * kB + j] * 0x0101u);
    const float rs = a.c.rs[src];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t v[4], w[4];
      e2m1x8_to_f16x2x4(e == 0 ? c.x : c.y, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = f16x2_mul(v[k], s2);  // exact
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
            : "=r"(w[k])
            : "f"(__fmul_rn(f16_hi(x), rs)), "f"(__fmul_rn(f16_lo(x), rs)));
      }
      o[e] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else if (j == 0) {
    store_status(a.status, MTP_ERR_ARG);
  }
  uint16_t* dst = (kind == 0 ? a.k_out + t * a.ld_k : a.v_out + t * a.ld_v) + h * D + j * kFp4Block;
  __stcs(reinterpret_cast<uint4*>(dst), o[0]);
  __stcs(reinterpret_cast<uint4*>(dst) + 1, o[1]);
}

cudaError_t launch_rows(const void* kern, const CacheRowsArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const int64_t n = static_cast<int64_t>(a.T) * 2 * a.c.heads * (a.c.D / kFp4Block);
  CacheRowsArgs p = a;
  void* args[] = {&p};
  return launch_pdl(kern, dim3(static_cast<unsigned>((n + kCThreads - 1) / kCThreads)), dim3(kCThreads), 0, stream, args);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsArgs& a, cudaStream_t stream) {
  return launch_rows(a.c.D == 64 ? reinterpret_cast<const void*>(cache_write_kernel<64>)
                                 : reinterpret_cast<const void*>(cache_write_kernel<128>),
                     a, stream);
}
cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t stream) {
  return launch_rows(a.c.D == 64 ? reinterpret_cast<const void*>(cache_read_kernel<64>)
                                 : reinterpret_cast<const void*>(cache_read_kernel<128>),
                     a, stream);
}

}  // namespace mtp
