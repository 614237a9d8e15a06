// Rows of keys and values into the paged FP4 cache, and back to BF16.
//
// A row (one token, one head, key or value) is quantised by itself, in the format and with the
// roundings of the FP4 copies (codes.cuh): E2M1 codes, an E4M3 scale per 16 columns, an fp32 scale per
// row. A warp takes a token (where it lives is found once for all its heads), D / 16 lanes a row, one block of
// 16 columns each (32 bytes in, 8 bytes of codes and one of scale out), so a row's maximum is a few
// shuffles and a warp's loads and stores are contiguous over whole heads. Reading takes D / 8 lanes a row. Bound by
// bytes in principle: 4 D in and 2 (D/2 + D/16 + 4) out for a token's key and value of one head, or the other way round.
// Measured at 16384 tokens of 8 heads, D = 128 (87 MB each way): 36 us for a write and the read after it, 4.8 TB/s;
// writing is as much bound by its arithmetic (issue slots 56 % busy: correctly rounded quotients), reading by
// the latency of small pieces (a row is 64, 8 and 4 bytes in three places). Few tokens: a launch each.
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

// Where row t of the packed rows lives. 0: found; -1: the row belongs to no sequence; -2: its place does not exist.
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

// Row r of a token's 2 heads rows (keys first).
struct RowOf {
  int kind, h;
  __device__ __forceinline__ RowOf(int r, int heads) : kind(r >= heads ? 1 : 0), h(r >= heads ? r - heads : r) {}
};

// `parts` warps share a token (1, or as many as keep the GPU busy when there are few tokens).
template <int D>
__global__ void __launch_bounds__(kCThreads) cache_write_kernel(const CacheRowsArgs a, int parts) {
  constexpr int kB = D / kFp4Block;  // blocks (and lanes) of a row
  constexpr int kR = 32 / kB;        // rows of a warp at a time
  constexpr int kAhead = 2;          // of these, loads in flight
  pdl_wait_prior_grid();
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kCThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(wid / parts), part = static_cast<int>(wid % parts);
  if (t >= a.T) return;
  const int lane = threadIdx.x & 31, j = lane % kB;
  const int rows = 2 * a.c.heads;
  const uint16_t* k = a.k_in + t * a.ld_k + j * kFp4Block;
  const uint16_t* v = a.v_in + t * a.ld_v + j * kFp4Block;
  uint4 u[kAhead][2];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kR;
      const RowOf ro(r, a.c.heads);
      u[i][0] = u[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const uint4* src = reinterpret_cast<const uint4*>((ro.kind ? v : k) + ro.h * D);
        u[i][0] = __ldcs(src);
        u[i][1] = __ldcs(src + 1);
      }
    }
  };
  const int first = part * kR * kAhead + lane / kB;
  load(first);  // (under the search for the token's place)
  Place p{0, 0};
  const int found = find_place(a, t, p);
  if (found != 0) {
    if (found == -2 && lane == 0) store_status(a.status, MTP_ERR_ARG);
    return;
  }
  const int64_t dst0 = static_cast<int64_t>(p.page) * 2 * a.c.heads * a.c.page + p.off;  // its first row in the page
  for (int r0 = first; r0 - lane / kB < rows; r0 += parts * kR * kAhead) {
    if (r0 != first) load(r0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kR;
      const uint32_t m = mag_max(mag_max(0u, u[i][0]), u[i][1]);
      uint32_t mx = max(m & 0xFFFFu, m >> 16);
#pragma unroll
      for (int s = kB / 2; s > 0; s >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      if (r >= rows) continue;
      float rs = __fdiv_rn(bf16_bits_to_f32(mx), 2688.0f);
      if (mx >= 0x7F80u) {  // a NaN or Inf in the row
        if (j == 0) store_status(a.status, MTP_ERR_NONFINITE);
        rs = 0.0f;
      }
      BlockCodes o{0u, 0u, 0u};
      if (rs > 0.0f) {
        const float r6 = rs >= kSmallRs ? recip(__fmul_rn(6.0f, rs)) : 0.0f;
        const float off = __fmaf_rn(rs, 2688.0f, -bf16_bits_to_f32(mx));  // its sign is that of the scale's rounding
        if (rs >= kSmallRs && off != 0.0f) {
          const float side = off > 0.0f ? kDn : kUp;
          o = block_codes_biased(u[i][0], u[i][1], rs, __fmul_rn(r6, side), side);
        } else {
          o = block_codes(u[i][0], u[i][1], rs, __fmul_rn(r6, kUp), __fmul_rn(r6, kDn));
        }
      }
      const int64_t dst = dst0 + r * a.c.page;
      *reinterpret_cast<uint2*>(a.c.q + dst * (D / 2) + j * 8) = make_uint2(o.c0, o.c1);
      a.c.bs[dst * kB + j] = static_cast<uint8_t>(o.sc);
      if (j == 0) a.c.rs[dst] = rs;
    }
  }
}

// Eight columns a lane: 4 bytes of codes in, 16 bytes out, neighbouring lanes neighbouring columns.
template <int D>
__global__ void __launch_bounds__(kCThreads, 6) cache_read_kernel(const CacheRowsArgs a, int parts) {
  constexpr int kL = D / 8;    // lanes of a row
  constexpr int kR = 32 / kL;  // rows of a warp at a time
  constexpr int kAhead = 4;
  pdl_wait_prior_grid();
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * kCThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(wid / parts), part = static_cast<int>(wid % parts);
  if (t >= a.T) return;
  const int lane = threadIdx.x & 31, j = lane % kL;
  Place p{0, 0};
  const int found = find_place(a, t, p);
  if (found == -1) return;
  if (found == -2 && lane == 0) store_status(a.status, MTP_ERR_ARG);
  const int rows = 2 * a.c.heads;
  uint16_t* k = a.k_out + t * a.ld_k + j * 8;
  uint16_t* v = a.v_out + t * a.ld_v + j * 8;
  const int64_t src0 = static_cast<int64_t>(p.page) * 2 * a.c.heads * a.c.page + p.off;
  for (int r0 = part * kR * kAhead + lane / kL; r0 < rows; r0 += parts * kR * kAhead) {
    uint32_t c[kAhead], sc[kAhead];
    float rs[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kR;
      const int64_t src = src0 + r * a.c.page;
      c[i] = sc[i] = 0u;  // (a row without a place: zeros)
      rs[i] = 0.0f;
      if (r < rows && found == 0) {
        c[i] = __ldcs(reinterpret_cast<const uint32_t*>(a.c.q + src * (D / 2)) + j);
        sc[i] = a.c.bs[src * (D / kFp4Block) + (j >> 1)];
        rs[i] = a.c.rs[src];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kR;
      if (r >= rows) continue;
      const RowOf ro(r, a.c.heads);
      const uint32_t s2 = e4m3x2_to_f16x2(sc[i] * 0x0101u);
      uint32_t x[4], w[4];
      e2m1x8_to_f16x2x4(c[i], x);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint32_t y = f16x2_mul(x[n], s2);  // exact
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
            : "=r"(w[n])
            : "f"(__fmul_rn(f16_hi(y), rs[i])), "f"(__fmul_rn(f16_lo(y), rs[i])));
      }
      __stcs(reinterpret_cast<uint4*>((ro.kind ? v : k) + ro.h * D), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

cudaError_t launch_rows(const void* kern, int rows_at_once, const CacheRowsArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  // few tokens: a warp for every batch of rows
  int parts = (2 * a.c.heads + rows_at_once - 1) / rows_at_once;
  const int64_t busy = static_cast<int64_t>(di.sm_count) * 32;
  while (parts > 1 && a.T * static_cast<int64_t>(parts) > busy) parts = (parts + 1) / 2;
  const int64_t warps = static_cast<int64_t>(a.T) * parts;
  CacheRowsArgs p = a;
  void* args[] = {&p, &parts};
  return launch_pdl(kern, dim3(static_cast<unsigned>((warps * 32 + kCThreads - 1) / kCThreads)), dim3(kCThreads), 0, stream, args);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRowsArgs& a, cudaStream_t stream) {
  return launch_rows(a.c.D == 64 ? reinterpret_cast<const void*>(cache_write_kernel<64>)
                                 : reinterpret_cast<const void*>(cache_write_kernel<128>),
                     2 * 512 / a.c.D, a, stream);
}
cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t stream) {
  return launch_rows(a.c.D == 64 ? reinterpret_cast<const void*>(cache_read_kernel<64>)
                                 : reinterpret_cast<const void*>(cache_read_kernel<128>),
                     4 * 256 / a.c.D, a, stream);
}

}  // namespace mtp
