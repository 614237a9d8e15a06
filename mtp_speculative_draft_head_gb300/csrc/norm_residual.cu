// The residual's addition, the norm of the sum, and an E4M3 copy of the normalised rows:
//   s = bf16( x + delta )                                  (the real sum rounded once; s = x without a delta)
//   y = bf16( s w / sqrt(mean s^2 + eps) )                 rms_norm_vanilla, as everywhere in this library
//   scale = fp32( max |y| / 448 ),  q = e4m3( fp32( y / scale ) )    of each row, or of 128 columns of it
//
// One read of x and delta: a row stays in the registers of the threads that share it, between the
// sum of its squares and the results. Sums of squares are double-floats of exact squares, 1/rms is
// formed in fp64, and y is rounded once from a double-float: y is the same whatever the number of
// threads. A row's squares leave the fp32 range beyond 2^64 or below 2^-75; such a row's sum is taken
// once more of 2^-80 or 2^80 of its elements, and its y is formed in fp64, as is an element's of any row
// whose factors leave the normal fp32 range on the way.
//
// Measured: 4096 rows of 6144 columns with all three outputs (227 MB) 46 us, 4.9 TB/s where a copy makes 6.7; a row that is not
// a multiple of 8 long costs its edges (1021 rows of 5003 columns without delta and codes, 20 MB: 10 us); 16 rows 5 us, a launch. Instructions bound
// the long rows (issue slots 64 % busy), the double-floats of exact squares among them, and the barriers between a row's phases.
#include <cuda_runtime.h>
#include <stdint.h>

#include "codes.cuh"
#include "common.cuh"
#include "internal.h"
#include "layer.h"
#include "tc.cuh"

namespace mtp {

namespace {

// Eight columns from c0 of a row that starts at flat element `at` of a 16-byte aligned array; at + c0 is a
// multiple of 8. Columns outside [0, H) are zeros and not read.
__device__ __forceinline__ uint4 load8(const uint16_t* base, int64_t at, int c0, int H) {
  const uint16_t* p = base + at + c0;
  if (c0 >= 0 && c0 + 8 <= H) return __ldcs(reinterpret_cast<const uint4*>(p));
  uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + i >= 0 && c0 + i < H) u[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(uint16_t* base, int64_t at, int c0, int H, const uint32_t (&u)[4]) {
  uint16_t* p = base + at + c0;
  if (c0 >= 0 && c0 + 8 <= H) {
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + i >= 0 && c0 + i < H) p[i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
}

// bf16( a + b ) of two BF16 pairs. The fp32 sum in between does no harm: it is inexact only when one number is below
// 2^-16 of the other, and then the sum is nowhere near a midpoint of BF16 values.
__device__ __forceinline__ uint32_t add_pair(uint32_t a, uint32_t b) {
  const uint64_t s = f2_add(bf16x2_to_f2(a), bf16x2_to_f2(b));
  uint32_t o;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(f2_hi(s)), "f"(f2_lo(s)));
  return o;
}
// bf16( x w r ) in fp64: x w is exact, so the product is within two roundings of 2^-53 of the real one. Rounded to odd on the
// way to fp32, so that the rounding to BF16 is that of the product. (A zero, the common case of such rows, costs nothing.)
__device__ __forceinline__ uint32_t scaled_fp64(float x, float w, double r) {
  if (x == 0.0f && fabsf(w) < __int_as_float(0x7f800000) && r < __longlong_as_double(0x7ff0000000000000ll))
    return (__float_as_uint(x) ^ __float_as_uint(w)) >> 16 & 0x8000u;
  const float f = to_odd(static_cast<double>(x) * static_cast<double>(w) * r);
  return f != f ? 0x7FC0u : bf16_bits_rn(f);
}

// 1 / rms of a row: up (rh + rl) with up a power of two and rh in [1, 2) where fp32 holds the sum of its squares, else up is 0 and
// rh and rl are the upper and lower half of its bits in fp64.
struct Root {
  float rh, rl, up;
};
__device__ __forceinline__ Root root_fp64(double r) {
  return Root{__int_as_float(__double2hiint(r)), __int_as_float(__double2loint(r)), 0.0f};
}
// a + b (|b| below a few units of a) rounded to odd: the neighbour nearer zero, its last bit set where that is not the sum. A
// following rounding to BF16 is that of the sum, without a branch.
__device__ __forceinline__ float sum_to_odd(float a, float b) {
  float s, err;
  two_sum(a, b, s, err);
  const uint32_t u = __float_as_uint(s);
  const uint32_t back = err != 0.0f && ((__float_as_uint(err) ^ u) >> 31) != 0u ? 1u : 0u;
  return __uint_as_float((u - back) | (err != 0.0f ? 1u : 0u));
}
// Eight columns by fp64; out of line, as it is long.
static __device__ __noinline__ uint4 scaled8_fp64(uint4 x, uint4 w, double d) {
  const uint32_t xu[4] = {x.x, x.y, x.z, x.w}, wu[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
    o[t] = scaled_fp64(bf16_lo(xu[t]), bf16_lo(wu[t]), d) | (scaled_fp64(bf16_hi(xu[t]), bf16_hi(wu[t]), d) << 16);
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// The eight anew. (Without a branch, and the fp64 part apart from it: a CTA waits for its slowest warp, and one in fifty comes
// here. With both in one place, 4096 rows of 6144 columns took 48 us, and 46 so.)
static __device__ __noinline__ uint4 scaled_exact(uint4 x, uint4 w, Root r) {
  const uint32_t xu[4] = {x.x, x.y, x.z, x.w}, wu[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4];
  float lo = __int_as_float(0x7f800000), hi = 0.0f;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    float z[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float p = __fmul_rn(__fmul_rn(e ? bf16_hi(xu[t]) : bf16_lo(xu[t]), r.up), e ? bf16_hi(wu[t]) : bf16_lo(wu[t]));
      const float yh = __fmul_rn(p, r.rh), yl = __fmaf_rn(p, r.rl, __fmaf_rn(p, r.rh, -yh));
      lo = fminf(lo, fabsf(yh)), hi = fmaxf(hi, fabsf(yh));
      z[e] = sum_to_odd(yh, yl);
    }
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[t]) : "f"(z[1]), "f"(z[0]));
  }
  // (double-floats hold it from 2^-101 on, where their parts are normal numbers)
  if (r.up != 0.0f && lo >= 0x1p-101f && hi < 0x1p127f) return make_uint4(o[0], o[1], o[2], o[3]);
  const double d = r.up != 0.0f ? (static_cast<double>(r.rh) + static_cast<double>(r.rl)) * static_cast<double>(r.up)
                                : __hiloint2double(__float_as_int(r.rh), __float_as_int(r.rl));
  return scaled8_fp64(x, w, d);
}
// Whether an x of the eight is not zero and x up is below 2^-142 (a power of two times eight bits from there on is exact).
__device__ __forceinline__ bool tiny_among(const uint32_t (&x)[4], float up) {
  bool some = false;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = fabsf(e ? bf16_hi(x[t]) : bf16_lo(x[t]));
      some |= v != 0.0f && __fmul_rn(v, up) <= 0x1p-142f;  // (at it: rounded up, perhaps)
    }
  return some;
}
// bf16( x w up (rh + rl) ) of eight columns: the fp32 product yh = ((x up) w) rh decides unless its low half is within two units
// of a BF16 midpoint; such a cell is redone as a whole, out of line. x up is at most sqrt(H) and p = (x up) w within a factor of
// two of y, so each leaves the fp32 range only where y does: both are exact (8 and 16 bits) but for p below 2^-134, which
// is off by half a unit of 2^-149, and yh is within 1.5 units of y. x up is not exact below 2^-142 (in rows with an rms of 2^9
// or more only): such an x becomes 0 with a weight below 2, and is redone with others.
__device__ __forceinline__ uint4 scaled(const uint32_t (&x)[4], const uint64_t (&w)[4], const Root& r) {
  const uint64_t r2 = f2_pack(r.rh, r.rh), up2 = f2_pack(r.up, r.up);
  uint32_t o[4], near = 0xFFFFFFFFu;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint64_t y = f2_mul(f2_mul(f2_mul(bf16x2_to_f2(x[t]), up2), w[t]), r2);
    const uint32_t lo = static_cast<uint32_t>(y), hi = static_cast<uint32_t>(y >> 32);
    near = min(near, min((lo - 0x7FFEu) << 16, (hi - 0x7FFEu) << 16));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[t]) : "f"(f2_hi(y)), "f"(f2_lo(y)));
  }
  bool redo = near <= 0x40000u;
  if (r.up < 0x1p-9f) {  // (the whole row alike)
    uint32_t any = 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t) any |= static_cast<uint32_t>(w[t]) | static_cast<uint32_t>(w[t] >> 32);
    redo |= r.up == 0.0f || ((any & 0x40000000u) != 0u && tiny_among(x, r.up));  // (the bit of magnitudes from 2 on)
  }
  if (redo) {
    auto pair = [](uint64_t v) { return __byte_perm(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32), 0x7632); };
    return scaled_exact(make_uint4(x[0], x[1], x[2], x[3]), make_uint4(pair(w[0]), pair(w[1]), pair(w[2]), pair(w[3])), r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Groups of a row that TPR threads hold in P pieces each, at most.
constexpr int max_groups(int tpr, int p) { return tpr * p * 8 / kNormGroup + 2; }

// TPR threads per row (a warp, or the whole CTA), P pieces of eight columns a thread. VEC: H is a
// multiple of 8. Otherwise pieces follow the arrays' 16-byte boundaries: a row's first and last may
// be partial, and w, q and the scales' groups are not aligned with them.
template <int TPR, int P, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, TPR == 256 && P <= 3 ? (VEC ? 5 : 4) : 1) norm_residual_kernel(const NormResidualArgs a) {
  // sums of the threads, then (not VEC, group > 0) the groups' maxima [kRows][kMaxGroups]
  extern __shared__ __align__(16) uint8_t dyn[];
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kWarpsHere = kThreads / 32;
  constexpr int kRows = kThreads / TPR;
  constexpr int kMaxGroups = max_groups(TPR, P);
  static_assert(TPR == 32 || kRows == 1, "a warp or a CTA per row");
  __shared__ float red[4];
  __shared__ uint32_t redm[kWarpsHere];
  float2* sums = reinterpret_cast<float2*>(dyn);  // TPR > 32: [kThreads]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  pdl_wait_prior_grid();
  if (row >= a.R) return;  // (whole warps: only where no CTA barrier follows)
  const int H = a.H;
  const int64_t at = row * H;
  const int off = VEC ? 0 : static_cast<int>(at & 7);
  auto row_sync = [] {
    if constexpr (TPR == 32)
      __syncwarp();
    else
      __syncthreads();
  };

  // ---- s
  uint32_t s[P][4];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c0 = 8 * (t + i * TPR) - off;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (c0 < H) v = load8(a.x, at, c0, H);
    s[i][0] = v.x, s[i][1] = v.y, s[i][2] = v.z, s[i][3] = v.w;
  }
  if (a.delta != nullptr) {
    uint4 d[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c0 = 8 * (t + i * TPR) - off;
      d[i] = make_uint4(0u, 0u, 0u, 0u);
      if (c0 < H) d[i] = load8(a.delta, at, c0, H);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      s[i][0] = add_pair(s[i][0], d[i].x);
      s[i][1] = add_pair(s[i][1], d[i].y);
      s[i][2] = add_pair(s[i][2], d[i].z);
      s[i][3] = add_pair(s[i][3], d[i].w);
    }
  }
  if (a.total != nullptr) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c0 = 8 * (t + i * TPR) - off;
      if (c0 < H) store8(a.total, at, c0, H, s[i]);
    }
  }
  if (a.y == nullptr && a.q == nullptr) return;

  // ---- 1 / rms. A CTA's sums go through shared memory to its first warp: adding double-floats across lanes costs a warp as
  // much as ten elements a lane, so one warp does it for all (and with it the one fp64 reciprocal root of the row).
  auto sum_squares = [&](float times) -> DF {  // of the elements times a power of two; TPR > 32: of warp 0 only
    DF2 acc{0ull, 0ull};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t f = bf16x2_to_f2(s[i][e]);
        if (times != 1.0f) f = f2_mul(f, f2_pack(times, times));
        df2_add(acc, f2_mul(f, f));
      }
    DF v = df_add(df2_x(acc), df2_y(acc));
    if constexpr (TPR > 32) {
      sums[threadIdx.x] = make_float2(v.hi, v.lo);
      __syncthreads();
      if (warp == 0) {
        for (int i = 1; i < kWarpsHere; ++i) {
          const float2 u = sums[32 * i + lane];
          v = df_add(v, DF{u.x, u.y});
        }
      }
    }
    if (TPR == 32 || warp == 0) {
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) v = df_add(v, shfl_xor_df(v, m));
    }
    return v;
  };
  auto root64 = [&](const DF& v, double factor2) {  // 1 / sqrt(mean + eps factor2), within an ulp or two of fp64
    const double ms = (static_cast<double>(v.hi) + static_cast<double>(v.lo)) * a.inv_h;
    return rsqrt(ms + static_cast<double>(a.eps) * factor2);
  };
  auto root = [&](const DF& v) {
    if (!(v.hi >= 0x1p-100f && v.hi < __int_as_float(0x7f800000))) return Root{1.0f, 0.0f, 0.0f};
    const double r = root64(v, 1.0);
    const float hi = static_cast<float>(r);
    const uint32_t e = __float_as_uint(hi) & 0x7F800000u;  // (2^-64 to 2^58)
    const float down = __uint_as_float(0x7F000000u - e);
    return Root{__fmul_rn(hi, down), __fmul_rn(static_cast<float>(r - static_cast<double>(hi)), down), __uint_as_float(e)};
  };
  DF tot = sum_squares(1.0f);
  Root r;
  if constexpr (TPR == 32) {
    r = root(tot);
  } else {
    if (threadIdx.x == 0) {
      const Root of = root(tot);
      red[0] = of.rh;
      red[1] = of.rl;
      red[2] = of.up;
    }
    __syncthreads();
    r = Root{red[0], red[1], red[2]};
  }
  if (r.up == 0.0f) {  // (the whole row alike) squares beyond fp32, or infinities or NaN among them
    uint32_t nan = 0u, inf = 0u, top = 0u;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      top = mag_max(top, make_uint4(s[i][0], s[i][1], s[i][2], s[i][3]));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = s[i][e] & 0x7FFFu, hi = (s[i][e] >> 16) & 0x7FFFu;
        nan |= (lo > 0x7F80u || hi > 0x7F80u) ? 1u : 0u;
        inf |= (lo == 0x7F80u || hi == 0x7F80u) ? 1u : 0u;
      }
    }
    uint32_t flags = __reduce_or_sync(0xffffffffu, nan | (inf << 1));
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    if constexpr (TPR > 32) {
      if (lane == 0) redm[warp] = flags | (top << 2);
      __syncthreads();
      flags = 0u, top = 0u;
      for (int i = 0; i < kWarpsHere; ++i) {
        flags |= redm[i] & 3u;
        top = max(top, redm[i] >> 2);
      }
    }
    const bool big = top >= 0x5000u;  // (2^33; squares of smaller rows do not overflow)
    const float f = big ? 0x1p-80f : 0x1p80f;
    tot = sum_squares(f);
    // an infinity makes the mean infinite (finite columns become 0), a NaN makes it NaN
    if (flags != 0u) tot = DF{__int_as_float((flags & 1u) ? 0x7fc00000 : 0x7f800000), 0.0f};
    const double factor2 = big ? 0x1p-160 : 0x1p160;
    if constexpr (TPR == 32) {
      r = root_fp64(root64(tot, factor2) * static_cast<double>(f));
    } else {
      if (threadIdx.x == 0) {
        const Root of = root_fp64(root64(tot, factor2) * static_cast<double>(f));
        red[0] = of.rh;
        red[1] = of.rl;
      }
      __syncthreads();
      r = Root{red[0], red[1], 0.0f};
    }
    if (flags == 0u && top == 0u && a.eps > 0.0f) r = Root{1.0f, 0.0f, 1.0f};  // a row of zeros stays one
  }

  // ---- y (in the place of s)
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c0 = 8 * (t + i * TPR) - off;
    if (c0 >= H) continue;
    uint64_t w[4];
    if constexpr (VEC) {
      const uint4 w4 = *reinterpret_cast<const uint4*>(a.w + c0);
      w[0] = bf16x2_to_f2(w4.x), w[1] = bf16x2_to_f2(w4.y), w[2] = bf16x2_to_f2(w4.z), w[3] = bf16x2_to_f2(w4.w);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = f2_pack(c0 + 2 * e >= 0 && c0 + 2 * e < H ? bf16_bits_to_f32(a.w[c0 + 2 * e]) : 0.0f,
                       c0 + 2 * e + 1 >= 0 && c0 + 2 * e + 1 < H ? bf16_bits_to_f32(a.w[c0 + 2 * e + 1]) : 0.0f);
    }
    const uint4 o = scaled(s[i], w, r);
    s[i][0] = o.x, s[i][1] = o.y, s[i][2] = o.z, s[i][3] = o.w;
    if constexpr (!VEC) {  // (a NaN factor leaves a NaN in the columns that are not the row's)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e < 0 || c0 + e >= H) s[i][e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
    if (a.y != nullptr) store8(a.y, at, c0, H, s[i]);
  }
  if (a.q == nullptr) return;

  // ---- the 8-bit copy
  // fp32( mx / 448 ), 0 for a NaN or Inf among the columns
  auto scale_value = [](uint32_t mx) {
    const float w = bf16_bits_to_f32(mx);
    if (mx < 0x1000u) return __fdiv_rn(w, 448.0f);  // (below 2^-95)
    const float q = __fmul_rn(w, 1.0f / 448.0f);    // one step from the product is the rounded quotient (codes.cuh)
    return mx >= 0x7F80u ? 0.0f : __fmaf_rn(__fmaf_rn(-q, 448.0f, w), 1.0f / 448.0f, q);
  };
  auto scale_of = [&](uint32_t mx) {
    if (mx >= 0x7F80u) store_status(a.status, MTP_ERR_NONFINITE);
    return scale_value(mx);
  };
  auto store_codes = [&](int c0, uint2 c) {
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(a.q + at + c0) = c;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e >= 0 && c0 + e < H) a.q[at + c0 + e] = static_cast<uint8_t>((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
    }
  };
  if (a.group == 0) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (8 * (t + i * TPR) - off < H) m = mag_max(m, make_uint4(s[i][0], s[i][1], s[i][2], s[i][3]));
    }
    uint32_t mx = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    if constexpr (TPR > 32) {
      if (lane == 0) redm[warp] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarpsHere; ++i) mx = max(mx, redm[i]);
    }
    const float sc = scale_value(mx);
    if (t == 0) a.q_scale[row] = scale_of(mx);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c0 = 8 * (t + i * TPR) - off;
      if (c0 < H) store_codes(c0, codes_e4m3x8(s[i], sc));
    }
    return;
  }
  const int groups = (H + kNormGroup - 1) / kNormGroup;
  float* scales = a.q_scale + row * groups;
  if constexpr (VEC) {
    // sixteen neighbouring lanes hold a group
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c0 = 8 * (t + i * TPR);
      uint32_t m = 0u;
      if (c0 < H) m = mag_max(0u, make_uint4(s[i][0], s[i][1], s[i][2], s[i][3]));
      uint32_t mx = max(m & 0xFFFFu, m >> 16);
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float sc = scale_value(mx);
      if (c0 < H) {
        if ((lane & 15) == 0) scales[c0 / kNormGroup] = scale_of(mx);
        store_codes(c0, codes_e4m3x8(s[i], sc));
      }
    }
  } else {
    // a piece meets at most two groups; the groups' maxima in shared memory
    uint32_t* gm = reinterpret_cast<uint32_t*>(dyn + (TPR > 32 ? kThreads * 8 : 0)) + (threadIdx.x / TPR) * kMaxGroups;
    for (int g = t; g < groups; g += TPR) gm[g] = 0u;
    row_sync();
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c0 = 8 * (t + i * TPR) - off;
      if (c0 >= H) continue;
      const int g0 = c0 < 0 ? 0 : c0 / kNormGroup;
      uint32_t m0 = 0u, m1 = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t v = (s[i][e >> 1] >> (16 * (e & 1))) & 0x7FFFu;
        if (c0 + e < (g0 + 1) * kNormGroup)
          m0 = max(m0, v);
        else
          m1 = max(m1, v);
      }
      atomicMax(&gm[g0], m0);
      if (m1 != 0u) atomicMax(&gm[g0 + 1], m1);
    }
    row_sync();
    for (int g = t; g < groups; g += TPR) scales[g] = scale_of(gm[g]);
    auto at_group = [&](int g) {
      return scale_value(g < groups ? gm[g] : 0u);
    };
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c0 = 8 * (t + i * TPR) - off;
      if (c0 >= H) continue;
      const int g0 = c0 < 0 ? 0 : c0 / kNormGroup;
      uint2 c = codes_e4m3x8(s[i], at_group(g0));
      const int n0 = (g0 + 1) * kNormGroup - c0;  // columns of the piece in its first group
      if (n0 < 8) {
        const uint2 d = codes_e4m3x8(s[i], at_group(g0 + 1));
        const uint64_t keep = (1ull << (8 * n0)) - 1ull;
        const uint64_t both = ((static_cast<uint64_t>(c.y) << 32 | c.x) & keep) | ((static_cast<uint64_t>(d.y) << 32 | d.x) & ~keep);
        c = make_uint2(static_cast<uint32_t>(both), static_cast<uint32_t>(both >> 32));
      }
      store_codes(c0, c);
    }
  }
}

template <int TPR, int P>
cudaError_t launch_form(const NormResidualArgs& a, cudaStream_t stream) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  const bool vec = a.H % 8 == 0;
  const void* kern = vec ? reinterpret_cast<const void*>(norm_residual_kernel<TPR, P, true>)
                                  : reinterpret_cast<const void*>(norm_residual_kernel<TPR, P, false>);
  const int rows = kThreads / TPR;
  const size_t smem = (TPR > 32 ? kThreads * 8 : 0) + (vec || a.group == 0 ? 0 : static_cast<size_t>(rows) * max_groups(TPR, P) * 4);
  NormResidualArgs p = a;
  void* args[] = {&p};
  return launch_pdl(kern, dim3(static_cast<unsigned>((a.R + rows - 1) / rows)), dim3(kThreads), smem, stream, args);
}

}  // namespace

cudaError_t launch_norm_residual(const NormResidualArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const int pieces = a.H % 8 == 0 ? a.H / 8 : (a.H + 14) / 8;  // of a row, at most
  if (pieces > 1024) return launch_form<512, 17>(a, stream);
  if (a.R <= di.sm_count && pieces > 256) return launch_form<1024, 1>(a, stream);
  if (pieces <= 128) return launch_form<32, 4>(a, stream);
  // as few registers as hold the row: more rows of an SM are in flight
  if (pieces <= 256) return launch_form<256, 1>(a, stream);
  if (pieces <= 512) return launch_form<256, 2>(a, stream);
  if (pieces <= 768) return launch_form<256, 3>(a, stream);
  return launch_form<256, 4>(a, stream);
}

}  // namespace mtp
