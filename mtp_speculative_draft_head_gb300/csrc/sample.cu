// Drafts drawn by sampling, and the acceptance of drafts.
//
// sample: one token per row of logits, by inversion of the cumulative distribution. With
// m = max_i l_i the weight of token i is w_i = exp((l_i - m) / T). Sorted by (logit descending,
// index ascending), the tokens kept are a prefix of that order: the first top_k; of those, the ones
// whose preceding mass is below top_p times the mass of all of them; of those, the ones with
// l_i >= m + T ln(min_p). The token is the lowest index whose cumulative kept mass, in index order,
// exceeds u times the whole.
//
// No sort of the row: a prefix is { i : key_i >= cut } for one 64-bit key (the logit's order bits,
// then the complement of the index). Two ways to the cut:
//  * a top_k whose entries fit one list (the usual case; up to 780 with four CTAs a row, 910 with 16, half the
//    threads of a single one): the k-th largest of the threads' own maxima
//    is a bound that the k-th largest logit cannot be below, and little more than k entries reach it.
//    These are gathered and sorted by one CTA, which finishes the row on the sorted list: no weight is
//    formed for any other entry, and shared-memory atomics (~50 cycles for a warp's worth, the cost
//    of a histogram of the whole row) are spent on one entry per thread.
//  * otherwise by a histogram of the row's masses (or entries) over the distance from the maximum, in 2048
//    bins over the distances at which a weight is more than nothing (entries further down, masked ones
//    among them, are left out of it). The bin that holds the cut is gathered and sorted when it has at
//    most kGather entries, and split by the key's bits, 11 at a time, until it has.
//
// Masses are 64-bit fixed-point numbers (2^62 / 2^ceil(log2 V) for a weight of one), so sums do not
// depend on the order of the atomics or of the threads: the same inputs give the same token
// whatever the cluster size. Each is off by half a unit at most, all together by V^2 2^-62 of a whole of at
// least one; beyond 2^20 tokens, where that passes 2^-22, a first sum of the row tells how much room it takes
// (a filter keeps the n largest weights of such a row; their n half units stay below V 2^-61 of their own sum). Weights are formed in fp32 from an exponent kept as a double-float:
// relative error ~2^-23, against the 2^-24 of the given random numbers.
//
// A cluster of CTAs shares a row; maxima, histograms and masses are combined through distributed
// shared memory. A slice is kept in shared memory where it fits beside the histograms, and is read
// again, from L2 mostly, where it does not (many rows).
//
// Measured at V = 154880: one row with top_k and top_p 12.6 to 16.6 us (as long as its list makes it), 16 BF16 rows
// with top_p 50 to 55 us (the distribution stored), 80 rows with both 49 us; bound by latency: exchanges of the cluster
// (1 to 1.5 us each), and with top_p alone the histogram (8 us of a row's 23: two atomics or one per entry, 1 to 1.5
// cycles a lane). A row of 2,000,000 with top_p 177 us, 35 of them its first sum. 16 sequences of the acceptance 14.6 us.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "sample.h"

namespace mtp {

namespace {

constexpr int kT = 512;           // threads per CTA
constexpr int kW = kT / 32;
constexpr int kMaxC = 16;         // CTAs per cluster
constexpr int kBins = 2048;
constexpr int kGather = 1024;     // candidates sorted at once
constexpr int kSliceUnit = 4 * kT;  // a slice is a multiple of this: every warp owns whole steps of 128 elements

typedef unsigned long long u64;

// ------------------------------------------------------------------------------- cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// "This CTA runs" (its shared memory may be written), said early; and the wait for all of them to have said it,
// before the first write to another's (one full barrier between the pass over the row and the exchange less: one
// row 12.4 -> 12.0 us, the acceptance of four sequences 9.4 -> 9.0).
__device__ __forceinline__ void cluster_here() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_here() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_peer32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ u64 ld_peer(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_peer32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
__device__ __forceinline__ u64 warp_inclusive(u64 v, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  return v;
}

// ------------------------------------------------------------------------------- numbers
// floor(u * z) for u in [0, 1); -0 is 0.
__device__ __forceinline__ u64 scale_floor(float u, u64 z) {
  const uint32_t b = __float_as_uint(u) & 0x7FFFFFFFu;
  const int e = static_cast<int>(b >> 23);
  const u64 m = e == 0 ? (b & 0x7FFFFFu) : ((b & 0x7FFFFFu) | 0x800000u);
  const int sh = 150 - (e == 0 ? 1 : e);  // u = m 2^-sh, sh >= 24
  const u64 hi = __umul64hi(m, z), lo = m * z;
  if (sh >= 128) return 0ull;
  if (sh >= 64) return hi >> (sh - 64);
  return (hi << (64 - sh)) | (lo >> sh);
}

// Whether part < p * whole, for 0 <= p < 1, exactly: part <= floor(p whole) unless p whole is whole.
__device__ __forceinline__ u64 scale_ceil(float p, u64 z) {
  const uint32_t b = __float_as_uint(p) & 0x7FFFFFFFu;
  const int e = static_cast<int>(b >> 23);
  const u64 m = e == 0 ? (b & 0x7FFFFFu) : ((b & 0x7FFFFFu) | 0x800000u);
  const int sh = 150 - (e == 0 ? 1 : e);
  const u64 hi = __umul64hi(m, z), lo = m * z;
  if (sh >= 128) return (hi | lo) ? 1ull : 0ull;
  if (sh >= 64) {
    const u64 q = hi >> (sh - 64);
    const u64 rem = (sh == 64 ? 0ull : hi << (128 - sh)) | lo;
    return q + (rem ? 1ull : 0ull);
  }
  const u64 q = (hi << (64 - sh)) | (lo >> sh);
  return q + ((lo << (64 - sh)) ? 1ull : 0ull);
}

// Order of floats as unsigned numbers (no NaN); -0 is taken as +0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// m 2^s to nearest, as a 64-bit number, for m < 2^24 and s <= 39.
__device__ __forceinline__ u64 shift_round(uint32_t m, int s) {
  const int up = s > 0 ? s : 0;
  const int dn = s < 0 ? (s > -31 ? -s : 31) : 0;
  return static_cast<u64>((m + ((1u << dn) >> 1)) >> dn) << up;
}

// exp(-(m - l) / T) for l <= m: the difference exactly (TwoSum), times log2(e) / T as a double-float,
// split into a whole power of two and 2^f, |f| <= 1/2, by the exponential series (eight terms:
// remainder 0.3466^8 / 8! < 2^-27). As a float, or as a fixed-point mass.
struct Weigh {
  float m, ch, cl;
  int frac;
  // 2^f's float and the whole power n: the weight is p 2^-n; false: nothing (below 2^-120, or no distance)
  __device__ __forceinline__ bool parts(float l, float& p, int& n) const {
    float dh, dl;
    two_sum(m, -l, dh, dl);
    float th = __fmul_rn(dh, ch);
    float tl = __fmaf_rn(dh, ch, -th) + __fmaf_rn(dh, cl, __fmul_rn(dl, ch));
    const bool some = th < 120.0f;  // (not for NaN: an infinite distance)
    th = some ? th : 0.0f;
    tl = some ? tl : 0.0f;
    const float r = rintf(th);
    n = static_cast<int>(r);
    const float y = ((r - th) - tl) * 0.69314718055994530942f;
    p = 1.0f / 5040.0f;
    p = __fmaf_rn(p, y, 1.0f / 720.0f);
    p = __fmaf_rn(p, y, 1.0f / 120.0f);
    p = __fmaf_rn(p, y, 1.0f / 24.0f);
    p = __fmaf_rn(p, y, 1.0f / 6.0f);
    p = __fmaf_rn(p, y, 0.5f);
    p = __fmaf_rn(p, y, 1.0f);
    p = __fmaf_rn(p, y, 1.0f);
    return some;
  }
  __device__ __forceinline__ float operator()(float l) const {
    float p;
    int n;
    const bool some = parts(l, p, n);
    const float w = __uint_as_float(__float_as_uint(p) - (static_cast<uint32_t>(n) << 23));
    return l == m ? 1.0f : (some ? w : 0.0f);
  }
  __device__ __forceinline__ u64 mass(float l) const {
    float p;
    int n;
    const bool some = parts(l, p, n) || l == m;  // (l = m = inf: distance NaN, p = 1, n = 0)
    const uint32_t b = __float_as_uint(p);       // 0.70 < p < 1.42
    const u64 w = shift_round((b & 0x7FFFFFu) | 0x800000u, static_cast<int>(b >> 23) - 150 + frac - n);
    return some ? w : 0ull;
  }
};

// ------------------------------------------------------------------------------- shared state
struct Shared {
  u64 wsum[kW];            // per-warp masses of this CTA
  u64 cta[kMaxC];          // every CTA's mass (pushed by its peers)
  uint32_t cmax[kMaxC];    // every CTA's largest / smallest logit (order bits)
  uint32_t cmin[kMaxC];
  uint32_t wmax[kW], wmin[kW];
  u64 scan[kW];
  uint32_t scan_n[kW];
  // the bin that holds the cut: number, entries and mass before it, its entries
  int hit;
  uint32_t before_n, hit_n;
  u64 before_m;
  uint32_t found;          // this CTA's candidates
  uint32_t counts[kMaxC];  // every CTA's candidates (pushed by its peers)
  u64 cut, cut_mass;       // published by the first CTA
  float ch, cl;            // log2(e) / T as a double-float
  float bh, bl;            // T ln(min_p) as a double-float
  float inv_z;
};
// Dynamic shared memory: Shared, the local histogram (u64 mass, u32 count), the cluster's, the
// gather buffer, then the slice.
constexpr size_t kHistBytes = kBins * 12;
constexpr size_t kFixedSmem = (sizeof(Shared) + 127) / 128 * 128 + 2 * kHistBytes + kGather * 8;

struct Hist {
  u64* mass;
  uint32_t* n;
};

// ------------------------------------------------------------------------------- inverse of the cdf
// The lowest index of the row whose cumulative mass exceeds floor(u z). Every warp owns `seg` consecutive
// elements of the slice that starts at i0 and ends by `end`; s.wsum holds this CTA's per-warp masses, s.cta
// every CTA's. The CTA that has it goes once more over the one warp's elements, a few consecutive ones a
// thread; the thread that finds it calls found(index). (By that warp alone, 128 elements at a time, this took
// longer than the pass over the whole slice.)
template <class MassFn, class Found>
__device__ void locate(Shared& s, uint32_t rank, u64 target, int64_t i0, int64_t seg, int64_t end, MassFn mass, Found found) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  u64 before = 0;
  for (uint32_t r = 0; r < rank; ++r) before += s.cta[r];
  int w = 0;
  if (target < before) return;  // an earlier CTA's
  while (w < kW && target - before >= s.wsum[w]) before += s.wsum[w++];
  if (w == kW) return;  // a later one's
  const int64_t b0 = i0 + w * seg, b1 = b0 + seg < end ? b0 + seg : end;
  const int64_t per = (seg + kT - 1) / kT;
  const int64_t t0 = b0 + tid * per, t1 = t0 + per < b1 ? t0 + per : b1;
  u64 sum = 0;
#pragma unroll 8
  for (int64_t i = t0; i < t1; ++i) sum += mass(i);
  const u64 inc = warp_inclusive(sum, lane);
  if (lane == 31) s.scan[warp] = inc;
  __syncthreads();
  before += inc - sum;
  for (int q = 0; q < warp; ++q) before += s.scan[q];
  if (target < before || target - before >= sum) return;
  for (int64_t i = t0; i < t1; ++i) {
    const u64 m = mass(i);
    if (target - before < m) {
      found(i);
      return;
    }
    before += m;
  }
}

// ------------------------------------------------------------------------------- sampler
// Sort, descending, of `size` (a power of two, 32 to kGather) 64-bit keys by the whole block; the keys other
// than 0 are distinct. Up to kT / 2 by counting; more by a bitonic sort, in which up to kT keys sit one to a
// thread: a step of distance below 32 is a shuffle, the others (10 of 45 at 512)
// go through shared memory. More sort in shared memory, where steps of distance up to 32 stay within
// the 64 keys of one warp's lanes.
__device__ void sort_desc(u64* key, int size) {
  const int tid = threadIdx.x;
  if (2 * size <= kT) {
    // few distinct keys (and zeros): each one's place is the number of larger ones, counted by two threads
    const u64 k = key[tid >> 1 & (size - 1)];
    uint32_t place = 0u;
    if (tid < 2 * size) {
      const ulonglong2* half = reinterpret_cast<const ulonglong2*>(key) + (tid & 1) * (size / 4);
#pragma unroll 4
      for (int j = 0; j < size / 4; ++j) {
        const ulonglong2 o = half[j];
        place += (o.x > k ? 1u : 0u) + (o.y > k ? 1u : 0u);
      }
      place += __shfl_xor_sync(0xffffffffu, place, 1);
    }
    __syncthreads();
    if (tid < size) key[tid] = 0ull;
    __syncthreads();
    if (tid < 2 * size && (tid & 1) == 0 && k != 0ull) key[place] = k;
    __syncthreads();
    return;
  }
  if (size <= kT) {
    const bool warp_on = (tid & ~31) < size;
    u64 k = warp_on ? key[tid] : 0ull;
    for (int w = 2; w <= size; w <<= 1)
      for (int d = w >> 1; d > 0; d >>= 1) {
        u64 o = 0ull;
        if (d >= 32) {
          __syncthreads();
          if (warp_on) key[tid] = k;
          __syncthreads();
          if (warp_on) o = key[tid ^ d];
        } else if (warp_on) {
          o = __shfl_xor_sync(0xffffffffu, k, d);
        }
        // the lower place of a descending run keeps the larger key
        const bool larger = ((tid & w) == 0) == ((tid & d) == 0);
        k = (o > k) == larger ? o : k;
      }
    __syncthreads();
    if (warp_on) key[tid] = k;
    __syncthreads();
    return;
  }
  for (int w = 2; w <= size; w <<= 1)
    for (int d = w >> 1; d > 0; d >>= 1) {
      for (int t = tid; t < size / 2; t += kT) {
        const int x = 2 * t - (t & (d - 1)), y = x + d;
        const u64 ka = key[x], kb = key[y];
        if ((ka < kb) == ((x & w) == 0)) {
          key[x] = kb;
          key[y] = ka;
        }
      }
      // the next step is (w, d / 2), or (2 w, w)
      if ((d > 1 ? d >> 1 : w) > 32) __syncthreads();
      else __syncwarp();
    }
  __syncthreads();
}

// LONG: a row of more than kLongRow tokens.
constexpr int64_t kLongRow = 1 << 20;
template <bool BF16, bool RES, bool LONG>
__global__ void __launch_bounds__(kT, 2) sample_kernel(const SampleArgs a, int nc, int64_t slice, int frac) {
  extern __shared__ __align__(128) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  uint8_t* p = dyn + (sizeof(Shared) + 127) / 128 * 128;
  Hist loc{reinterpret_cast<u64*>(p), reinterpret_cast<uint32_t*>(p + kBins * 8)};
  p += kHistBytes;
  Hist all{reinterpret_cast<u64*>(p), reinterpret_cast<uint32_t*>(p + kBins * 8)};
  p += kHistBytes;
  u64* cand = reinterpret_cast<u64*>(p);
  p += kGather * 8;
  float* res = reinterpret_cast<float*>(p);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = nc > 1 ? cluster_rank() : 0u;
  const int64_t row = blockIdx.x / nc;
  const int64_t V = a.V;
  const int64_t i0 = rank * slice;                       // this CTA's slice: [i0, i1)
  const int64_t i1 = i0 + slice < V ? i0 + slice : V;
  const int64_t seg = slice / kW;                        // elements per warp, a multiple of 32
  auto sync = [nc]() {
    if (nc > 1) cluster_sync_all();
    else __syncthreads();
  };
  for (int b = tid; b < kBins; b += kT) {
    loc.mass[b] = 0ull;
    loc.n[b] = 0u;
  }
  if (tid == 0) s.found = 0u;
  if (nc > 1) cluster_here();
  pdl_wait_prior_grid();

  // ---- the row's parameters
  float T = a.temperature ? a.temperature[row] : 1.0f;
  int64_t k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f;
  const float min_p = a.min_p ? a.min_p[row] : 0.0f;
  const float u = a.u ? a.u[row] : 0.0f;
  const bool bad = !(T >= 0.0f && T <= 3.402823466e38f) || !(top_p >= 0.0f) || !(min_p >= 0.0f && min_p <= 1.0f) ||
                   !(u >= 0.0f && u < 1.0f);
  if (T == 0.0f) {  // greedy: the first token of the order
    T = 1.0f;
    k = 1;
  }

  const char* base = static_cast<const char*>(a.logits) + row * a.ld * (BF16 ? 2 : 4);
  auto number = [](float v) { return v == v ? v : -INFINITY; };  // NaN never wins
  auto raw = [&](int64_t i) -> float {
    if constexpr (BF16) return number(bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(base) + i)));
    else return number(__ldg(reinterpret_cast<const float*>(base) + i));
  };
  // Four elements as they lie in memory: one load where the row is aligned and has all four (`end`: where it,
  // or the slice, ends), -inf past the end.
  using Quad = typename std::conditional<BF16, uint2, float4>::type;
  const bool wide = (reinterpret_cast<uintptr_t>(base) & (BF16 ? 7u : 15u)) == 0;
  auto load4 = [&](int64_t i, int64_t end) -> Quad {
    if (wide && i + 4 <= end) {
      if constexpr (BF16) return __ldg(reinterpret_cast<const uint2*>(base + 2 * i));
      else return __ldg(reinterpret_cast<const float4*>(base + 4 * i));
    }
    if constexpr (BF16) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = i + j < end ? __ldg(reinterpret_cast<const uint16_t*>(base) + i + j) : 0xFF80u;
      return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = i + j < end ? __ldg(reinterpret_cast<const float*>(base) + i + j) : -INFINITY;
      return make_float4(x[0], x[1], x[2], x[3]);
    }
  };
  auto unpack = [&](const Quad& q) {
    if constexpr (BF16) return make_float4(number(bf16_lo(q.x)), number(bf16_hi(q.x)), number(bf16_lo(q.y)), number(bf16_hi(q.y)));
    else return make_float4(number(q.x), number(q.y), number(q.z), number(q.w));
  };
  // fn(four elements, index of the first) for i, i + stride, ... below `end` (`first`: the same for a whole
  // warp), four loads ahead: the body is long, so the loop is rolled and the loads queue in registers.
  // The lanes of a warp are called together: past the end with -inf, which counts for nothing.
  auto from_row = [&](int64_t first, int64_t i, int stride, int64_t end, auto fn) {
    const int64_t off = i - first;
    Quad q0 = load4(i, end), q1 = load4(i + stride, end), q2 = load4(i + 2 * stride, end), q3 = load4(i + 3 * stride, end);
#pragma unroll 1
    for (; first < end; first += stride) {
      const Quad now = q0;
      q0 = q1;
      q1 = q2;
      q2 = q3;
      q3 = load4(first + off + 4 * stride, end);
      fn(unpack(now), first + off);
    }
  };
  auto walk = [&](int64_t first, int64_t i, int stride, int64_t end, auto fn) {
    if constexpr (RES) {  // (shared memory holds -inf from the end of the slice to the next multiple of 128)
      const int64_t off = i - first;
#pragma unroll 1
      for (; first < end; first += stride) fn(*reinterpret_cast<const float4*>(res + (first + off - i0)), first + off);
    } else {
      from_row(first, i, stride, end, fn);
    }
  };
  auto value = [&](int64_t i) -> float {
    if constexpr (RES) return res[i - i0];
    else return raw(i);
  };
  // this CTA's slice of probs, zeros: 16 bytes at a time between ragged ends
  auto zero_row = [&] {
    float* dst = a.probs + row * V;
    int64_t b = i0, e = i1;
    if (b >= e) return;
    while (b < e && (reinterpret_cast<uintptr_t>(dst + b) & 15u) != 0) ++b;
    const int64_t q = (e - b) / 4;
    for (int64_t i = i0 + tid; i < b; i += kT) dst[i] = 0.0f;
    for (int64_t i = tid; i < q; i += kT) __stcs(reinterpret_cast<float4*>(dst + b) + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    for (int64_t i = b + 4 * q + tid; i < e; i += kT) dst[i] = 0.0f;
  };
  // 2^frac / z, for one thread
  auto inverse = [&frac](u64 z) {
    return static_cast<float>(__longlong_as_double(static_cast<long long>(1023 + frac) << 52) / static_cast<double>(z));
  };

  // ---- pass 1: the slice into shared memory, its largest and smallest finite-or-+inf logit
  float most = -INFINITY, least = INFINITY;
  from_row(i0 + 128 * warp, i0 + 4 * tid, 4 * kT, i1, [&](const float4& v, int64_t i) {
    if constexpr (RES) *reinterpret_cast<float4*>(res + (i - i0)) = v;
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      most = fmaxf(most, x[j]);
      least = fminf(least, x[j] > -INFINITY ? x[j] : INFINITY);
    }
  });
  // as order bits; 0 and all ones: none
  uint32_t hi = most > -INFINITY ? order_bits(most) : 0u;
  uint32_t lo = most > -INFINITY ? order_bits(least) : 0xFFFFFFFFu;
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) {
    s.wmax[warp] = hi;
    s.wmin[warp] = lo;
  }
  __syncthreads();
  if (nc > 1) cluster_wait_here();
  if (warp == 0) {
    hi = __reduce_max_sync(0xffffffffu, lane < kW ? s.wmax[lane] : 0u);
    lo = __reduce_min_sync(0xffffffffu, lane < kW ? s.wmin[lane] : 0xFFFFFFFFu);
    if (lane < nc) {
      if (nc > 1) {
        st_peer32(peer(&s.cmax[rank], lane), hi);
        st_peer32(peer(&s.cmin[rank], lane), lo);
      } else {
        s.cmax[0] = hi;
        s.cmin[0] = lo;
      }
    }
  } else if (lane == 0) {
    // fp64 is slow here: one thread each, under the exchange of the maxima (by all threads, the division
    // and the logarithm cost 4,000 and 15,000 cycles)
    auto split = [](double v, float& h, float& l) {
      h = static_cast<float>(v);
      l = isinf(h) ? 0.0f : static_cast<float>(v - static_cast<double>(h));
    };
    if (warp == 1) split(1.4426950408889634074 / static_cast<double>(T), s.ch, s.cl);
    if (warp == 2)
      split(min_p > 0.0f && min_p < 1.0f ? static_cast<double>(T) * log(static_cast<double>(min_p)) : 0.0, s.bh, s.bl);
  }
  sync();
  uint32_t mx = 0u, mn = 0xFFFFFFFFu;
  for (int r = 0; r < nc; ++r) {
    mx = s.cmax[r] > mx ? s.cmax[r] : mx;
    mn = s.cmin[r] < mn ? s.cmin[r] : mn;
  }
  auto from_order = [](uint32_t o) { return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o); };

  if (bad || mx == 0u) {  // uniform over the cluster
    if (bad && tid == 0 && rank == 0) store_status(a.status, MTP_ERR_ARG);
    if (tid == 0 && rank == 0) {
      if (a.token) a.token[row] = -1;
      if (a.prob) a.prob[row] = 0.0f;
    }
    if (a.probs) zero_row();
    return;
  }
  const float m = from_order(mx);
  const bool inf = isinf(m);  // then only the infinite logits have weight
  Weigh weigh;
  weigh.m = m;
  weigh.ch = s.ch;
  weigh.cl = s.cl;
  weigh.frac = frac;
  // This thread's part of the row's mass into s.wsum and s.cta (every CTA's, on every CTA); the row's.
  auto share_mass = [&](u64 sum) -> u64 {
    sum = warp_sum(sum);
    if (lane == 0) s.wsum[warp] = sum;
    __syncthreads();
    u64 mine = 0ull;
    for (int q = 0; q < kW; ++q) mine += s.wsum[q];
    if (tid < nc) {
      if (nc > 1) st_peer(peer(&s.cta[rank], tid), mine);
      else s.cta[0] = mine;
    }
    sync();
    u64 z = 0ull;
    for (int r = 0; r < nc; ++r) z += s.cta[r];
    return z;
  };
  if constexpr (LONG) {
    u64 sum = 0ull;
    const int64_t w0 = i0 + warp * seg, w1 = w0 + seg < i1 ? w0 + seg : i1;
    walk(w0, w0 + 4 * lane, 128, w1, [&](const float4& v, int64_t) {
      sum += weigh.mass(v.x) + weigh.mass(v.y) + weigh.mass(v.z) + weigh.mass(v.w);
    });
    // (z + V is more than the sum, V roundings included; a unit is then at most 2^-60 of the whole)
    const u64 z = share_mass(sum) + static_cast<u64>(V);
    frac += 62 - (64 - __clzll(static_cast<long long>(z)));
    weigh.frac = frac;
    sync();  // s.cta has been read everywhere before it is written again
  }
  auto counted = [&](float l) { return inf ? l == m : l > -INFINITY; };
  auto weight = [&](float l) -> float { return counted(l) ? weigh(l) : 0.0f; };
  auto key64 = [&](float l, int64_t i) -> u64 {
    return (static_cast<u64>(order_bits(l)) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(i));
  };
  // min_p as a bound on the logit: the smallest float not below m + T ln(min_p)
  float bound = -INFINITY;
  if (min_p > 0.0f) {
    // m + bh + bl = bound + e exactly; a sum above bound takes the next float (no sum: infinities)
    float e;
    two_sum(m, s.bh, bound, e);
    if (isinf(m)) bound = m;
    else if (isinf(bound)) bound = -3.402823466e38f;
    else if (e + s.bl > 0.0f) bound = nextafterf(bound, INFINITY);
  }

  // ---- the cut: tokens with key >= cut are kept
  u64 cut = 0ull;
  const bool use_k = k > 0 && k < V, use_p = top_p < 1.0f;
  if (use_k || use_p) {
    // Distances at which a weight still counts for something: below 2^-(frac + 2) of the maximum's it
    // rounds to no mass. The bins divide them (or the row's range where that is less).
    float reach = __fmul_rn(T, 0.6931472f * static_cast<float>(frac + 2));
    const float range = inf ? 0.0f : __fsub_rn(m, from_order(mn));
    reach = range < reach ? range : reach;
    float inv = __fdiv_rn(static_cast<float>(kBins), reach);
    if (!(inv <= 3.0e38f) || !(reach <= 3.0e38f)) inv = 0.0f;  // nothing to divide, or not in fp32: one bin
    // (bitwise: the predicates of every element, kept free of branches)
    auto live = [&](float l) { return (l == m) | ((l > -INFINITY) & (__fsub_rn(m, l) <= reach)); };
    auto bin1 = [&](float l) -> int {
      const int b = min(static_cast<int>(__fmul_rn(__fsub_rn(m, l), inv)), kBins - 1);
      return l == m ? 0 : b;
    };
    // The bins of loc summed over the cluster into `all` on every CTA (each sums one section and hands it
    // on); loc is left zero.
    auto share_bins = [&](bool with_mass) {
      sync();
      const int per = kBins / nc;
      for (int b = rank * per + tid; b < static_cast<int>(rank + 1) * per; b += kT) {
        u64 w = 0ull;
        uint32_t n = 0u;
        for (int r = 0; r < nc; ++r) {
          n += nc > 1 ? ld_peer32(peer(&loc.n[b], r)) : loc.n[b];
          if (with_mass) w += nc > 1 ? ld_peer(peer(&loc.mass[b], r)) : loc.mass[b];
        }
        for (int r = 0; r < nc; ++r) {
          if (nc > 1) {
            st_peer32(peer(&all.n[b], r), n);
            if (with_mass) st_peer(peer(&all.mass[b], r), w);
          } else {
            all.n[b] = n;
            all.mass[b] = w;
          }
        }
      }
      sync();
      for (int b = tid; b < kBins; b += kT) {
        loc.mass[b] = 0ull;
        loc.n[b] = 0u;
      }
    };
    // One histogram round over the elements that `in` selects, of entries and / or of masses. (Masses are
    // formed outside the branches, so that an element's chain runs beside its neighbours'.)
    auto histogram = [&](bool with_n, bool with_mass, auto in, auto bin) {
      walk(i0 + 128 * warp, i0 + 4 * tid, 4 * kT, i1, [&](const float4& v, int64_t i) {
        const float x[4] = {v.x, v.y, v.z, v.w};
        bool on[4];
        int b[4];
        bool any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          on[j] = in(x[j], i + j);
          b[j] = on[j] ? bin(x[j], i + j) : -1;
          any = any || on[j];
        }
        if (!__any_sync(0xffffffffu, any)) return;
        if (with_n) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // a whole warp in one bin (equal or far-away logits) adds once
            if (__all_sync(0xffffffffu, b[j] == __shfl_sync(0xffffffffu, b[j], 0))) {
              if (on[j] && lane == 0) atomicAdd(&loc.n[b[j]], 32u);
            } else if (on[j]) {
              atomicAdd(&loc.n[b[j]], 1u);
            }
          }
        }
        if (with_mass) {
          u64 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = weigh.mass(x[j]);
          // 64-bit sums by 32-bit atomics (a 64-bit one is a compare-and-swap loop in shared memory): a lower half's
          // old value tells its carry, the upper half is touched when there is something to add. The four lower
          // halves first, so that their round trips overlap (80 rows with top_p 154 -> 147 us).
          uint32_t carry[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = static_cast<uint32_t>(w[j]);
            uint32_t old = 0u;
            if (on[j] && lo != 0u) old = atomicAdd(reinterpret_cast<uint32_t*>(&loc.mass[b[j]]), lo);
            carry[j] = old > ~lo ? 1u : 0u;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t hi = static_cast<uint32_t>(w[j] >> 32) + carry[j];
            if (on[j] && hi != 0u) atomicAdd(reinterpret_cast<uint32_t*>(&loc.mass[b[j]]) + 1, hi);
          }
        }
      });
      share_bins(with_mass);
    };
    // The first bin at whose end the running count (by_mass: the running mass) reaches lim, given what
    // precedes bin 0. Sets s.hit (-1: none), s.before_n, s.before_m, s.hit_n.
    auto find = [&](bool by_mass, u64 lim, uint32_t base_n, u64 base_m) {
      constexpr int kPer = kBins / kT;
      u64 w[kPer], wt = 0ull;
      uint32_t n[kPer], nt = 0u;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        w[j] = all.mass[tid * kPer + j];
        n[j] = all.n[tid * kPer + j];
        wt += w[j];
        nt += n[j];
      }
      const u64 wi = warp_inclusive(wt, lane);
      const uint32_t ni = static_cast<uint32_t>(warp_inclusive(nt, lane));
      __syncthreads();
      if (lane == 31) {
        s.scan[warp] = wi;
        s.scan_n[warp] = ni;
      }
      if (tid == 0) s.hit = -1;
      __syncthreads();
      u64 bw = base_m + wi - wt;
      u64 bn = base_n + ni - nt;
      for (int q = 0; q < warp; ++q) {
        bw += s.scan[q];
        bn += s.scan_n[q];
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const u64 x0 = by_mass ? bw : bn, x1 = by_mass ? bw + w[j] : bn + n[j];
        if (x0 < lim && x1 >= lim) {
          s.hit = tid * kPer + j;
          s.before_n = static_cast<uint32_t>(bn);
          s.before_m = bw;
          s.hit_n = n[j];
        }
        bw += w[j];
        bn += n[j];
      }
      __syncthreads();
    };
    // The entries that `in` selects to the first CTA's list, if they are at most kGather; returns how many
    // there are, on every CTA. Each CTA lists its own first (an atomic on another CTA's shared memory takes
    // some 2,000 cycles), in the upper half of `all`, which no list overwrites.
    auto gather = [&](auto in, auto then) -> int {
      u64* mine = nc > 1 ? all.mass + kGather : cand;
      walk(i0 + 128 * warp, i0 + 4 * tid, 4 * kT, i1, [&](const float4& v, int64_t i) {
        uint32_t on = (in(v.x, i) ? 1u : 0u) | (in(v.y, i + 1) ? 2u : 0u) | (in(v.z, i + 2) ? 4u : 0u) | (in(v.w, i + 3) ? 8u : 0u);
        while (on != 0u) {
          const int j = __ffs(on) - 1;
          on &= on - 1u;
          const float l = j < 2 ? (j == 0 ? v.x : v.y) : (j == 2 ? v.z : v.w);
          const uint32_t at = atomicAdd(&s.found, 1u);
          if (at < kGather) mine[at] = key64(l, i + j);
        }
      });
      then();  // (what the first CTA's own stores, after the barriers, must find done)
      __syncthreads();
      const uint32_t own = s.found;
      if (nc > 1) {
        if (tid < nc) st_peer32(peer(&s.counts[rank], tid), own);
        cluster_sync_all();
        uint32_t n = 0u, at = 0u;
        for (int r = 0; r < nc; ++r) {
          if (r == static_cast<int>(rank)) at = n;
          n += s.counts[r];
        }
        if (n <= kGather)
          for (uint32_t j = tid; j < own; j += kT) st_peer(peer(&cand[at + j], 0), mine[j]);
        if (tid == 0) s.found = 0u;
        cluster_sync_all();
        return static_cast<int>(n < 0x7FFFFFFFu ? n : 0x7FFFFFFFu);
      }
      __syncthreads();
      if (tid == 0) s.found = 0u;
      return static_cast<int>(own);
    };
    // (first CTA) the list sorted, descending, and its entries' running masses in `list_mass`, from `base`
    u64* list_mass = all.mass;  // [kGather]; the histogram is not needed any more when this is used
    auto sort_list = [&](int n, bool with_mass, u64 base_m) {
      int size = 32;
      while (size < n) size <<= 1;
      for (int j = n + tid; j < size; j += kT) cand[j] = 0ull;
      __syncthreads();
      sort_desc(cand, size);
      u64 w2[2] = {0ull, 0ull};  // two entries a thread
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (with_mass && 2 * tid + j < n) w2[j] = weigh.mass(from_order(static_cast<uint32_t>(cand[2 * tid + j] >> 32)));
      const u64 inc = warp_inclusive(w2[0] + w2[1], lane);
      if (lane == 31) s.scan[warp] = inc;
      __syncthreads();
      u64 before = base_m + inc - w2[0] - w2[1];
      for (int q = 0; q < warp; ++q) before += s.scan[q];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        before += w2[j];
        if (2 * tid + j < kGather) list_mass[2 * tid + j] = before;
      }
      __syncthreads();
    };

    // (list_k is not above nc kT / 2; asked of k alone, the code around came out 0.4 us slower for one row)
    if (use_k && 2 * k <= static_cast<int64_t>(nc) * kT && k <= a.list_k) {
      // ---- the whole row on one sorted list: the bins of the threads' maxima first
      if (live(most)) atomicAdd(&loc.n[bin1(most)], 1u);
      share_bins(false);
      find(false, static_cast<u64>(k), 0u, 0ull);
      const int b1 = s.hit;
      const float upto = b1 == kBins - 1 ? INFINITY : static_cast<float>(b1 + 1);  // bin1(l) <= b1
      const int n = b1 < 0 ? kGather + 1 : gather([&](float l, int64_t) {
        return live(l) & ((l == m) | (__fmul_rn(__fsub_rn(m, l), inv) < upto));
      }, [&] {
        // after the row's last read: written earlier, the zeros of many rows push the logits out of L2
        if (a.probs) zero_row();
      });
      if (n <= kGather) {
        if (rank != 0) return;
        sort_list(n, true, 0ull);
        // kept: the first k; of those, preceding mass < top_p * theirs; of those, logit >= bound
        const u64 lim = use_p ? scale_ceil(top_p, list_mass[k - 1]) : ~0ull;
        int mine = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = 2 * tid + j;
          if (e < static_cast<int>(k))
            mine += (e == 0 || list_mass[e - 1] < lim) && from_order(static_cast<uint32_t>(cand[e] >> 32)) >= bound ? 1 : 0;
        }
        mine = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine)));
        if (lane == 0) s.scan_n[warp] = static_cast<uint32_t>(mine);
        __syncthreads();
        int kept_n = 0;
        for (int q = 0; q < kW; ++q) kept_n += static_cast<int>(s.scan_n[q]);
        const u64 z = list_mass[kept_n - 1];
        if (tid == 0) s.inv_z = inverse(z);
        __syncthreads();
        const float inv_z = s.inv_z;
        if (a.probs)
          for (int e = tid; e < kept_n; e += kT)
            a.probs[row * V + static_cast<int64_t>(~static_cast<uint32_t>(cand[e]))] =
                __fmul_rn(weight(from_order(static_cast<uint32_t>(cand[e] >> 32))), inv_z);
        if (!a.token && !a.prob) return;
        const u64 target = scale_floor(u, z);
        auto take = [&](int e) {
          const u64 key = cand[e];
          if (a.token) a.token[row] = static_cast<int32_t>(~static_cast<uint32_t>(key));
          if (a.prob) a.prob[row] = __fmul_rn(weight(from_order(static_cast<uint32_t>(key >> 32))), inv_z);
        };
        auto mass_of = [&](int e) { return list_mass[e] - (e > 0 ? list_mass[e - 1] : 0ull); };
        u64* order = loc.mass;  // [kGather]
        if (kept_n <= 128) {
          // few: each entry sums the masses of the lower indices (larger complements) itself
          for (int e = tid; e < kept_n; e += kT) order[e] = mass_of(e);
          __syncthreads();
          if (tid < kept_n) {
            const uint32_t me = static_cast<uint32_t>(cand[tid]);
            u64 before = 0ull;
            for (int j = 0; j < kept_n; ++j) before += static_cast<uint32_t>(cand[j]) > me ? order[j] : 0ull;
            if (before <= target && target - before < order[tid]) take(tid);
          }
          return;
        }
        // the kept entries in index order: sorted by (complement of the index, place)
        int size = 32;
        while (size < kept_n) size <<= 1;
        for (int e = tid; e < size; e += kT)
          order[e] = e < kept_n ? (static_cast<u64>(static_cast<uint32_t>(cand[e])) << 32) | static_cast<uint32_t>(e) : 0ull;
        __syncthreads();
        sort_desc(order, size);
        u64 w2[2];
        int place[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = 2 * tid + j;
          place[j] = e < kept_n ? static_cast<int>(static_cast<uint32_t>(order[e])) : -1;
          w2[j] = place[j] < 0 ? 0ull : mass_of(place[j]);
        }
        const u64 inc = warp_inclusive(w2[0] + w2[1], lane);
        if (lane == 31) s.scan[warp] = inc;
        __syncthreads();
        u64 before = inc - w2[0] - w2[1];
        for (int q = 0; q < warp; ++q) before += s.scan[q];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (before <= target && target - before < w2[j]) take(place[j]);
          before += w2[j];
        }
        return;
      }
    }
    // ---- the general case. The cut for a limit: the key of the entry at which the count (the mass)
    // reaches it; returns the mass up to and with that entry (when masses are kept: use_p). binned: `all`
    // holds the live entries by bin1; otherwise all entries count, from the key's first bits on.
    auto resolve = [&](bool by_mass, u64 lim, bool binned, u64& cut_out) -> u64 {
      u64 prefix = 0ull;  // bits of the key fixed so far (from the top)
      int bits = 0, b1 = -1;
      uint32_t bn = 0u;
      u64 bm = 0ull;
      auto in_now = [&](float l, int64_t i) {
        const bool in = b1 < 0 ? counted(l) : live(l) & (bin1(l) == b1);
        return bits == 0 ? in : in & ((key64(l, i) >> (64 - bits)) == prefix);
      };
      int n = kGather + 1;
      if (binned) {
        find(by_mass, lim, 0u, 0ull);
        if (s.hit < 0) return ~0ull;
        b1 = s.hit;
        bn = s.before_n;
        bm = s.before_m;
        n = gather(in_now, [] {});
      }
      while (n > kGather) {
        const int step = bits + 11 <= 64 ? 11 : 64 - bits;
        const int sh = 64 - bits - step;
        __syncthreads();
        // a larger key comes first: bins by the complement of the digit
        histogram(true, use_p, in_now, [&](float l, int64_t i) {
          return static_cast<int>((1u << step) - 1u - (static_cast<uint32_t>(key64(l, i) >> sh) & ((1u << step) - 1u)));
        });
        find(by_mass, lim, bn, bm);
        if (s.hit < 0) return ~0ull;  // fewer entries than the limit
        prefix = (prefix << step) | ((1u << step) - 1u - static_cast<uint32_t>(s.hit));
        bits += step;
        bn = s.before_n;
        bm = s.before_m;
        n = gather(in_now, [] {});
      }
      if (rank == 0) {
        sort_list(n, use_p, bm);
        for (int e = tid; e < n; e += kT) {
          const u64 before = e > 0 ? list_mass[e - 1] : bm;
          const u64 x0 = by_mass ? before : bn + static_cast<u64>(e), x1 = by_mass ? list_mass[e] : x0 + 1ull;
          if (x0 < lim && x1 >= lim) {
            s.cut = cand[e];
            s.cut_mass = list_mass[e];
          }
        }
        __syncthreads();
        if (tid > 0 && tid < nc) {
          st_peer(peer(&s.cut, tid), s.cut);
          st_peer(peer(&s.cut_mass, tid), s.cut_mass);
        }
      }
      sync();
      cut_out = s.cut;
      return s.cut_mass;
    };
    const auto is_live = [&](float l, int64_t) { return live(l); };
    const auto by_bin1 = [&](float l, int64_t) { return bin1(l); };
    u64 total = ~0ull;  // mass of the tokens that top_k keeps (~0: all of them)
    if (use_k) {
      __syncthreads();
      histogram(true, use_p, is_live, by_bin1);
      total = resolve(false, static_cast<u64>(k), true, cut);
      // the k-th entry may lie among those without mass: by the key's bits over the whole row (it changes
      // which of them are kept, and no mass)
      if (cut == 0ull) (void)resolve(false, static_cast<u64>(k), false, cut);
    }
    if (use_p) {
      __syncthreads();
      histogram(false, true, is_live, by_bin1);
      if (total == ~0ull) {
        u64 t = 0ull;
        for (int b = tid; b < kBins; b += kT) t += all.mass[b];
        t = warp_sum(t);
        if (lane == 0) s.scan[warp] = t;
        __syncthreads();
        total = 0ull;
        for (int q = 0; q < kW; ++q) total += s.scan[q];
      }
      // kept: preceding mass < top_p * total, so the cut is where the running mass reaches it
      u64 lim = scale_ceil(top_p, total);
      if (lim == 0ull) lim = 1ull;  // the first token is always kept
      u64 cut_p = 0ull;
      (void)resolve(true, lim, true, cut_p);
      cut = cut_p > cut ? cut_p : cut;
    }
  }
  // kept: above the cut's (or min_p's) logit, or at it and not behind the cut's index; without either,
  // anything but -inf, and with an infinite maximum only that
  float edge = -INFINITY;
  uint32_t edge_index = 0xFFFFFFFFu;  // complement of the last index kept at the edge (all ones: none)
  if (cut != 0ull) {
    edge = from_order(static_cast<uint32_t>(cut >> 32));
    edge_index = static_cast<uint32_t>(cut);
  }
  if (bound > edge) {
    edge = bound;
    edge_index = 0u;
  }
  if (inf && !(edge == m)) {
    edge = m;
    edge_index = 0u;
  }
  auto kept = [&](float l, int64_t i) {
    return (l > edge) | ((l == edge) & (static_cast<uint32_t>(~static_cast<uint32_t>(i)) >= edge_index));
  };

  // ---- masses of the kept tokens per warp segment, CTA and row
  u64 sum = 0ull;
  {
    const int64_t w0 = i0 + warp * seg, w1 = w0 + seg < i1 ? w0 + seg : i1;
    walk(w0, w0 + 4 * lane, 128, w1, [&](const float4& v, int64_t i) {
      const float x[4] = {v.x, v.y, v.z, v.w};
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) on[j] = kept(x[j], i + j);
      if (!__any_sync(0xffffffffu, on[0] || on[1] || on[2] || on[3])) return;
      u64 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = weigh.mass(x[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += on[j] ? w[j] : 0ull;
    });
  }
  const u64 z = share_mass(sum);  // the last exchange: after it every CTA reads its own shared memory only
  if (tid == 0) s.inv_z = inverse(z);
  __syncthreads();
  const float inv_z = s.inv_z;
  if (a.token || a.prob)
    locate(s, rank, scale_floor(u, z), i0, seg, i1,
           [&](int64_t i) {
             const float l = value(i);
             return kept(l, i) ? weigh.mass(l) : 0ull;
           },
           [&](int64_t i) {
             if (a.token) a.token[row] = static_cast<int32_t>(i);
             if (a.prob) a.prob[row] = __fmul_rn(weight(value(i)), inv_z);
           });
  if (a.probs) {
    float* dst = a.probs + row * V;
    const bool wide_out = (reinterpret_cast<uintptr_t>(dst) & 15u) == 0;
    walk(i0 + 128 * warp, i0 + 4 * tid, 4 * kT, i1, [&](const float4& v, int64_t i) {
      const float x[4] = {v.x, v.y, v.z, v.w};
      float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) on[j] = kept(x[j], i + j);
      if (__any_sync(0xffffffffu, on[0] || on[1] || on[2] || on[3])) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = weigh(x[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = on[j] ? __fmul_rn(w[j], inv_z) : 0.0f;
      }
      const float4 o = make_float4(w[0], w[1], w[2], w[3]);
      if (wide_out && i + 4 <= i1) {
        __stcs(reinterpret_cast<float4*>(dst + i), o);
      } else {
        if (i < i1) dst[i] = o.x;
        if (i + 1 < i1) dst[i + 1] = o.y;
        if (i + 2 < i1) dst[i + 2] = o.z;
        if (i + 3 < i1) dst[i + 3] = o.w;
      }
    });
  }
}

// ------------------------------------------------------------------------------- acceptance
// Drafts x_0 .. x_{n-1} of a sequence against the target's distributions p_0 .. p_n and the drafter's
// q_0 .. q_{n-1}: draft i is accepted while u_i q_i(x_i) < p_i(x_i) (probability min(1, p / q)); the
// token after the a accepted ones comes from max(p_a - q_a, 0), or from p_n when all are accepted,
// by inversion with u_D. Emitted tokens are then distributed as the target's. Bound by the read of
// one row of p and one of q per sequence.
//
// Masses are whole numbers, 2^f times the residual, each off by half a unit at most. f = frac leaves room for V
// ones; where the whole then has fewer than V 2^21 units (a row scaled far below one, a residual in p's last bits, a
// row beyond 2^20 tokens), and the roundings together could pass 2^-22 of it, the row is summed once more with
// the f that its sum allows, up to 2^149, at which every fp32 number is whole.
__global__ void __launch_bounds__(kT, 2) verify_kernel(const VerifyArgs a, int nc, int64_t slice, int frac) {
  __shared__ Shared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = nc > 1 ? cluster_rank() : 0u;
  const int64_t b = blockIdx.x / nc;
  const int64_t V = a.V, D = a.D;
  const int64_t i0 = rank * slice, i1 = i0 + slice < V ? i0 + slice : V, seg = slice / kW;
  if (nc > 1) cluster_here();
  pdl_wait_prior_grid();
  int n = a.draft_len ? a.draft_len[b] : a.D;
  const float ud = a.u[b * (D + 1) + D];
  auto unit = [](float u) { return u >= 0.0f && u < 1.0f; };
  // a sequence with a bad length or random number is refused as a whole (every warp decides for
  // itself, alike; the return is uniform over the cluster)
  bool bad = n < 0 || n > a.D || !unit(ud);
  for (int i = lane; !bad && i < n; i += 32) bad = !unit(a.u[b * (D + 1) + i]);
  if (__any_sync(0xffffffffu, bad)) {
    if (nc > 1) cluster_wait_here();
    if (rank == 0) {
      for (int i = tid; i <= a.D; i += kT) a.tokens[b * (D + 1) + i] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        if (a.prob) a.prob[b] = 0.0f;
        store_status(a.status, MTP_ERR_ARG);
      }
    }
    return;
  }
  // the acceptance, 32 drafts at a time; a draft outside [0, V) is rejected
  int acc = 0, rejected_token = -1;
  bool outside = false;
  while (acc < n) {
    const int i = acc + lane;
    bool ok = false;
    int32_t x = -1;
    if (i < n) {
      x = a.draft_tokens[b * D + i];
      if (x >= 0 && x < V) {
        const float u = a.u[b * (D + 1) + i];
        // both taken into [0, 1] (NaN saturates to 0), but a NaN q refuses the draft: nothing is known of how it was
        // drawn, and what is emitted then comes from p alone
        const float p = __saturatef(a.target_probs[(b * (D + 1) + i) * V + x]);
        const float qr = a.draft_probs ? a.draft_probs[(b * D + i) * V + x] : 1.0f;
        const float q = __saturatef(qr);
        // u q < p exactly: the rounded product, and its error where it ties (in fp64, which is slow here, only
        // where the error may leave the fp32 range)
        const float h = __fmul_rn(u, q);
        ok = h < p || (h == p && __fmaf_rn(u, q, -h) < 0.0f);
        if (h < 1e-30f && p < 1e-30f) ok = static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
        ok = ok && qr == qr;
      }
    }
    const uint32_t no = __ballot_sync(0xffffffffu, !ok);
    const int run = no ? __ffs(no) - 1 : 32;
    const int left = n - acc;
    if (run < left && run < 32) {
      rejected_token = __shfl_sync(0xffffffffu, x, run);
      outside = rejected_token < 0 || rejected_token >= V;
      acc += run;
      break;
    }
    acc += run < left ? run : left;
  }
  const bool all = acc == n;
  const float* p = a.target_probs + (b * (D + 1) + acc) * V;
  const float* q = !all && a.draft_probs ? a.draft_probs + (b * D + acc) * V : nullptr;
  auto left_of = [&](float pv, float qv, int64_t i) -> float {
    if (!q) qv = i == rejected_token ? 1.0f : 0.0f;
    qv = all ? 0.0f : __saturatef(qv);  // (NaN saturates to 0)
    return __saturatef(__fsub_rn(__saturatef(pv), qv));
  };
  // 2^bits r to the nearest whole number (a subnormal's mantissa, and a zero's, get a bit too much here: they round
  // to nothing all the same while bits <= 63)
  auto whole = [](float r, int bits) -> u64 {
    const uint32_t u = __float_as_uint(r);
    return shift_round((u & 0x7FFFFFu) | 0x800000u, static_cast<int>(u >> 23) - 150 + bits);
  };
  const bool wide = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
  const int64_t w0 = i0 + warp * seg, w1 = w0 + seg < i1 ? w0 + seg : i1;
  // The row's mass from the lanes' sums; s.wsum and s.cta keep the warps' and the CTAs'.
  auto share = [&](u64 sum, bool first) -> u64 {
    sum = warp_sum(sum);
    if (lane == 0) s.wsum[warp] = sum;
    __syncthreads();
    u64 mine = 0ull;
    for (int w = 0; w < kW; ++w) mine += s.wsum[w];
    if (nc > 1) {  // the peers run, and have read the previous pass's masses
      if (first) cluster_wait_here();
      else cluster_sync_all();
    }
    if (tid < nc) {
      if (nc > 1) st_peer(peer(&s.cta[rank], tid), mine);
      else s.cta[0] = mine;
    }
    if (nc > 1) cluster_sync_all();
    else __syncthreads();
    u64 z = 0ull;
    for (int r = 0; r < nc; ++r) z += s.cta[r];
    return z;
  };
  u64 z;
  {
    u64 sum = 0ull;
    // steps of 128 elements, two steps' loads under the work on the two before
    auto load4 = [&](const float* row, int64_t i) {
      if (wide && i + 4 <= w1) return __ldg(reinterpret_cast<const float4*>(row + i));
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < w1 ? __ldg(row + i + e) : 0.0f;
      return make_float4(x[0], x[1], x[2], x[3]);
    };
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kBatch = 2;
    float4 pn[kBatch], qn[kBatch];
    auto fetch = [&](int64_t i) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        pn[j] = load4(p, i + 128 * j);
        qn[j] = q ? load4(q, i + 128 * j) : none;
      }
    };
    auto mass = [&](float pv, float qv, int64_t i) { return whole(left_of(pv, qv, i), frac); };
    fetch(w0 + 4 * lane);
#pragma unroll 1
    for (int64_t i = w0 + 4 * lane; i - 4 * lane < w1; i += 128 * kBatch) {
      float4 pv[kBatch], qv[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        pv[j] = pn[j];
        qv[j] = qn[j];
      }
      fetch(i + 128 * kBatch);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t at = i + 128 * j;  // (past the end the loads gave zeros)
        sum += mass(pv[j].x, qv[j].x, at) + mass(pv[j].y, qv[j].y, at + 1) + mass(pv[j].z, qv[j].z, at + 2) +
               mass(pv[j].w, qv[j].w, at + 3);
      }
    }
    z = share(sum, true);
  }
  // Too coarse: again, with what the sum leaves room for. f is the fraction bits of the masses that z, s.wsum and
  // s.cta hold; a residual is lifted out of the subnormal range first where f needs it. (A loop of its own: one loop
  // for both cost the ordinary row 5 to 9 %.)
  constexpr int kExact = 149, kLift = 86;
  const u64 enough = static_cast<u64>(V) << 21;
  bool plain = false;  // the residual is empty: the target's own row
  int f = frac;
  auto residual = [&](int64_t i) -> float {
    const float pv = __ldg(p + i);
    return plain ? __saturatef(pv) : left_of(pv, q ? __ldg(q + i) : 0.0f, i);
  };
  auto mass_at = [&](int64_t i) -> u64 {
    const float r = residual(i);
    return f > 62 ? whole(__fmul_rn(r, 0x1p86f), f - kLift) : whole(r, f);
  };
#pragma unroll 1
  while (z < enough) {  // the same on every CTA
    if (f < kExact) {   // z + V is more than the sum, and 2^61 is room enough
      const int room = 61 - (64 - __clzll(static_cast<long long>(z + static_cast<u64>(V))));
      f = f + room < kExact ? f + room : kExact;
    } else if (z == 0ull && !all && !plain) {
      plain = true;
      f = frac;
    } else {
      break;
    }
    u64 sum = 0ull;
#pragma unroll 4
    for (int64_t i = w0 + lane; i < w1; i += 32) sum += mass_at(i);
    z = share(sum, false);
  }
  if (rank == 0) {
    for (int i = tid; i <= a.D; i += kT)
      if (i != acc) a.tokens[b * (D + 1) + i] = i < acc ? a.draft_tokens[b * D + i] : -1;
    if (tid == 0) {
      a.accepted[b] = acc;
      if (outside) store_status(a.status, MTP_ERR_TOKEN_RANGE);
      if (z == 0ull) {
        a.tokens[b * (D + 1) + acc] = -1;
        if (a.prob) a.prob[b] = 0.0f;
      }
    }
  }
  if (z != 0ull)
    locate(s, rank, scale_floor(ud, z), i0, seg, i1,
           mass_at,
           [&](int64_t i) {
             a.tokens[b * (D + 1) + acc] = static_cast<int32_t>(i);
             if (a.prob)
               a.prob[b] = static_cast<float>(static_cast<double>(residual(i)) *
                                              __longlong_as_double(static_cast<long long>(1023 + f) << 52) /
                                              static_cast<double>(z));
           });
}

// ------------------------------------------------------------------------------- host side
cudaError_t launch_cluster(const void* kernel, unsigned grid, int nc, size_t smem, cudaStream_t stream, void** args) {
  static std::mutex mu;
  static bool done[64][8] = {};
  static const void* kernels[8] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    int slot = 0;
    while (kernels[slot] != nullptr && kernels[slot] != kernel) ++slot;
    kernels[slot] = kernel;
    if (!done[dev][slot]) {
      DeviceInfo di;
      err = device_info(&di);
      if (err != cudaSuccess) return err;
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin);
      if (err != cudaSuccess) return err;
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (err != cudaSuccess) return err;
      done[dev][slot] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(nc);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = nc > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Longest slice that a CTA keeps in shared memory: of 227 KB, or of half of an SM's (two CTAs).
constexpr int64_t kHeldSlice = static_cast<int64_t>((227 * 1024 - kFixedSmem) / 4 / kSliceUnit * kSliceUnit);
static_assert(kMaxC * kHeldSlice <= kLongRow, "a long row is never held");
constexpr int64_t kHeldSliceOfTwo = static_cast<int64_t>((113 * 1024 - kFixedSmem) / 4 / kSliceUnit * kSliceUnit);

int64_t slice_of(int64_t V, int nc) { return ((V + nc - 1) / nc + kSliceUnit - 1) / kSliceUnit * kSliceUnit; }

// Fraction bits of a mass: V weights of at most one stay below 2^62 (plus their roundings).
int mass_bits(int64_t V) {
  int lg = 0;
  while ((static_cast<int64_t>(1) << lg) < V) ++lg;
  return 62 - lg;
}

// Whether a cluster of nc can be of use: each warp has more than a step of its own.
bool worth(int64_t V, int nc) { return V > static_cast<int64_t>(nc) * kSliceUnit; }

// CTAs per row of the sampler (a power of two up to kMaxC). Clusters of 16 as long as they all run at once:
// with two CTAs on an SM 14 of them fit the GPU's SM groups. Without top_k each CTA's time is in the histogram's
// shared-memory atomics, so the spread over more SMs still pays for a short second wave. Beyond that clusters of
// four, and single CTAs for short rows that fill the GPU anyway. At V = 154880, rows in L2: 16 rows with top_k and
// top_p take 25.5 us with 16 CTAs, 26.8 with 8 and 20.6 with 4; with top_p alone 53.5, 56.4 and 61.0; 24 rows 31.4,
// 28.0 and 20.9, and 71.6, 75.7 and 59.9. 160 rows of V = 32000 with top_k take 33.1 with one CTA and 39.3 with 4.
int sample_cluster(int64_t rows, int64_t V, bool top_k, int sm_count) {
  int nc = 4;
  if (rows <= (top_k ? 14 : 18)) nc = kMaxC;
  else if (rows >= sm_count && V <= kHeldSlice) nc = 1;
  while (nc > 1 && !worth(V, nc)) nc /= 2;
  return nc;
}

// The largest top_k that is finished on one sorted list. Of a cluster's n threads, n ln(n / (n - k)) entries reach the
// k-th largest maximum on average: at most k + 2/3 k^2 / n where that is near the list's length (k below n / 2.6; with
// fewer threads the list is long enough for any k up to n / 2). The rest of the list is for the spread and the bin's
// width. (A list that does not fit costs its row the passes made for it: with k = 1024 and no such rule 80 rows took
// 236 us and one row 44.7, by the histogram at once 206 and 37.3; at k = 700 with a list 57, without 203.)
int list_limit(int nc) {
  const int64_t n = static_cast<int64_t>(nc) * kT;
  int64_t k = n / 2 < kGather ? n / 2 : kGather;
  while (k * (3 * n + 2 * k) > 3 * (kGather - 44) * n) --k;
  return static_cast<int>(k);
}

// CTAs per sequence of the acceptance: one on each SM. 16 sequences at V = 154880 take 17.7 us with 16 CTAs each
// (two waves), 14.8 with 8, 14.4 with 4; 80 at V = 32000 take 12.0 with one CTA and 14.5 with two.
int verify_cluster(int64_t rows, int64_t V, int sm_count) {
  int nc = 1;
  while (nc < kMaxC && rows * nc * 2 <= sm_count && worth(V, nc * 2)) nc *= 2;
  return nc;
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& in, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  SampleArgs a = in;
  int nc = sample_cluster(a.R, a.V, a.top_k != nullptr, di.sm_count);
  a.list_k = list_limit(nc);
  int64_t slice = slice_of(a.V, nc);
  // A slice is kept in shared memory where that leaves room for as many CTAs per SM as there are to run (two hide
  // each other's loads: 80 rows with top_k and top_p, out of HBM, 66 us, and 74 with one and its slice held).
  const bool one_each = static_cast<int64_t>(a.R) * nc <= di.sm_count || nc == 1;
  const bool res = slice <= (one_each ? kHeldSlice : kHeldSliceOfTwo);
  int frac = mass_bits(a.V);
  const bool is_long = a.V > kLongRow;  // (more than any cluster holds: never with res)
  const void* kern = a.bf16 ? (is_long ? reinterpret_cast<const void*>(sample_kernel<true, false, true>)
                               : res   ? reinterpret_cast<const void*>(sample_kernel<true, true, false>)
                                       : reinterpret_cast<const void*>(sample_kernel<true, false, false>))
                            : (is_long ? reinterpret_cast<const void*>(sample_kernel<false, false, true>)
                               : res   ? reinterpret_cast<const void*>(sample_kernel<false, true, false>)
                                       : reinterpret_cast<const void*>(sample_kernel<false, false, false>));
  void* args[] = {&a, &nc, &slice, &frac};
  return launch_cluster(kern, static_cast<unsigned>(a.R) * nc, nc,
                        kFixedSmem + (res ? static_cast<size_t>(slice) * 4 : 0), stream, args);
}

cudaError_t launch_verify(const VerifyArgs& in, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  VerifyArgs a = in;
  int nc = verify_cluster(a.B, a.V, di.sm_count);
  int64_t slice = slice_of(a.V, nc);
  int frac = mass_bits(a.V);
  void* args[] = {&a, &nc, &slice, &frac};
  return launch_cluster(reinterpret_cast<const void*>(verify_kernel), static_cast<unsigned>(a.B) * nc, nc, 0, stream,
                        args);
}

}  // namespace mtp
