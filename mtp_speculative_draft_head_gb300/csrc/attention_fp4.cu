// Attention of a few query rows per sequence over its pages of the FP4 cache (a draft step's row, or a
// verification's rows):
//   o_i = sum_j p_ij v_j,   p_ij = softmax_j( scale q_i . k_j ),   j < length - n + i + 1
//
// A CTA takes one sequence, one key head, up to 16 of the rows that share it (n rows x the query heads of
// the group) and a range of the sequence's tokens; its four warps take 32 tokens at a time in turn, each
// with running maxima, sum and outputs of its own, so nothing synchronises the warps until the range
// ends. The ranges' results meet in the workspace, where the CTA that finishes last joins them in order.
//
// The rows are the M side of warp-level MMAs (m16n8k16, f16 operands, fp32 sums); keys and values go from
// shared memory to MMA operands in registers. Codes are widened to f16 pairs by the hardware
// conversion and block scales multiply in f16, which is exact (six significant bits). The fp32 row scales
// stay out of the operands: a key's multiplies its scores, a value's goes into the exponent of its
// weight. With x_ij the score in powers of two and v_j = r_j u_j, the warp keeps
//   l_i = sum_j 2^(x_ij - m_i)      and      O_i = sum_j 2^(x_ij + log2 r_j - m'_i) u_j
// with separate maxima m and m', so the f16 weights of O are of order one whatever the values' sizes.
// Query rows are BF16 values times a power of two that brings their largest near 2^7: exact in f16 but
// for elements below 2^-24 of that.
//
// Tokens and columns are MMA indexes in an order that fits the operands: in a tile of eight keys the
// columns are tokens 0 4 1 5 2 6 3 7, so that a thread's score columns are the tokens of its value
// operands; a thread reads D/4 consecutive columns of a key, and D/8 of a value.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "layer.h"
#include "tc.cuh"

namespace mtp {

namespace {

constexpr int kAWarps = 4;
constexpr int kAThreads = kAWarps * 32;
constexpr int kStep = 32;                    // tokens of a warp's step
constexpr int kChunkTok = kAWarps * kStep;   // tokens of a CTA's round
constexpr int kARows = 16;                   // rows of a CTA
constexpr int kAStages = 3;
constexpr int kMaxSplits = 128;
constexpr int kSlots = 152 * 3;              // CTAs that run at once
constexpr int kLongRange = 4096;             // a range of tokens is no longer than this where splits allow

template <int D>
struct AStage {  // one warp's stage: keys and values of 32 tokens
  static constexpr int kCode = kStep * D / 2, kScale = kStep * D / kFp4Block, kRow = kStep * 4;
  static constexpr int kV = kCode + kScale + kRow;
  static constexpr int kBytes = 2 * kV;
  // merge buffer: a row's quarters (one per lane of a quad) with gaps against bank conflicts
  static constexpr int kQuarter = D / 4 + 8, kMergeRow = 4 * kQuarter + 4;
  static constexpr size_t kRing = static_cast<size_t>(kAWarps) * kAStages * kBytes;
  static constexpr size_t kMerge = static_cast<size_t>(kAWarps) * kARows * kMergeRow * 4;
  static constexpr size_t kStats = static_cast<size_t>(kMaxSplits) * kARows * 16;
  static constexpr size_t kLarger = kRing > kMerge ? kRing : kMerge;
  static constexpr size_t kSmem = kLarger > kStats ? kLarger : kStats;
};

struct Plan {
  int groups, splits;
};
// Ranges per (sequence, key head, group of rows): enough for four CTAs per one that runs (equal shares
// of unequal sequences), and for ranges of at most kLongRange tokens, as far as kMaxSplits go.
inline Plan plan(int B, int Q, int q_heads, int kv_heads, int64_t max_len) {
  Plan p;
  p.groups = (Q * (q_heads / kv_heads) + kARows - 1) / kARows;
  const int64_t pairs = static_cast<int64_t>(B) * kv_heads * p.groups;
  int64_t s = (4 * kSlots + pairs - 1) / pairs;
  const int64_t by_length = (max_len + kLongRange - 1) / kLongRange, chunks = (max_len + kChunkTok - 1) / kChunkTok;
  if (s < by_length) s = by_length;
  if (s > chunks) s = chunks;
  if (s > kMaxSplits) s = kMaxSplits;
  p.splits = s < 1 ? 1 : static_cast<int>(s);
  return p;
}
inline int rows_kept(int Q, int G) { return Q * G < kARows ? Q * G : kARows; }
inline size_t counters_bytes(int64_t pairs) { return (static_cast<size_t>(pairs) * 4 + 255) / 256 * 256; }

struct Params {
  AttentionFp4Args a;
  int groups, splits, kept, G;
  float* part_o;     // [pairs, splits, kept, D]
  float* part_stat;  // [pairs, splits, kept, 4]: m, l, m'
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ float lds_f(uint32_t a) { return __uint_as_float(lds32(a)); }
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one load");
  if constexpr (N == 1)
    w[0] = lds32(a);
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a)
                 : "memory");
}
constexpr float kNegInf = -INFINITY;

template <int D>
__global__ void __launch_bounds__(kAThreads, 3) attention_fp4_kernel(const Params p) {
  using ST = AStage<D>;
  constexpr int kKSteps = D / 16, kTiles = D / 8, kBlocks = D / kFp4Block;
  constexpr int kKWords = D / 32, kVWords = D / 64;  // words of codes that a thread takes of a key, of a value
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float st_m[kAWarps][kARows], st_l[kAWarps][kARows], st_n[kAWarps][kARows];
  __shared__ int last_s;
  const AttentionFp4Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int sp = static_cast<int>(blockIdx.x % p.splits);
  const int64_t pair = blockIdx.x / p.splits;
  const int grp = static_cast<int>(pair % p.groups);
  const int h = static_cast<int>(pair / p.groups % a.c.heads);
  const int b = static_cast<int>(pair / p.groups / a.c.heads);
  pdl_wait_prior_grid();

  int n = a.rows != nullptr ? a.rows[b] : a.Q;
  int len = a.length[b];
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.c.page;
  if (n < 0 || n > a.Q || len < 0 || len > cap) {
    if (threadIdx.x == 0 && sp == 0) store_status(a.status, MTP_ERR_ARG);
    n = a.Q;  // its rows see nothing
    len = 0;
  }
  const int r0 = grp * kARows;
  int nrows = n * p.G - r0;  // rows of this CTA
  if (nrows <= 0) return;
  if (nrows > kARows) nrows = kARows;
  int seen = len - n + (r0 + nrows - 1) / p.G + 1;  // tokens that its last row sees
  if (seen < 0) seen = 0;
  const int chunks = (seen + kChunkTok - 1) / kChunkTok;
  const int per = (chunks + p.splits - 1) / p.splits;  // chunks of a range
  const int active = chunks == 0 ? 1 : (chunks + per - 1) / per;
  if (sp >= active) return;
  const int begin = sp * per * kChunkTok;
  const int end = min(seen, begin + per * kChunkTok);

  // ---- copies: a warp's step into its own ring
  const uint32_t ring = smem_addr(smem) + warp * kAStages * ST::kBytes;
  const int first = begin + warp * kStep;
  const int* table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int page_shift = __ffs(a.c.page) - 1;
  auto page_of = [&](int tok) {  // of the 16 tokens from tok
    if (tok >= end) return 0;
    const int pg = table[tok >> page_shift];
    if (pg >= 0 && pg < a.c.pages) return pg;
    if (lane == 0) store_status(a.status, MTP_ERR_ARG);
    return -1;  // (its tokens count as zeros)
  };
  auto copy_step = [&](int tok0, int stage, int pg0, int pg1) {
    const uint32_t dst = ring + stage * ST::kBytes;
    int64_t row[2];  // the first row of each half in the cache's rows, key; values follow after heads * page
    row[0] = ((static_cast<int64_t>(max(pg0, 0)) * 2) * a.c.heads + h) * a.c.page + (tok0 & (a.c.page - 1));
    row[1] = ((static_cast<int64_t>(max(pg1, 0)) * 2) * a.c.heads + h) * a.c.page + ((tok0 + 16) & (a.c.page - 1));
    const int64_t to_v = static_cast<int64_t>(a.c.heads) * a.c.page;
    const int have0 = pg0 < 0 ? 0 : end - tok0, have1 = pg1 < 0 ? 0 : end - tok0 - 16;  // tokens of each half
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const uint32_t d = dst + kind * ST::kV;
      constexpr int kPer = D / 32;  // 16-byte pieces of a token's codes
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = lane + 32 * i, tok = piece / kPer, c = piece % kPer, half = tok >> 4, in = tok & 15;
        const int slot = kind == 0 ? ((in & 8) | ((in & 3) << 1) | ((in >> 2) & 1)) + 16 * half : tok;
        const int cc = kind == 1 && D == 128 ? c ^ (tok & 2) : c;
        const int64_t src = (half ? row[1] : row[0]) + in + kind * to_v;
        const bool on = in < (half ? have1 : have0);
        cp16(d + slot * (D / 2) + cc * 16, a.c.q + (on ? src * (D / 2) + c * 16 : 0), on ? 16u : 0u);
      }
      constexpr int kScalePieces = kStep * kBlocks / 16, kTokPer = 16 / kBlocks;  // 16-byte pieces of scales
      if (lane < kScalePieces + kStep / 4) {
        const bool sc = lane < kScalePieces;
        const int tok = sc ? lane * kTokPer : (lane - kScalePieces) * 4, half = tok >> 4, in = tok & 15;
        const int item = sc ? kBlocks : 4;
        int have = (half ? have1 : have0) - in;
        have = min(max(have, 0) * item, 16);
        const int64_t src = have > 0 ? (half ? row[1] : row[0]) + in + kind * to_v : 0;
        cp16(d + ST::kCode + (sc ? 0 : ST::kScale) + tok * item,
             sc ? static_cast<const void*>(a.c.bs + src * kBlocks) : static_cast<const void*>(a.c.rs + src),
             static_cast<uint32_t>(have));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int stride = kChunkTok;
  int next_tok = first;
  int pg0 = page_of(next_tok), pg1 = page_of(next_tok + 16);
#pragma unroll
  for (int i = 0; i < kAStages - 1; ++i) {
    if (next_tok < end)
      copy_step(next_tok, i, pg0, pg1);
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
    next_tok += stride;
    pg0 = page_of(next_tok), pg1 = page_of(next_tok + 16);
  }

  // ---- queries: rows g and g + 8 as f16 operands
  uint32_t qa[kKSteps][4];
  // From a row's MMA sums to scores in powers of two: f1 times the key's row scale times f2, so that no product
  // leaves the fp32 range on the way.
  float f1[2], f2[2];
  int limit[2];  // tokens that a row sees
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + g + 8 * i;
    const bool on = g + 8 * i < nrows;
    const int qi = on ? r / p.G : 0;
    limit[i] = on ? len - n + qi + 1 : 0x7FFFFFFF;  // (a row that is not there: whatever it sees)
    const uint16_t* src = a.query + (static_cast<int64_t>(b) * a.Q + qi) * a.ld_q +
                          static_cast<int64_t>(h * p.G + (on ? r % p.G : 0)) * D + t * (D / 4);
    uint32_t u[D / 8];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint4 v = on ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0u, 0u, 0u, 0u);
      u[4 * k] = v.x, u[4 * k + 1] = v.y, u[4 * k + 2] = v.z, u[4 * k + 3] = v.w;
    }
    float mx = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 8; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(u[k])), fabsf(bf16_hi(u[k]))));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;  // (a subnormal: -127)
    e = mx > 0.0f && e < 128 ? max(min(7 - e, 126), -126) : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    f1[i] = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
    f2[i] = a.scale * 1.44269504088896341f * __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
#pragma unroll
    for (int s = 0; s < kKSteps; ++s) {
      qa[s][i] = f16x2_bits(bf16_lo(u[2 * s]) * up, bf16_hi(u[2 * s]) * up);
      qa[s][2 + i] = f16x2_bits(bf16_lo(u[2 * s + 1]) * up, bf16_hi(u[2 * s + 1]) * up);
    }
  }

  float o[kTiles][4];
#pragma unroll
  for (int j = 0; j < kTiles; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[j][c] = 0.0f;
  float m[2] = {kNegInf, kNegInf}, mv[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
  const int least = min(limit[0], limit[1]);  // tokens before it are seen by both rows

  int stage = 0;
  for (int tok0 = first; tok0 < end; tok0 += stride) {
    {
      const int s = stage == 0 ? kAStages - 1 : stage - 1;
      if (next_tok < end)
        copy_step(next_tok, s, pg0, pg1);
      else
        asm volatile("cp.async.commit_group;" ::: "memory");
      next_tok += stride;
      pg0 = page_of(next_tok), pg1 = page_of(next_tok + 16);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kAStages - 1) : "memory");
    __syncwarp();
    const uint32_t kb = ring + stage * ST::kBytes, vb = kb + ST::kV;

    // scores of two halves of two tiles of eight tokens
    float x[2][2][4];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        float(&acc)[4] = x[hf][tl];
        acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
        uint32_t w[kKWords];
        lds_words<kKWords>(kb + (hf * 16 + tl * 8 + g) * (D / 2) + t * (D / 8), w);
        const int tok = hf * 16 + tl * 8 + (g >> 1) + 4 * (g & 1);
        uint32_t sc0, sc1;
        if constexpr (D == 128) {
          const uint32_t s2 = e4m3x2_to_f16x2(lds16(kb + ST::kCode + tok * kBlocks + 2 * t));
          sc0 = __byte_perm(s2, s2, 0x1010);
          sc1 = __byte_perm(s2, s2, 0x3232);
        } else {
          sc0 = sc1 = e4m3x2_to_f16x2(lds8(kb + ST::kCode + tok * kBlocks + t) * 0x0101u);
        }
#pragma unroll
        for (int i = 0; i < kKWords; ++i) {
          uint32_t v[4];
          e2m1x8_to_f16x2x4(w[i], v);
          const uint32_t sc = i < kKWords / 2 ? sc0 : sc1;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = f16x2_mul(v[k], sc);
          mma_f16(acc, qa[2 * i], v[0], v[1]);
          mma_f16(acc, qa[2 * i + 1], v[2], v[3]);
        }
      }
    }
    // to powers of two, masked; and the values' row scales into exponents
    float xm[2] = {kNegInf, kNegInf}, ym[2] = {kNegInf, kNegInf};
    float lv[2][2][2];
    const bool edge = !__all_sync(0xffffffffu, tok0 + kStep <= least);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
      {
        const int tok = hf * 16 + tl * 8 + t;
        const uint32_t rk = kb + ST::kCode + ST::kScale + tok * 4, rv = vb + ST::kCode + ST::kScale + tok * 4;
        const uint64_t r2 = f2_pack(lds_f(rk), lds_f(rk + 16));
        lv[hf][tl][0] = lg2(lds_f(rv));
        lv[hf][tl][1] = lg2(lds_f(rv + 16));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t y = f2_mul(f2_mul(f2_mul(f2_pack(x[hf][tl][2 * i], x[hf][tl][2 * i + 1]), f2_pack(f1[i], f1[i])), r2),
                                    f2_pack(f2[i], f2[i]));
          x[hf][tl][2 * i] = f2_lo(y);
          x[hf][tl][2 * i + 1] = f2_hi(y);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float& v = x[hf][tl][2 * i + c];
            if (edge && tok0 + tok + 4 * c >= limit[i]) v = kNegInf;
            xm[i] = fmaxf(xm[i], v);
            ym[i] = fmaxf(ym[i], v + lv[hf][tl][c]);
          }
        }
      }
    // The maxima move only when a score passes one by 2^8: below that the weights stay within f16's range.
    bool up = false, upv = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xm[i] = fmaxf(xm[i], __shfl_xor_sync(0xffffffffu, xm[i], 1));
      xm[i] = fmaxf(xm[i], __shfl_xor_sync(0xffffffffu, xm[i], 2));
      ym[i] = fmaxf(ym[i], __shfl_xor_sync(0xffffffffu, ym[i], 1));
      ym[i] = fmaxf(ym[i], __shfl_xor_sync(0xffffffffu, ym[i], 2));
      up |= xm[i] > m[i] + 8.0f;
      upv |= ym[i] > mv[i] + 8.0f;
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float to = fmaxf(m[i], xm[i]);
        l[i] *= m[i] == kNegInf ? 0.0f : ex2(m[i] - to);
        m[i] = to;
      }
    }
    if (__any_sync(0xffffffffu, upv)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float to = fmaxf(mv[i], ym[i]);
        const float k = mv[i] == kNegInf ? 0.0f : ex2(mv[i] - to);
        mv[i] = to;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          o[j][2 * i] *= k;
          o[j][2 * i + 1] *= k;
        }
      }
    }
    const float ms[2] = {m[0] == kNegInf ? 0.0f : m[0], m[1] == kNegInf ? 0.0f : m[1]};
    const float ns[2] = {mv[0] == kNegInf ? 0.0f : mv[0], mv[1] == kNegInf ? 0.0f : mv[1]};

    // outputs: 16 tokens at a time
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t pw[4];
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x0 = x[hf][tl][2 * i], x1 = x[hf][tl][2 * i + 1];
          l[i] += ex2(x0 - ms[i]) + ex2(x1 - ms[i]);
          pw[2 * tl + i] = f16x2_bits(ex2(x0 + lv[hf][tl][0] - ns[i]), ex2(x1 + lv[hf][tl][1] - ns[i]));
        }
      uint32_t v[4][4 * kVWords];  // four tokens' pairs of columns
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = hf * 16 + t + 4 * k;
        uint32_t w[kVWords], s2;
        if constexpr (D == 128) {
          lds_words<kVWords>(vb + tok * (D / 2) + (((g >> 1) ^ (t & 2)) << 4) + (g & 1) * 8, w);
          s2 = e4m3x2_to_f16x2(lds8(vb + ST::kCode + tok * kBlocks + g) * 0x0101u);
        } else {
          lds_words<kVWords>(vb + tok * (D / 2) + g * 4, w);
          s2 = e4m3x2_to_f16x2(lds8(vb + ST::kCode + tok * kBlocks + (g >> 1)) * 0x0101u);
        }
#pragma unroll
        for (int i = 0; i < kVWords; ++i) {
          uint32_t u[4];
          e2m1x8_to_f16x2x4(w[i], u);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[k][4 * i + e] = f16x2_mul(u[e], s2);
        }
      }
#pragma unroll
      for (int j = 0; j < kTiles / 2; ++j) {
        mma_f16(o[2 * j], pw, __byte_perm(v[0][j], v[1][j], 0x5410), __byte_perm(v[2][j], v[3][j], 0x5410));
        mma_f16(o[2 * j + 1], pw, __byte_perm(v[0][j], v[1][j], 0x7632), __byte_perm(v[2][j], v[3][j], 0x7632));
      }
    }
    __syncwarp();  // the stage is free for the copies of the next round
    stage = stage == kAStages - 1 ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // the rings become the merge buffer

  // ---- the warps' results
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (t == 0) {
      st_m[warp][g + 8 * i] = m[i];
      st_l[warp][g + 8 * i] = l[i];
      st_n[warp][g + 8 * i] = mv[i];
    }
    // row g + 8 i, columns t D/4 ..: n-tile j holds column j of the even and of the odd eighth
    float* dst = reinterpret_cast<float*>(smem) + (warp * kARows + g + 8 * i) * ST::kMergeRow + t * ST::kQuarter;
#pragma unroll
    for (int j = 0; j < kTiles; j += 4) {
      *reinterpret_cast<float4*>(dst + j) = make_float4(o[j][2 * i], o[j + 1][2 * i], o[j + 2][2 * i], o[j + 3][2 * i]);
      *reinterpret_cast<float4*>(dst + kTiles + j) =
          make_float4(o[j][2 * i + 1], o[j + 1][2 * i + 1], o[j + 2][2 * i + 1], o[j + 3][2 * i + 1]);
    }
  }
  __syncthreads();
  auto store_row = [&](int r, int c, float4 v, float k) {  // four columns of row r, times k
    const int qi = (r0 + r) / p.G;
    uint16_t* dst = a.out + (static_cast<int64_t>(b) * a.Q + qi) * a.ld_out +
                    static_cast<int64_t>(h * p.G + (r0 + r) % p.G) * D + c;
    uint32_t lo, hi;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(v.y * k), "f"(v.x * k));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(v.w * k), "f"(v.z * k));
    *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
  };
  auto store_lse = [&](int r, float mm, float ll) {
    if (a.lse != nullptr)
      a.lse[(static_cast<int64_t>(b) * a.Q + (r0 + r) / p.G) * a.q_heads + h * p.G + (r0 + r) % p.G] =
          ll > 0.0f || ll != ll ? (mm + log2f(ll)) * 0.693147180559945309f : kNegInf;
  };
  // a sum of ranges with maxima m, m' and sums l: outputs' factor
  auto out_factor = [](float mm, float ll, float nn) {
    return ll > 0.0f || ll != ll ? (nn == kNegInf ? 0.0f : exp2f(nn - mm)) / ll : 0.0f;
  };
  const int64_t slot = pair * p.splits + sp;
  for (int it = threadIdx.x; it < nrows * (D / 4); it += kAThreads) {
    const int r = it / (D / 4), c = (it % (D / 4)) * 4;
    float M = kNegInf, N = kNegInf, L = 0.0f;
#pragma unroll
    for (int w = 0; w < kAWarps; ++w) {
      M = fmaxf(M, st_m[w][r]);
      N = fmaxf(N, st_n[w][r]);
    }
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kAWarps; ++w) {
      L += st_m[w][r] != kNegInf ? st_l[w][r] * ex2(st_m[w][r] - M) : st_l[w][r];  // (0, or the NaN of a NaN query)
      const float k = st_n[w][r] != kNegInf ? ex2(st_n[w][r] - N) : 0.0f;
      const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                        (w * kARows + r) * ST::kMergeRow + c / (D / 4) * ST::kQuarter + c % (D / 4));
      if (k > 0.0f || k != k) {
        v.x += u.x * k;
        v.y += u.y * k;
        v.z += u.z * k;
        v.w += u.w * k;
      }
    }
    if (active == 1) {
      store_row(r, c, v, out_factor(M, L, N));
      if (c == 0) store_lse(r, M, L);
    } else {
      *reinterpret_cast<float4*>(p.part_o + (slot * p.kept + r) * D + c) = v;
      if (c == 0) *reinterpret_cast<float4*>(p.part_stat + (slot * p.kept + r) * 4) = make_float4(M, L, N, 0.0f);
    }
  }
  if (active == 1) return;

  // ---- the CTA that comes last joins the ranges, in their order
  __threadfence();
  __syncthreads();
  int* counter = reinterpret_cast<int*>(a.ws) + pair;
  if (threadIdx.x == 0) last_s = atomicAdd(counter, 1) == active - 1;
  __syncthreads();
  if (!last_s) return;
  __threadfence();
  if (threadIdx.x == 0) *counter = 0;
  float* stat = reinterpret_cast<float*>(smem);  // [active][kept][4], then each range's factor in place of m'
  const int64_t slot0 = pair * p.splits;
  for (int it = threadIdx.x; it < active * p.kept; it += kAThreads)
    if (it % p.kept < nrows)
      reinterpret_cast<float4*>(stat)[it] = __ldcg(reinterpret_cast<const float4*>(p.part_stat + slot0 * p.kept * 4) + it);
  __syncthreads();
  for (int it = threadIdx.x; it < nrows * (D / 4); it += kAThreads) {
    const int r = it / (D / 4), c = (it % (D / 4)) * 4;
    float M = kNegInf, N = kNegInf, L = 0.0f;
    for (int s = 0; s < active; ++s) {
      M = fmaxf(M, stat[(s * p.kept + r) * 4]);
      N = fmaxf(N, stat[(s * p.kept + r) * 4 + 2]);
    }
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < active; ++s) {
      const float4 q4 = reinterpret_cast<const float4*>(stat)[s * p.kept + r];
      const float4 u = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((slot0 + s) * p.kept + r) * D + c));
      L += q4.x != kNegInf ? q4.y * ex2(q4.x - M) : q4.y;
      const float k = q4.z != kNegInf ? ex2(q4.z - N) : 0.0f;
      if (k > 0.0f || k != k) {
        v.x += u.x * k;
        v.y += u.y * k;
        v.z += u.z * k;
        v.w += u.w * k;
      }
    }
    store_row(r, c, v, out_factor(M, L, N));
    if (c == 0) store_lse(r, M, L);
  }
}

}  // namespace

// Counters first, the ranges' results at the workspace's end: with both bounded by what grows with B, Q and
// max_len, a workspace serves every smaller call, whose results never reach another's counters.
size_t attention_fp4_workspace_bytes(int B, int Q, int q_heads, int kv_heads, int D, int64_t max_len) {
  const Plan p = plan(B, Q, q_heads, kv_heads, max_len);
  const int64_t pairs = static_cast<int64_t>(B) * kv_heads * p.groups;
  int64_t by_length = (max_len + kLongRange - 1) / kLongRange;
  if (by_length > kMaxSplits) by_length = kMaxSplits;
  const int64_t a = pairs + 4 * kSlots, b = pairs * by_length;
  return counters_bytes(pairs) +
         static_cast<size_t>(a > b ? a : b) * rows_kept(Q, q_heads / kv_heads) * (static_cast<size_t>(D) + 4) * 4;
}

cudaError_t launch_attention_fp4(const AttentionFp4Args& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const Plan pl = plan(a.B, a.Q, a.q_heads, a.c.heads, static_cast<int64_t>(a.max_pages) * a.c.page);
  const int64_t pairs = static_cast<int64_t>(a.B) * a.c.heads * pl.groups;
  Params p;
  p.a = a;
  p.groups = pl.groups;
  p.splits = pl.splits;
  p.G = a.q_heads / a.c.heads;
  p.kept = rows_kept(a.Q, p.G);
  const size_t kept_rows = static_cast<size_t>(pairs) * pl.splits * p.kept;
  p.part_o = reinterpret_cast<float*>(a.ws + (a.ws_bytes / 16 * 16 - kept_rows * (a.c.D + 4) * 4));
  p.part_stat = p.part_o + kept_rows * a.c.D;
  void* args[] = {&p};
  if (a.c.D == 64)
    return launch_pdl(reinterpret_cast<const void*>(attention_fp4_kernel<64>), dim3(static_cast<unsigned>(pairs * pl.splits)),
                      dim3(kAThreads), AStage<64>::kSmem, stream, args);
  return launch_pdl(reinterpret_cast<const void*>(attention_fp4_kernel<128>), dim3(static_cast<unsigned>(pairs * pl.splits)),
                    dim3(kAThreads), AStage<128>::kSmem, stream, args);
}

}  // namespace mtp
