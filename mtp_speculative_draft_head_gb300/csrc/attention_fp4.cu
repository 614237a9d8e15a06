// Attention of a few query rows per sequence over its pages of the FP4 cache (a draft step's row, or a
// verification's rows):
//   o_i = sum_j p_ij v_j,   p_ij = softmax_j( scale q_i . k_j ),   j < length - n + i + 1
//
// A CTA takes one sequence, one key head, up to 16 of the rows that share it (n rows x the query heads of
// the group) and a range of the sequence's tokens; its four warps take 32 tokens at a time in turn, each
// with running maxima, sum and outputs of its own, so nothing synchronises the warps until the range
// ends. The ranges' results meet in the workspace, where the CTA that finishes last joins them in order.
//
// Tokens are the M side of warp-level MMAs (m16n8k16, f16 operands, fp32 sums), rows the N side, eight a
// tile: S^T = K Q^T, then O^T += V^T P^T with P^T out of S^T by a transposition within the warp. A step of one
// row per sequence pays for eight, and every key and value is widened once for all rows of the CTA. Codes
// go from shared memory to MMA operands in registers: the hardware conversion makes f16 pairs of them, block
// scales multiply in f16, which is exact (six significant bits). A value pair is the same column of two
// tokens: their codes are interleaved as nibbles before the conversion. The fp32 row scales
// stay out of the operands: a key's multiplies its scores, a value's goes into the exponent of its
// weight. With x_ij the score in powers of two and v_j = r_j u_j, the warp keeps
//   l_i = sum_j 2^(x_ij - m_i)      and      O_i = sum_j 2^(x_ij + log2 r_j - m'_i) u_j
// with separate maxima m and m', so the f16 weights of O are of order one whatever the values' sizes.
// Query rows are BF16 values times a power of two that brings their largest near 2^7: exact in f16 but
// for elements below 2^-24 of that. The maxima move only when a score passes one by 2^8; until then no lane
// asks another for its scores.
//
// A warp's step arrives by 16-byte asynchronous copies into a ring of its own: codes, block scales and row scales of 32
// tokens are six contiguous pieces of a page, so a lane's addresses are a few multiply-adds. (Bulk copies of the pieces
// took more instructions: their operands go through uniform registers, one lane after another.)
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
constexpr int kRowTile = 8;                  // rows of an MMA
constexpr int kMaxTiles = 2;                 // row tiles of a CTA
constexpr int kAStages = 2;
constexpr int kMaxSplits = 128;
constexpr int kSlots = 152 * 4;              // CTAs that run at once, about
constexpr int kLongRange = 4096;             // a range of tokens is no longer than this where splits allow,
constexpr int kShortRange = 512;             // and no shorter than this once every SM has its CTAs

template <int D>
struct AStage {  // one warp's stage: keys and values of 32 tokens
  static constexpr int kCode = kStep * D / 2, kScale = kStep * D / kFp4Block, kRow = kStep * 4;
  static constexpr int kV = kCode + kScale + kRow;
  static constexpr int kBytes = 2 * kV;
  // merge buffer, a tile of rows at a time: eighths of a row (one per g) with gaps against bank conflicts
  static constexpr int kEighth = D / 8 + 4, kMergeRow = 8 * kEighth + 4;
  static constexpr size_t kRing = static_cast<size_t>(kAWarps) * kAStages * kBytes;
  static constexpr size_t kMerge = static_cast<size_t>(kAWarps) * kRowTile * kMergeRow * 4;
  static constexpr size_t kStats = static_cast<size_t>(kMaxSplits) * kRowTile * 16;
  static constexpr size_t kLarger = kRing > kMerge ? kRing : kMerge;
  static constexpr size_t kSmem = kLarger > kStats ? kLarger : kStats;
};

struct Plan {
  int groups, splits, tiles;  // tiles: of eight rows, of a CTA
};
// Ranges per (sequence, key head, group of rows): enough for two CTAs per one that runs (sequences are unequal),
// but fewer rather than ranges below kShortRange; at least one for every CTA that can run, and enough for ranges
// of at most kLongRange, as far as kMaxSplits go.
inline Plan plan(int B, int Q, int q_heads, int kv_heads, int64_t max_len) {
  Plan p;
  const int rows = Q * (q_heads / kv_heads);
  // as few CTAs as hold the rows, then as few tiles in each
  const int tiles = (rows + kRowTile - 1) / kRowTile;
  p.groups = (tiles + kMaxTiles - 1) / kMaxTiles;
  p.tiles = (tiles + p.groups - 1) / p.groups;
  const int64_t pairs = static_cast<int64_t>(B) * kv_heads * p.groups;
  const int64_t chunks = (max_len + kChunkTok - 1) / kChunkTok;
  int64_t s = (2 * kSlots + pairs - 1) / pairs;
  const int64_t wave = (kSlots + pairs - 1) / pairs, by_length = (max_len + kLongRange - 1) / kLongRange;
  if (s > max_len / kShortRange) s = max_len / kShortRange;
  if (s < wave) s = wave;
  if (s < by_length) s = by_length;
  if (s > chunks) s = chunks;
  if (s > kMaxSplits) s = kMaxSplits;
  p.splits = s < 1 ? 1 : static_cast<int>(s);
  return p;
}
inline int rows_kept(int Q, int G) { return Q * G < kMaxTiles * kRowTile ? Q * G : kMaxTiles * kRowTile; }
inline size_t counters_bytes(int64_t pairs) { return (static_cast<size_t>(pairs) * 4 + 255) / 256 * 256; }

struct Params {
  AttentionFp4Args a;
  int groups, splits, kept, G;
  float* part_o;     // [pairs, splits, kept, D]
  float* part_stat;  // [pairs, splits, kept, 4]: m, l, m'
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one load");
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}
// (not volatile: the compiler may move these past one another)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
constexpr float kNegInf = -INFINITY;
// The transposed 8 x 8 matrix of 16-bit elements (two a lane).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Token of row r of a unit of 16: pairs of rows stay pairs of tokens, every other one the other way round, so that
// neither the keys' nor the values' reads of shared memory meet on the same banks.
__device__ __forceinline__ int token_of(int r) { return r ^ ((r >> 1) & 1); }

template <bool V>
struct Edge {
  static constexpr bool value = V;
};

// NT tiles of eight rows.
template <int D, int NT>
__global__ void __launch_bounds__(kAThreads, NT == 2 ? 3 : D == 64 ? 5 : 4) attention_fp4_kernel(const Params p) {
  using ST = AStage<D>;
  constexpr int kRows = NT * kRowTile;
  constexpr int kKSteps = D / 16, kBlocks = D / kFp4Block;
  constexpr int kKWords = D / 32, kVWords = D / 64;  // words of codes that a thread takes of a key, of a value
  constexpr int kOTiles = D / 16;                    // tiles of 16 columns of the outputs
  constexpr int kUnits = 2;                          // units of 16 tokens of a step
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float st_m[kAWarps][kRowTile], st_l[kAWarps][kRowTile], st_n[kAWarps][kRowTile];
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
  const int r0 = grp * kRows;
  int nrows = n * p.G - r0;  // rows of this CTA
  if (nrows <= 0) return;
  if (nrows > kRows) nrows = kRows;
  int seen = len - n + (r0 + nrows - 1) / p.G + 1;  // tokens that its last row sees
  if (seen < 0) seen = 0;
  const int chunks = (seen + kChunkTok - 1) / kChunkTok;
  const int per = (chunks + p.splits - 1) / p.splits;  // chunks of a range
  const int active = chunks == 0 ? 1 : (chunks + per - 1) / per;
  if (sp >= active) return;
  const int begin = sp * per * kChunkTok;
  const int end = min(seen, begin + per * kChunkTok);

  // ---- copies: a warp's steps into its own ring
  const uint32_t ring = smem_addr(smem) + warp * kAStages * ST::kBytes;
  const int first = begin + warp * kStep;
  const int* table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int page_shift = __ffs(a.c.page) - 1;
  // Addresses: what is the lane's own, plus units of 16 rows of the cache times their bytes.
  constexpr int kPieces = D / 32;                      // 16-byte pieces of codes a lane, key or value
  constexpr int kScalePieces = ST::kScale / 16;        // of block scales, all lanes
  const uint32_t page_units = static_cast<uint32_t>(2 * a.c.heads * a.c.page) / 16;
  const int64_t head_rows = static_cast<int64_t>(h) * a.c.page, to_v = static_cast<int64_t>(a.c.heads) * a.c.page;
  const uint8_t* k_at = a.c.q + head_rows * (D / 2) + lane * 16;
  const int64_t code_to_v = to_v * (D / 2);
  const int s_kind = lane / kScalePieces & 1, s_piece = lane % kScalePieces, s_half = s_piece / (kScalePieces / 2);
  const uint8_t* s_at = a.c.bs + (head_rows + s_kind * to_v) * kBlocks + s_piece % (kScalePieces / 2) * 16;
  const uint32_t s_to = ring + s_kind * ST::kV + ST::kCode + s_piece * 16;
  const int r_kind = lane >> 3 & 1, r_half = lane >> 2 & 1;
  const float* r_at = a.c.rs + head_rows + r_kind * to_v + (lane & 3) * 4;
  const uint32_t r_to = ring + r_kind * ST::kV + ST::kCode + ST::kScale + (lane & 7) * 16;
  auto copy_step = [&](int tok0, int stage, int pg0, int pg1) {
    const uint32_t d = stage * ST::kBytes;
    const uint32_t u0 = pg0 * page_units + static_cast<uint32_t>(tok0 & (a.c.page - 1)) / 16;
    const uint32_t u1 = pg1 * page_units + static_cast<uint32_t>((tok0 + 16) & (a.c.page - 1)) / 16;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if ((half ? pg1 : pg0) < 0) continue;  // (the whole warp)
      const uint8_t* k = k_at + static_cast<uint64_t>(half ? u1 : u0) * (8 * D);
      const uint8_t* v = k + code_to_v;
#pragma unroll
      for (int i = 0; i < kPieces / 2; ++i) {
        cp16(ring + d + lane * 16 + (half * kPieces / 2 + i) * 512, k + i * 512);
        cp16(ring + d + ST::kV + lane * 16 + (half * kPieces / 2 + i) * 512, v + i * 512);
      }
    }
    if (lane < 2 * kScalePieces && (s_half ? pg1 : pg0) >= 0)
      cp16(s_to + d, s_at + static_cast<uint64_t>(s_half ? u1 : u0) * (16 * kBlocks));
    if (lane < 16 && (r_half ? pg1 : pg0) >= 0) cp16(r_to + d, r_at + static_cast<uint64_t>(r_half ? u1 : u0) * 16);
  };
  // Pages of the coming steps: 16 steps at a time, lane 2 i (2 i + 1) the first (second) half of the i-th; -1: none (its
  // tokens are left out).
  int pages = 0, pages_left = 0;
  int next_tok = first;
  uint32_t out_of = 0;  // bits 2 s and 2 s + 1: the halves of stage s have no page
  auto copy_next = [&](int stage) {
    if (next_tok < end) {
      if (pages_left == 0) {
        const int tok = next_tok + (lane >> 1) * kChunkTok + (lane & 1) * 16;
        pages = -1;
        if (tok < end) {
          pages = table[tok >> page_shift];
          if (pages < 0 || pages >= a.c.pages) {
            store_status(a.status, MTP_ERR_ARG);
            pages = -1;
          }
        }
        pages_left = 32;
      }
      const int pg0 = __shfl_sync(0xffffffffu, pages, 32 - pages_left), pg1 = __shfl_sync(0xffffffffu, pages, 33 - pages_left);
      pages_left -= 2;
      copy_step(next_tok, stage, pg0, pg1);
      out_of = (out_of & ~(3u << (2 * stage))) | (pg0 < 0 ? 1u << (2 * stage) : 0u) | (pg1 < 0 ? 2u << (2 * stage) : 0u);
      next_tok += kChunkTok;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAStages - 1; ++i) copy_next(i);

  // ---- queries: row g of each tile as an f16 operand
  uint32_t qb[NT][kKSteps][2];
  // From a row's MMA sums to scores in powers of two: f1 times the key's row scale times f2, so that no product
  // leaves the fp32 range on the way. Of this thread's score columns, rows 2 t and 2 t + 1 of a tile.
  uint64_t f1[NT], f2[NT];
  int limit[NT][2];  // tokens that such a row sees
  int least = 0x7FFFFFFF;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rr = nt * kRowTile + g;
    const bool on = rr < nrows;
    const int r = r0 + (on ? rr : 0);
    const uint16_t* src = a.query + (static_cast<int64_t>(b) * a.Q + r / p.G) * a.ld_q +
                          static_cast<int64_t>(h * p.G + r % p.G) * D + t * (D / 4);
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
    const float d1 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
    const float d2 = a.scale * 1.44269504088896341f * __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
    f1[nt] = f2_pack(__shfl_sync(0xffffffffu, d1, 8 * t), __shfl_sync(0xffffffffu, d1, 8 * t + 4));
    f2[nt] = f2_pack(__shfl_sync(0xffffffffu, d2, 8 * t), __shfl_sync(0xffffffffu, d2, 8 * t + 4));
#pragma unroll
    for (int s = 0; s < kKSteps; ++s) {
      qb[nt][s][0] = f16x2_bits(bf16_lo(u[2 * s]) * up, bf16_hi(u[2 * s]) * up);
      qb[nt][s][1] = f16x2_bits(bf16_lo(u[2 * s + 1]) * up, bf16_hi(u[2 * s + 1]) * up);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int rc = nt * kRowTile + 2 * t + c;
      // (a row that is not there: whatever it sees)
      limit[nt][c] = rc < nrows ? len - n + (r0 + rc) / p.G + 1 : 0x7FFFFFFF;
      least = min(least, limit[nt][c]);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);  // tokens before it are seen by every row

  float o[NT][kOTiles][4];
  float m[NT][2], mv[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < kOTiles; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = mv[nt][c] = kNegInf;
      l[nt][c] = 0.0f;
    }
  }

  int stage = 0;
  auto step = [&](int tok0, auto edge_tag) {
    constexpr bool edge = decltype(edge_tag)::value;
    const uint8_t* kb = smem + (warp * kAStages + stage) * ST::kBytes;
    const uint8_t* vb = kb + ST::kV;
    const float* kr = reinterpret_cast<const float*>(kb + ST::kCode + ST::kScale);
    const float* vr = reinterpret_cast<const float*>(vb + ST::kCode + ST::kScale);
    const uint32_t gone = (out_of >> (2 * stage)) & 3u;

    {
      // ---- scores: x[unit][tile][2 i + c], token token_of(g + 8 i), row 2 t + c
      float x[kUnits][NT][4], lv[kUnits][2];
#pragma unroll
      for (int un = 0; un < kUnits; ++un) {
        const int t0 = un * 16 + token_of(g);
        uint32_t w[2][kKWords], sc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_words<kKWords>(kb + (t0 + 8 * i) * (D / 2) + t * (D / 8), w[i]);
          if constexpr (D == 128) {
            const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(kb + ST::kCode + (t0 + 8 * i) * kBlocks + 2 * t));
            sc[i][0] = __byte_perm(s2, s2, 0x1010);
            sc[i][1] = __byte_perm(s2, s2, 0x3232);
          } else {
            sc[i][0] = sc[i][1] = e4m3x2_to_f16x2(kb[ST::kCode + (t0 + 8 * i) * kBlocks + t] * 0x0101u);
          }
        }
        float even[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // one tile: every other step's sums, so that two chains of MMAs run
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[un][nt][c] = 0.0f;
#pragma unroll
        for (int i = 0; i < kKWords; ++i) {
          uint32_t v[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            e2m1x8_to_f16x2x4(w[k][i], v[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k][e] = f16x2_mul(v[k][e], sc[k][i < kKWords / 2 ? 0 : 1]);
          }
          const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]}, a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(NT == 1 ? even : x[un][nt], a0, qb[nt][2 * i][0], qb[nt][2 * i][1]);
            mma(x[un][nt], a1, qb[nt][2 * i + 1][0], qb[nt][2 * i + 1][1]);
          }
        }
        // to powers of two
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float rk = kr[t0 + 8 * i];
          const uint64_t rk2 = f2_pack(rk, rk);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint64_t s = f2_pack(x[un][nt][2 * i], x[un][nt][2 * i + 1]);
            if constexpr (NT == 1) s = f2_add(s, f2_pack(even[2 * i], even[2 * i + 1]));
            const uint64_t y = f2_mul(f2_mul(f2_mul(s, f1[nt]), rk2), f2[nt]);
            x[un][nt][2 * i] = f2_lo(y);
            x[un][nt][2 * i + 1] = f2_hi(y);
          }
          float rv = vr[t0 + 8 * i];
          if constexpr (edge) {
            const int tok = tok0 + t0 + 8 * i;
            const bool none = tok >= end || ((gone >> un) & 1u) != 0u;
            if (none) rv = 1.0f;  // (its stage holds anything)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (none || tok >= limit[nt][c]) x[un][nt][2 * i + c] = kNegInf;
          }
          lv[un][i] = lg2(rv);
        }
      }

      // ---- the maxima, if a score has passed one by 2^8
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float xm = kNegInf, ym = kNegInf;
#pragma unroll
          for (int un = 0; un < kUnits; ++un)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              xm = fmaxf(xm, x[un][nt][2 * i + c]);
              ym = fmaxf(ym, x[un][nt][2 * i + c] + lv[un][i]);
            }
          up |= xm > m[nt][c] + 8.0f || ym > mv[nt][c] + 8.0f;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float xm = kNegInf, ym = kNegInf;
#pragma unroll
            for (int un = 0; un < kUnits; ++un)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                xm = fmaxf(xm, x[un][nt][2 * i + c]);
                ym = fmaxf(ym, x[un][nt][2 * i + c] + lv[un][i]);
              }
#pragma unroll
            for (int k = 4; k < 32; k *= 2) {
              xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, k));
              ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, k));
            }
            const float to = fmaxf(m[nt][c], xm), to_v = fmaxf(mv[nt][c], ym);
            l[nt][c] *= m[nt][c] == kNegInf ? 0.0f : ex2(m[nt][c] - to);
            const float k = mv[nt][c] == kNegInf ? 0.0f : ex2(mv[nt][c] - to_v);
            m[nt][c] = to;
            mv[nt][c] = to_v;
#pragma unroll
            for (int j = 0; j < kOTiles; ++j) {
              o[nt][j][c] *= k;
              o[nt][j][2 + c] *= k;
            }
          }
      }

      // ---- weights, transposed: tokens along k
      uint32_t pb[kUnits][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float nm[2], nv[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          nm[c] = m[nt][c] == kNegInf ? 0.0f : m[nt][c];
          nv[c] = mv[nt][c] == kNegInf ? 0.0f : mv[nt][c];
        }
#pragma unroll
        for (int un = 0; un < kUnits; ++un)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x0 = x[un][nt][2 * i], x1 = x[un][nt][2 * i + 1], v = lv[un][i];
            l[nt][0] += ex2(x0 - nm[0]);
            l[nt][1] += ex2(x1 - nm[1]);
            pb[un][nt][i] = transpose8x8(f16x2_bits(ex2(x0 + v - nv[0]), ex2(x1 + v - nv[1])));
          }
      }

      // ---- outputs
#pragma unroll
      for (int un = 0; un < kUnits; ++un) {
        uint32_t lo[2][kVWords], hi[2][kVWords], s2[2];  // even and odd columns of pairs of tokens, and their block scales
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ta = un * 16 + 8 * k + token_of(2 * t), tb = un * 16 + 8 * k + token_of(2 * t + 1);
          uint32_t wa[kVWords], wb[kVWords];
          load_words<kVWords>(vb + ta * (D / 2) + g * (D / 16), wa);
          load_words<kVWords>(vb + tb * (D / 2) + g * (D / 16), wb);
#pragma unroll
          for (int i = 0; i < kVWords; ++i) {
            lo[k][i] = (wa[i] & 0x0F0F0F0Fu) | ((wb[i] << 4) & 0xF0F0F0F0u);
            hi[k][i] = ((wa[i] >> 4) & 0x0F0F0F0Fu) | (wb[i] & 0xF0F0F0F0u);
          }
          uint32_t sa = vb[ST::kCode + ta * kBlocks + (D == 128 ? g : g >> 1)];
          uint32_t sb = vb[ST::kCode + tb * kBlocks + (D == 128 ? g : g >> 1)];
          if constexpr (edge) {
            const bool none = ((gone >> un) & 1u) != 0u;
            if (none || tok0 + ta >= end) sa = 0u;
            if (none || tok0 + tb >= end) sb = 0u;
          }
          s2[k] = e4m3x2_to_f16x2(sa | (sb << 8));
        }
#pragma unroll
        for (int i = 0; i < kVWords; ++i) {
          uint32_t v[2][2][4];  // [pair][even, odd][column]
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            e2m1x8_to_f16x2x4(lo[k][i], v[k][0]);
            e2m1x8_to_f16x2x4(hi[k][i], v[k][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[k][0][e] = f16x2_mul(v[k][0][e], s2[k]);
              v[k][1][e] = f16x2_mul(v[k][1][e], s2[k]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t av[4] = {v[0][0][e], v[0][1][e], v[1][0][e], v[1][1][e]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(o[nt][4 * i + e], av, pb[un][nt][0], pb[un][nt][1]);
          }
        }
      }
    }
  };
  for (int tok0 = first; tok0 < end; tok0 += kChunkTok) {
    copy_next(stage == 0 ? kAStages - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAStages - 1) : "memory");
    __syncwarp();
    // (edge: some token of the step is not there, or not seen by some row)
    if (tok0 + kStep > least || tok0 + kStep > end || ((out_of >> (2 * stage)) & 3u) != 0u)
      step(tok0, Edge<true>{});
    else
      step(tok0, Edge<false>{});
    __syncwarp();  // the stage has been read by all lanes
    if (++stage == kAStages) stage = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

  // ---- the warps' results, a tile of rows at a time
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
  auto add = [](float4& v, const float4& u, float k) {
    if (k > 0.0f || k != k) {
      v.x += u.x * k;
      v.y += u.y * k;
      v.z += u.z * k;
      v.w += u.w * k;
    }
  };
  const int64_t slot = pair * p.splits + sp;
  float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (nt * kRowTile >= nrows) break;
    __syncthreads();  // the rings, or the tile before, have been read
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float s = l[nt][c];
#pragma unroll
      for (int k = 4; k < 32; k *= 2) s += __shfl_xor_sync(0xffffffffu, s, k);
      if (g == 0) {
        st_m[warp][2 * t + c] = m[nt][c];
        st_l[warp][2 * t + c] = s;
        st_n[warp][2 * t + c] = mv[nt][c];
      }
      float* dst = merge + (warp * kRowTile + 2 * t + c) * ST::kMergeRow + g * ST::kEighth;
#pragma unroll
      for (int j = 0; j < kOTiles; j += 2)
        *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nt][j][c], o[nt][j][2 + c], o[nt][j + 1][c], o[nt][j + 1][2 + c]);
    }
    __syncthreads();
    const int here = min(nrows - nt * kRowTile, kRowTile);
    for (int it = threadIdx.x; it < here * (D / 4); it += kAThreads) {
      const int rt = it / (D / 4), r = nt * kRowTile + rt, c = (it % (D / 4)) * 4;
      float M = kNegInf, N = kNegInf, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kAWarps; ++w) {
        M = fmaxf(M, st_m[w][rt]);
        N = fmaxf(N, st_n[w][rt]);
      }
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kAWarps; ++w) {
        L += st_m[w][rt] != kNegInf ? st_l[w][rt] * ex2(st_m[w][rt] - M) : st_l[w][rt];  // (0, or the NaN of a NaN query)
        add(v, *reinterpret_cast<const float4*>(merge + (w * kRowTile + rt) * ST::kMergeRow + c / (D / 8) * ST::kEighth + c % (D / 8)),
            st_n[w][rt] != kNegInf ? ex2(st_n[w][rt] - N) : 0.0f);
      }
      if (active == 1) {
        store_row(r, c, v, out_factor(M, L, N));
        if (c == 0) store_lse(r, M, L);
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * p.kept + r) * D + c) = v;
        if (c == 0) *reinterpret_cast<float4*>(p.part_stat + (slot * p.kept + r) * 4) = make_float4(M, L, N, 0.0f);
      }
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
  float4* stat = reinterpret_cast<float4*>(smem);  // [active][8]
  const int64_t slot0 = pair * p.splits;
  for (int nt = 0; nt * kRowTile < nrows; ++nt) {
    const int here = min(nrows - nt * kRowTile, kRowTile);
    __syncthreads();
    for (int it = threadIdx.x; it < active * kRowTile; it += kAThreads)
      if (it % kRowTile < here)
        stat[it] = __ldcg(reinterpret_cast<const float4*>(p.part_stat) + (slot0 + it / kRowTile) * p.kept + nt * kRowTile + it % kRowTile);
    __syncthreads();
    for (int it = threadIdx.x; it < here * (D / 4); it += kAThreads) {
      const int rt = it / (D / 4), r = nt * kRowTile + rt, c = (it % (D / 4)) * 4;
      float M = kNegInf, N = kNegInf, L = 0.0f;
      for (int s = 0; s < active; ++s) {
        M = fmaxf(M, stat[s * kRowTile + rt].x);
        N = fmaxf(N, stat[s * kRowTile + rt].z);
      }
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int s = 0; s < active; ++s) {
        const float4 q4 = stat[s * kRowTile + rt];
        const float4 u = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((slot0 + s) * p.kept + r) * D + c));
        L += q4.x != kNegInf ? q4.y * ex2(q4.x - M) : q4.y;
        add(v, u, q4.z != kNegInf ? ex2(q4.z - N) : 0.0f);
      }
      store_row(r, c, v, out_factor(M, L, N));
      if (c == 0) store_lse(r, M, L);
    }
  }
}

template <int D>
const void* kernel_of(int tiles) {
  return tiles == 1 ? reinterpret_cast<const void*>(attention_fp4_kernel<D, 1>)
                    : reinterpret_cast<const void*>(attention_fp4_kernel<D, kMaxTiles>);
}

}  // namespace

// Counters first, the ranges' results at the workspace's end: with both bounded by what grows with B, Q and
// max_len, a workspace serves every smaller call, whose results never reach another's counters.
size_t attention_fp4_workspace_bytes(int B, int Q, int q_heads, int kv_heads, int D, int64_t max_len) {
  const Plan p = plan(B, Q, q_heads, kv_heads, max_len);
  const int64_t pairs = static_cast<int64_t>(B) * kv_heads * p.groups;
  int64_t by_length = (max_len + kLongRange - 1) / kLongRange;
  if (by_length > kMaxSplits) by_length = kMaxSplits;
  const int64_t a = pairs + 2 * kSlots, b = pairs * by_length;
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
  return launch_pdl(a.c.D == 64 ? kernel_of<64>(pl.tiles) : kernel_of<128>(pl.tiles), dim3(static_cast<unsigned>(pairs * pl.splits)),
                    dim3(kAThreads), a.c.D == 64 ? AStage<64>::kSmem : AStage<128>::kSmem, stream, args);
}

}  // namespace mtp
