// Attention of a few query rows per sequence over its pages of the FP4 cache (a draft step's row, or a
// verification's rows):
//   o_i = sum_j p_ij v_j,   p_ij = softmax_j( scale q_i . k_j ),   j < length - n + i + 1
//
// A round is 128 tokens of one sequence, one key head and up to 16 of the rows that share it (n rows x the
// query heads of the group); the four warps take 32 of its tokens each, with running maxima, sum and outputs
// of their own, so nothing synchronises them until a range of rounds ends. As many CTAs as run at once take
// equal shares of all rounds, one after another: sequences differ in length, and a CTA that starts and one that
// ends cost about 5 us together, so ranges cut sequence by sequence, in two waves of CTAs, took 93 and 143 us
// where this takes 82 and 124 (the sizes below). Where it takes no more CTAs, every group of rows begins a share (16
// instead of 20 us for 7 sequences of up to 5000 tokens). Many short groups, and a few very short ones, have CTAs of
// their own (see Plan). A group's ranges meet in the workspace, where the CTA that finishes last joins them in order.
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
// asks another for its scores, and the second weight is the first times r_j 2^(m_i - m'_i).
//
// A warp's step arrives by 16-byte asynchronous copies into a ring of its own: codes, block scales and row scales of 32
// tokens are six contiguous pieces of a page, so a lane's addresses are a few multiply-adds. (Bulk copies of the pieces
// took more instructions: their operands go through uniform registers, one lane after another.)
//
// Measured at 8 key heads of 6 query heads, D = 128: one row of each of 16 sequences of up to 32768 tokens (369 MB) 82 us,
// 4.5 TB/s; five rows of each of 16 of up to 16384 (186 MB) 124 us; one sequence of 2048 tokens 14 us (block tables as
// wide as the longest sequence, here and below). Instructions
// bound it, not memory: a lane's word of eight codes with its conversions, scales and one row tile's MMA takes 18 cycles of an
// SM's quarter, and a second tile of rows 8 more. Four row tiles a warp left too few warps (180 us for the five rows);
// wide operands in shared memory for the larger tensor-core instructions took longer to write than they saved (187 us).
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
constexpr int kMaxRanges = 128;              // ranges that one sequence is cut into
constexpr int kSms = 152;
constexpr int kMaxCtas = kSms * 5;           // that share rounds out
constexpr int kLongRange = 4096;

template <int D>
struct AStage {  // one warp's stage: keys and values of 32 tokens
  static constexpr int kCode = kStep * D / 2, kScale = kStep * D / kFp4Block, kRow = kStep * 4;
  static constexpr int kV = kCode + kScale + kRow;
  static constexpr int kBytes = 2 * kV;
  // merge buffer, a tile of rows at a time: eighths of a row (one per g) with gaps against bank conflicts
  static constexpr int kEighth = D / 8 + 4, kMergeRow = 8 * kEighth + 4;
  static constexpr size_t kRing = static_cast<size_t>(kAWarps) * kAStages * kBytes;
  static constexpr size_t kMerge = static_cast<size_t>(kAWarps) * kRowTile * kMergeRow * 4;
  static constexpr size_t kStats = static_cast<size_t>(kMaxRanges) * kRowTile * 16;
  static constexpr size_t kLarger = kRing > kMerge ? kRing : kMerge;
  static constexpr size_t kSmem = kLarger > kStats ? kLarger : kStats;
};

// As few CTAs as hold the rows of a sequence's key head, then as few tiles in each.
struct Groups {
  int groups, tiles;
  Groups(int Q, int G) {
    const int all = (Q * G + kRowTile - 1) / kRowTile;
    groups = (all + kMaxTiles - 1) / kMaxTiles;
    tiles = (all + groups - 1) / groups;
  }
};
constexpr int ctas_per_sm(int D, int tiles) { return tiles == 2 ? 3 : D == 64 ? 5 : 4; }
inline int rows_kept(int Q, int G) { return Q * G < kMaxTiles * kRowTile ? Q * G : kMaxTiles * kRowTile; }
inline size_t counters_bytes(int64_t pairs) { return (static_cast<size_t>(pairs) * 4 + 255) / 256 * 256; }
// The CTAs of a launch. Either no more than run at once, which share the rounds out: the GPU is evenly busy to the end, but each
// CTA first sums up all lengths, and groups of rows are cut where shares end. Or one for every range of at most
// kLongRange tokens of every group: their starts hide under others' work, but the last ones run alone. The latter where there
// are more groups than CTAs at once, and tables too narrow for their number: us with shares and with ranges for 800 groups
// of up to 500 tokens 24 and 20, of up to 3000 66 and 68, for 2048 groups of up to 500 61 and 38, 4000 169 and 159, 16000
// 534 and 557. Or, where the whole call is no more than a round a CTA, one for every round (8 groups of 2048 tokens: 13.9 us,
// 14.8 in shares). The host knows the table's width only: with lengths well below it the last two are not taken (in a table of 32768
// tokens the 8 groups of 2048 take 16 to 17 us and the 2048 groups of up to 500 take 59).
struct Plan {
  int ctas, splits;  // splits: 0 where CTAs share rounds out, else ranges per group
  Plan(int64_t pairs, int64_t max_len, int per_sm, int sms) {
    const int64_t rounds = rounds_of(max_len), room = kSms * per_sm;
    const int at_once = sms * per_sm < kMaxCtas ? sms * per_sm : kMaxCtas;
    splits = 0;
    if (pairs * rounds <= at_once && rounds <= kMaxRanges)
      splits = static_cast<int>(rounds);
    else if (pairs > room && rounds * room < 16 * pairs)
      splits = static_cast<int>(ranges_of(max_len));
    ctas = static_cast<int>(splits > 0 ? pairs * splits : pairs * rounds < at_once ? pairs * rounds : at_once);
  }
  size_t parts() const { return splits == 0 ? 2 * static_cast<size_t>(ctas) : splits == 1 ? 0 : static_cast<size_t>(ctas); }
  static int64_t rounds_of(int64_t max_len) { return (max_len + kChunkTok - 1) / kChunkTok; }
  static int64_t ranges_of(int64_t max_len) {
    const int64_t r = (max_len + kLongRange - 1) / kLongRange;
    return r < kMaxRanges ? r : kMaxRanges;
  }
  // No fewer than the parts of any call of no more groups and no larger max_len: with ranges, their number is below
  // groups / (2 CTAs at once) + 1; with a CTA a round there is a part for each, half of what shares take.
  static size_t most_parts(int64_t pairs, int64_t max_len) {
    constexpr int64_t kFewest = kSms * ctas_per_sm(128, kMaxTiles);
    const int64_t rounds = pairs * rounds_of(max_len), shares = 2 * (rounds < kMaxCtas ? rounds : kMaxCtas);
    const int64_t ranges = ranges_of(max_len), top = pairs / (2 * kFewest) + 1, splits = ranges < top ? ranges : top;
    const int64_t cut = pairs > kFewest && splits > 1 ? pairs * splits : 0;
    return static_cast<size_t>(shares > cut ? shares : cut);
  }
};

struct Params {
  AttentionFp4Args a;
  int groups, kept, G, splits;
  float* part_o;     // [parts, kept, D]
  float* part_stat;  // [parts, kept, 4]: m, l, m'
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__global__ void __launch_bounds__(kAThreads, ctas_per_sm(D, NT)) attention_fp4_kernel(const Params p) {
  using ST = AStage<D>;
  constexpr int kRows = NT * kRowTile;
  constexpr int kKSteps = D / 16, kBlocks = D / kFp4Block;
  constexpr int kKWords = D / 32, kVWords = D / 64;  // words of codes that a thread takes of a key, of a value
  constexpr int kOTiles = D / 16;                    // tiles of 16 columns of the outputs
  constexpr int kUnits = 2;                          // units of 16 tokens of a step
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float st_m[kAWarps][kRowTile], st_l[kAWarps][kRowTile], st_n[kAWarps][kRowTile];
  __shared__ int last_s;
  // Where this CTA is; held here because registers are few.
  __shared__ struct {
    uint32_t share, unit, pos, pos_end;  // in rounds of the whole call
    uint32_t at, each, pair_at;          // sequence b's first, a group's number of them, this group's first
    uint32_t cta0;                       // the CTA whose share begins with round 0
    int b, groups, h, grp, nrows, round1, active;
  } now_s;
  const AttentionFp4Args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait_prior_grid();

  // ---- this CTA's share of all rounds
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.c.page;
  struct Sequence {
    int n, len, rounds, groups;  // query rows, tokens; rounds of one of its groups of rows, groups of a key head
    bool bad;
  };
  auto sequence = [&](int b) {
    Sequence s;
    s.n = a.rows != nullptr ? a.rows[b] : a.Q;
    s.len = a.length[b];
    s.bad = s.n < 0 || s.n > a.Q || s.len < 0 || s.len > cap;
    if (s.bad) s.n = a.Q, s.len = 0;  // its rows see nothing
    s.rounds = s.len == 0 ? 1 : (s.len + kChunkTok - 1) / kChunkTok;
    s.groups = (s.n * p.G + kRows - 1) / kRows;
    return s;
  };
  auto set_sequence = [&](int b, const Sequence& s, uint32_t each) {
    now_s.b = b;
    now_s.groups = s.groups;
    now_s.each = each;
    if (s.bad) store_status(a.status, MTP_ERR_ARG);
  };
  int b;
  uint32_t pos, pos_end, at, each;  // (of now_s)
  Sequence seq;
  if (p.splits > 0) {
    const uint32_t sp = blockIdx.x % p.splits, pair = blockIdx.x / p.splits;
    const int row_group = static_cast<int>(pair % p.groups), head = static_cast<int>(pair / p.groups % a.c.heads);
    b = static_cast<int>(pair / p.groups / a.c.heads);
    seq = sequence(b);
    const uint32_t share = (seq.rounds + p.splits - 1u) / p.splits;
    each = (seq.rounds + share - 1) / share * share;
    if (row_group >= seq.groups || sp * share >= each) return;
    pos = (head * seq.groups + row_group) * each + sp * share;
    pos_end = pos + share;
    at = 0;
    if (threadIdx.x == 0) {
      now_s.share = share;
      now_s.pos = pos;
      now_s.pos_end = pos_end;
      now_s.at = at;
      now_s.cta0 = blockIdx.x - pos / share;
      set_sequence(b, seq, each);
    }
  } else {
    if (warp == 0) {
      const int per_lane = (a.B + 31) / 32, b0 = min(lane * per_lane, a.B), b1 = min(b0 + per_lane, a.B);
      Sequence own{};  // the lane's first
      if (b0 < b1) own = sequence(b0);
      uint32_t mine = static_cast<uint32_t>(own.rounds) * own.groups;
      int most = own.rounds;
#pragma unroll 1
      for (int b = b0 + 1; b < b1; ++b) {
        const Sequence s = sequence(b);
        mine += static_cast<uint32_t>(s.rounds) * s.groups;
        most = max(most, s.rounds);
      }
      const uint32_t heads = a.c.heads;
      // no sequence in more than kMaxRanges pieces, the two that are cut off at its ends among them
      const uint32_t share = max((__reduce_add_sync(0xffffffffu, mine) * heads + gridDim.x - 1) / gridDim.x,
                                 (__reduce_max_sync(0xffffffffu, most) + kMaxRanges - 2u) / (kMaxRanges - 1u));
      // whole shares for every group, where that takes no more CTAs
      const uint32_t own_pieces = (own.rounds + share - 1) / share;
      uint32_t pieces = own_pieces * own.groups, unit = 1, own_each = own.rounds;
#pragma unroll 1
      for (int b = b0 + 1; b < b1; ++b) {
        const Sequence s = sequence(b);
        pieces += (s.rounds + share - 1) / share * s.groups;
      }
      if (__reduce_add_sync(0xffffffffu, min(pieces, 4096u)) * heads <= gridDim.x) {
        unit = share;
        own_each = own_pieces * share;
        mine = pieces * share;
      }
      mine *= heads;
      uint32_t upto = mine;
#pragma unroll 1
      for (int k = 1; k < 32; k *= 2) {
        const uint32_t other = __shfl_up_sync(0xffffffffu, upto, k);
        if (lane >= k) upto += other;
      }
      const uint32_t pos = share * blockIdx.x;
      if (lane == 31) {
        now_s.share = share;
        now_s.unit = unit;
        now_s.pos = pos;
        now_s.pos_end = min(pos + share, upto);
        now_s.cta0 = 0;
        now_s.b = -1;  // (no share: it stays so)
      }
      __syncwarp();
      if (upto > pos && upto - mine <= pos) {
        uint32_t at = upto - mine, each = own_each;
        int b = b0;
#pragma unroll 1
        while (pos >= at + each * own.groups * heads && b + 1 < b1) {
          at += each * own.groups * heads;
          own = sequence(++b);
          each = (own.rounds + unit - 1) / unit * unit;
        }
        now_s.at = at;
        set_sequence(b, own, each);
      }
    }
    __syncthreads();
    b = now_s.b;
    if (b < 0) return;  // no share
    pos = now_s.pos, pos_end = now_s.pos_end, at = now_s.at, each = now_s.each;
    seq = sequence(b);
  }

  while (true) {
    const int n = seq.n, len = seq.len;
    const uint32_t pair_b = (pos - at) / each, pair_at = at + pair_b * each;
    const int h = static_cast<int>(pair_b) / seq.groups, grp = static_cast<int>(pair_b) % seq.groups;
    const int r0 = grp * kRows;
    const int nrows = min(n * p.G - r0, kRows);  // rows of this CTA
    const int seen = max(len - n + (r0 + nrows - 1) / p.G + 1, 0);  // tokens that its last row sees
    const int begin = static_cast<int>(pos - pair_at) * kChunkTok;
    const uint32_t round1 = min(each, pos_end - pair_at);
    const int end = min(seen, min(static_cast<int>(round1), seq.rounds) * kChunkTok);

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
    if (threadIdx.x == 0) {
      now_s.pair_at = pair_at;
      now_s.h = h;
      now_s.grp = grp;
      now_s.nrows = nrows;
      now_s.round1 = round1;
      now_s.active = static_cast<int>((pair_at + each - 1) / now_s.share - pair_at / now_s.share) + 1;
    }

    // ---- queries: row g of each tile as an f16 operand
    uint32_t qb[NT][kKSteps][2];
    // From a row's MMA sums to scores in powers of two: f1 times the key's row scale times f2, so that no product
    // leaves the fp32 range on the way. Of this thread's score columns, rows 2 t and 2 t + 1 of a tile.
    uint64_t f1[NT], f2[NT];
    int limit[NT][2];  // tokens that such a row sees
    int least = 0x7FFFFFFF;
    float f_most = 0.0f;
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
      const uint64_t f = f2_mul(f1[nt], f2[nt]);
      f_most = fmaxf(f_most, fmaxf(f2_lo(f), f2_hi(f)));
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
    // Key scales up to which f1 times f2 times the scale stays far from the end of fp32 (sums of products are below 2^27).
    const float k_most = f_most <= 0x1p60f ? 0x1p30f : -1.0f;

    float o[NT][kOTiles][4];
    float m[NT][2], mv[NT][2], l[NT][2];
    uint64_t apart[NT];     // 2^(m - m')
    bool settled = false;  // every row of this thread has maxima, less than 2^40 apart
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
      apart[nt] = 0ull;
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
        float x[kUnits][NT][4], rv[kUnits][2];
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
          const float rk[2] = {kr[t0], kr[t0 + 8]};
          rv[un][0] = vr[t0], rv[un][1] = vr[t0 + 8];
          const bool near = fmaxf(fabsf(rk[0]), fabsf(rk[1])) <= k_most;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint64_t s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s[i] = f2_pack(x[un][nt][2 * i], x[un][nt][2 * i + 1]);
              if constexpr (NT == 1) s[i] = f2_add(s[i], f2_pack(even[2 * i], even[2 * i + 1]));
            }
            if (near) {
              const uint64_t f = f2_mul(f1[nt], f2[nt]);
#pragma unroll
              for (int i = 0; i < 2; ++i) s[i] = f2_mul(s[i], f2_mul(f2_pack(rk[i], rk[i]), f));
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i) s[i] = f2_mul(f2_mul(f2_mul(s[i], f1[nt]), f2_pack(rk[i], rk[i])), f2[nt]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              x[un][nt][2 * i] = f2_lo(s[i]);
              x[un][nt][2 * i + 1] = f2_hi(s[i]);
            }
          }
          if constexpr (edge) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int tok = tok0 + t0 + 8 * i;
              const bool none = tok >= end || ((gone >> un) & 1u) != 0u;
              if (none) rv[un][i] = 1.0f;  // (its stage holds anything)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (none || tok >= limit[nt][c]) x[un][nt][2 * i + c] = kNegInf;
            }
          }
        }

        // ---- weights, transposed: tokens along k
        uint32_t pb[kUnits][NT][2];
        const float r_most = fmaxf(fmaxf(rv[0][0], rv[0][1]), fmaxf(rv[1][0], rv[1][1]));
        const float v_most = lg2(r_most);
        // has a score passed its row's maximum by 2^8, or may it have with its value's scale?
        bool up = !settled || !(r_most <= 0x1p40f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float xm = fmaxf(fmaxf(x[0][nt][c], x[0][nt][2 + c]), fmaxf(x[1][nt][c], x[1][nt][2 + c]));
            up |= xm > m[nt][c] + 8.0f || xm + v_most > mv[nt][c] + 8.0f;
          }
        if (!__any_sync(0xffffffffu, up)) {
          // 2^(x + log2 r - m') as 2^(x - m) times r 2^(m - m'): the latter is below 2^80, so where the former leaves the
          // fp32 range the weight is below what f16 holds
#pragma unroll
          for (int un = 0; un < kUnits; ++un)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint64_t r2 = f2_pack(rv[un][i], rv[un][i]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint64_t e = f2_add(f2_pack(x[un][nt][2 * i], x[un][nt][2 * i + 1]), f2_pack(-m[nt][0], -m[nt][1]));
                const uint64_t w = f2_pack(ex2(f2_lo(e)), ex2(f2_hi(e)));
                const uint64_t sum = f2_add(f2_pack(l[nt][0], l[nt][1]), w);
                l[nt][0] = f2_lo(sum), l[nt][1] = f2_hi(sum);
                const uint64_t u = f2_mul(w, f2_mul(r2, apart[nt]));
                pb[un][nt][i] = transpose8x8(f16x2_bits(f2_lo(u), f2_hi(u)));
              }
            }
        } else {
          float lv[kUnits][2];
#pragma unroll
          for (int un = 0; un < kUnits; ++un)
#pragma unroll
            for (int i = 0; i < 2; ++i) lv[un][i] = lg2(rv[un][i]);
          settled = true;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float nm[2], nv[2], k[2];
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
              for (int s = 4; s < 32; s *= 2) {
                xm = fmaxf(xm, __shfl_xor_sync(0xffffffffu, xm, s));
                ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, s));
              }
              const float to = fmaxf(m[nt][c], xm), to_v = fmaxf(mv[nt][c], ym);
              l[nt][c] *= m[nt][c] == kNegInf ? 0.0f : ex2(m[nt][c] - to);
              const float down = mv[nt][c] == kNegInf ? 0.0f : ex2(mv[nt][c] - to_v);
              m[nt][c] = to;
              mv[nt][c] = to_v;
#pragma unroll
              for (int j = 0; j < kOTiles; ++j) {
                o[nt][j][c] *= down;
                o[nt][j][2 + c] *= down;
              }
              settled &= fabsf(to - to_v) <= 40.0f;  // (not where one of them is infinite)
              k[c] = ex2(to - to_v);
              nm[c] = to == kNegInf ? 0.0f : to;
              nv[c] = to_v == kNegInf ? 0.0f : to_v;
            }
            apart[nt] = f2_pack(k[0], k[1]);
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
    __syncthreads();  // the rings have been read
    const int rows_here = now_s.nrows, active = now_s.active;
    auto store_row = [&](int r, int c, float4 v, float k) {  // four columns of row r, times k
      const int qi = (now_s.grp * kRows + r) / p.G;
      uint16_t* dst = a.out + (static_cast<int64_t>(now_s.b) * a.Q + qi) * a.ld_out +
                      static_cast<int64_t>(now_s.h * p.G + (now_s.grp * kRows + r) % p.G) * D + c;
      uint32_t lo, hi;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(v.y * k), "f"(v.x * k));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(v.w * k), "f"(v.z * k));
      *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    };
    auto store_lse = [&](int r, float mm, float ll) {
      if (a.lse != nullptr)
        a.lse[(static_cast<int64_t>(now_s.b) * a.Q + (now_s.grp * kRows + r) / p.G) * a.q_heads + now_s.h * p.G +
              (now_s.grp * kRows + r) % p.G] =
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
    const int64_t slot = p.splits > 0 ? blockIdx.x : 2 * static_cast<int64_t>(blockIdx.x) + (now_s.pos > now_s.share * blockIdx.x ? 1 : 0);
    float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt * kRowTile >= rows_here) break;
      if (nt > 0) __syncthreads();  // the tile before has been read
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
      const int here = min(rows_here - nt * kRowTile, kRowTile);
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
    // ---- the CTA that comes last joins the ranges, in their order
    bool last = false;
    if (active > 1) {
      __threadfence();
      __syncthreads();
      int* counter = reinterpret_cast<int*>(a.ws) + (static_cast<int64_t>(now_s.b) * a.c.heads + now_s.h) * p.groups + now_s.grp;
      if (threadIdx.x == 0) {
        last_s = atomicAdd(counter, 1) == active - 1;
        if (last_s) *counter = 0;
      }
      __syncthreads();
      last = last_s != 0;
      __threadfence();
    }
    float4* stat = reinterpret_cast<float4*>(smem);  // [active][8]
    // the first range ends its CTA's share, and is that CTA's second unless it begins it too; the others begin theirs
    const uint32_t first_cta = now_s.cta0 + now_s.pair_at / now_s.share;
    const int64_t slot0 = p.splits > 0 ? first_cta : 2 * static_cast<int64_t>(first_cta);
    const bool second = now_s.pair_at % now_s.share != 0u;
    auto slot_of = [&](int s) { return p.splits > 0 ? slot0 + s : slot0 + 2 * s + (s == 0 && second ? 1 : 0); };
    for (int nt = 0; last && nt * kRowTile < rows_here; ++nt) {
      const int here = min(rows_here - nt * kRowTile, kRowTile);
      __syncthreads();
      for (int it = threadIdx.x; it < active * kRowTile; it += kAThreads)
        if (it % kRowTile < here)
          stat[it] = __ldcg(reinterpret_cast<const float4*>(p.part_stat) + slot_of(it / kRowTile) * p.kept + nt * kRowTile + it % kRowTile);
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
          const float4 u = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot_of(s) * p.kept + r) * D + c));
          L += q4.x != kNegInf ? q4.y * ex2(q4.x - M) : q4.y;
          add(v, u, q4.z != kNegInf ? ex2(q4.z - N) : 0.0f);
        }
        store_row(r, c, v, out_factor(M, L, N));
        if (c == 0) store_lse(r, M, L);
      }
    }

    // ---- on to the next group of rows, key head or sequence
    pos = now_s.pair_at + now_s.round1;
    if (pos >= now_s.pos_end) return;
    __syncthreads();  // shared memory has been read
    if (warp == 0) {
      if (lane == 0) now_s.pos = pos;
      const uint32_t after = now_s.at + now_s.each * now_s.groups * a.c.heads;
      if (pos >= after) {
        int next = now_s.b + 1;
        uint32_t found = 0u;
        while (next < a.B) {  // past sequences without rows
          const bool some = next + lane < a.B && sequence(next + lane).n > 0;
          found = __ballot_sync(0xffffffffu, some);
          if (found != 0u) break;
          next += 32;
        }
        __syncwarp();
        if (lane == 0) {
          now_s.at = after;
          if (found != 0u) {
            next += __ffs(found) - 1;
            const Sequence s = sequence(next);
            set_sequence(next, s, (s.rounds + now_s.unit - 1) / now_s.unit * now_s.unit);
          } else {
            now_s.b = -1;
          }
        }
      }
    }
    __syncthreads();
    b = now_s.b;
    if (b < 0) return;  // (there is another with rows: pos_end is not behind the last)
    pos_end = now_s.pos_end, at = now_s.at, each = now_s.each;
    seq = sequence(b);
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
  const int G = q_heads / kv_heads;
  const int64_t pairs = static_cast<int64_t>(B) * kv_heads * Groups(Q, G).groups;
  return counters_bytes(pairs) + Plan::most_parts(pairs, max_len) * rows_kept(Q, G) * (static_cast<size_t>(D) + 4) * 4;
}

cudaError_t launch_attention_fp4(const AttentionFp4Args& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  Params p;
  p.a = a;
  p.G = a.q_heads / a.c.heads;
  const Groups g(a.Q, p.G);
  p.groups = g.groups;
  p.kept = rows_kept(a.Q, p.G);
  const Plan plan(static_cast<int64_t>(a.B) * a.c.heads * g.groups, static_cast<int64_t>(a.max_pages) * a.c.page,
                  ctas_per_sm(a.c.D, g.tiles), di.sm_count);
  p.splits = plan.splits;
  const size_t kept_rows = plan.parts() * p.kept;
  p.part_o = reinterpret_cast<float*>(a.ws + (a.ws_bytes / 16 * 16 - kept_rows * (a.c.D + 4) * 4));
  p.part_stat = p.part_o + kept_rows * a.c.D;
  void* args[] = {&p};
  return launch_pdl(a.c.D == 64 ? kernel_of<64>(g.tiles) : kernel_of<128>(g.tiles), dim3(static_cast<unsigned>(plan.ctas)),
                    dim3(kAThreads), a.c.D == 64 ? AStage<64>::kSmem : AStage<128>::kSmem, stream, args);
}

}  // namespace mtp
