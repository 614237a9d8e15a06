// Causal attention over packed prompts, BF16, grouped heads:
//   o_i = sum_{j <= i} p_ij v_j,   p_ij = softmax_j( scale q_i . k_j )    within each sequence
//
// A piece of work is 256 query rows of one head of one sequence, as two tiles of 128, over the
// sequence's keys and values in tiles of 128 that both share. The products run on the fifth-generation
// tensor cores: S = Q K^T into tensor memory, one warpgroup per tile turns a row of S per thread into
// weights (running maximum and sum in registers) and writes them back over S as BF16, and O += P V
// takes them from there. While one tile is in its softmax the tensor cores work on the other's
// products. The running maximum moves only when a score passes it by 2^8 (weights up to 256 cost
// nothing in BF16 or fp32), so the sums in tensor memory are rescaled a few times a row at most.
//
// The grid has a CTA for every piece, longest pieces of a sequence first, but a CTA that runs takes over the pieces of
// CTAs that have not started (cluster launch control): the next piece's Q, K and V are on their way and its
// first product runs while the tiles of the piece before are divided and stored.
//
// Warp roles: 0..3 and 4..7 softmax and epilogue of tile 0 and 1 (warp w reads TMEM lanes
// 32 (w % 4) ..), 8 copies (2-D TMA, 128-byte swizzle), 9 tensor-memory allocation and MMA issue, 10 the next pieces, 11
// only fills its warpgroup.
// Every wait is bounded, as in context.cu. A warp decides alone when it gives up, so between the start and the end of
// the kernel nothing but these bounded waits joins several warps: no barrier of a warpgroup, which has no limit.
//
// Measured at 48 query heads over 8 key heads, D = 128: 8 packed prompts of 16384 rows in all (0.52 TFLOP) 487 us, one prompt of
// 16384 (3.3 TFLOP) 2.2 ms, 1.5 PFLOP/s; without the softmax, so as products and copies alone, they take 422 us and 1.9 ms. The
// exponentials of a tile (eight a clock in a quarter of an SM) and its products run one under the other, with what both
// wait for at a tile's ends on top. Slower: four softmax warpgroups, two threads a row (508 us, 2.33 ms), a second warp that
// issues MMAs (509, 2.58), the next piece's first scores ahead of the last step (517 and up), a ring of 5 stages (492), 224
// registers for the softmax (499), sleeping between polls (490).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "codes.cuh"
#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "layer.h"
#include "tc.cuh"

namespace mtp {

namespace {

constexpr int kPThreads = 384;
// Registers: the launch gives a thread 168; the warps that copy and issue keep 56 of them, the two softmax
// warpgroups (a row of 128 scores a thread) take 216: 2 x 216 + 56 <= 3 x 168.
constexpr int kRegsOthers = 56, kRegsSoftmax = 216;
constexpr int kTile = 128;                 // query rows of a tile, keys of a step
constexpr uint32_t kPTmemCols = 512;

template <int D>
struct PTile {
  static constexpr int kBytes = kTile * D * 2;             // a tile of Q, K or V: D / 64 boxes of 128 rows x 128 bytes
  static constexpr int kStages = 4;                        // K, V, K, V ..
  static constexpr int kBars = 2 * kStages + 18;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(2 + kStages) * kBytes + kBars * 8 + 96;
  static constexpr uint32_t kOCol = 256;                   // O of tile i at kOCol + i D, S (and P) at 128 i
};

struct PromptParams {
  const uint16_t* v;
  int64_t ld_v;
  const int32_t* row_start;
  uint16_t* out;
  float* lse;
  int32_t* status;
  int64_t ld_out;
  int T, B, q_heads, G, D;
  float c;  // scale * log2(e)
  unsigned long long wait_ns;  // give-up time of the waits, but for those for the kernel's own copies and products at its end
};

// ------------------------------------------------------------------------------- PTX
// Descriptor of an operand whose rows of 128 bytes run along its M or N side (128-byte swizzle, groups of
// eight rows 1024 bytes apart along K, pieces of 64 elements `lead` bytes apart).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr, uint32_t lead) {
  uint64_t d = static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// D (TMEM) += A (TMEM, 128 x 16 BF16, two a column) * B (16 x N, shared memory).
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 columns of this thread's lane; the values are there after tmem_arrived.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// (what follows may not be moved in front of the wait that precedes this)
__device__ __forceinline__ void tmem_arrived(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// All ones in the halves of a BF16 pair that are infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite(uint32_t pair) { return __vcmpeq2(pair & 0x7F807F80u, 0x7F807F80u); }

// Which rows piece `item` of a whole warp's question is: the sequences' pairs of tiles in order, a sequence's last (and
// longest) first, each for every head. x: first row of the sequence, y: its rows (0: no such piece), z: pair, w: head.
__device__ __forceinline__ int4 find_work(const PromptParams& p, int piece) {
  const int lane = threadIdx.x & 31;
  int item = piece / p.q_heads;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int s0 = 0, n = 0;
    if (b < p.B) {
      s0 = p.row_start[b];
      const int s1 = p.row_start[b + 1];
      n = s1 - s0;
      if (s0 < 0 || s1 < s0 || s1 > p.T) {
        store_status(p.status, MTP_ERR_ARG);
        n = 0;
      }
    }
    const int mine = (n + 2 * kTile - 1) / (2 * kTile);
    int upto = mine;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += v;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, item < upto && item >= upto - mine);
    if (here != 0u) {
      const int from = __ffs(here) - 1;
      return make_int4(__shfl_sync(0xffffffffu, s0, from), __shfl_sync(0xffffffffu, n, from),
                       __shfl_sync(0xffffffffu, upto, from) - 1 - item, piece % p.q_heads);
    }
    item -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return make_int4(0, 0, 0, 0);
}

// ------------------------------------------------------------------------------- kernel
template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const PromptParams p) {
  using TL = PTile<D>;
  constexpr int kStages = TL::kStages, kHalves = D / 64, kBox = kTile * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_s = smem_addr(smem), ring = q_s + 2 * TL::kBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(2 + kStages) * TL::kBytes);
  uint64_t* empty = full + kStages;
  uint64_t* q_full = empty + kStages;  // [2]
  uint64_t* q_empty = q_full + 2;      // [2]
  uint64_t* s_full = q_empty + 2;      // [2]: a tile's S, and the sums of the step before, are in tensor memory
  uint64_t* p_full = s_full + 2;       // [2][2]: the first and the second half of its weights are
  uint64_t* o_full = p_full + 4;       // [2]: its last sums are
  uint64_t* work_full = o_full + 2;    // [2]
  uint64_t* work_empty = work_full + 2;  // [2]
  uint64_t* asked = work_empty + 2;    // the answer about the next piece is there
  uint64_t* done = asked + 1;          // the MMAs that were issued have ended
  int4* answer = reinterpret_cast<int4*>(full + TL::kBars);
  int4* work = answer + 1;             // [2]: first row of the sequence, its rows (0: no more work), pair of tiles, head
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(work + 2);
  // [4][2]: the piece (count + 1) in which a tile's own values last held infinities or NaN. A piece has the pair count & 3:
  // no warp takes piece c + 4 before every warp has taken c + 2, and so has read the pair for c.
  int* unusual = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&full[i]), 1);
      mbar_init(smem_addr(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&q_full[i]), 1);
      mbar_init(smem_addr(&q_empty[i]), 1);
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&p_full[i]), kTile);
      mbar_init(smem_addr(&p_full[2 + i]), kTile);
      mbar_init(smem_addr(&o_full[i]), 2);  // the products, and the warp that has seen all weights come
      mbar_init(smem_addr(&work_full[i]), 1);
      mbar_init(smem_addr(&work_empty[i]), 10);  // the warps that work
    }
    for (int i = 0; i < 8; ++i) unusual[i] = 0;
    mbar_init(smem_addr(asked), 1);
    mbar_init(smem_addr(done), 1);
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_slot), kPTmemCols);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_prior_grid();
  auto give_up = [&] { store_status(p.status, MTP_ERR_TIMEOUT); };
  // A warp's bounded wait. Where the limit is 0 no role begins, so that a wait that finds its data is one poll (with a look at
  // the limit in front of each, 8 prompts took 518 instead of 485 us).
  const bool begin = p.wait_ns != 0;
  auto come = [&](uint32_t bar, uint32_t parity) {
    bool there = mbar_try_wait(bar, parity);
    if (!there) {
      const unsigned long long t0 = global_timer_ns();
      do {
        there = mbar_try_wait(bar, parity);
      } while (!there && global_timer_ns() - t0 <= p.wait_ns);
    }
    return __all_sync(0xffffffffu, there) != 0;
  };
  // The next piece: a warp's own count of them, and whether all went well.
  struct Piece {
    int s0, n, pair, h;
    int steps0, steps1;  // of each tile: up to and with the keys of its own rows
    __device__ __forceinline__ int steps() const { return steps1 > steps0 ? steps1 : steps0; }
  };
  auto next_piece = [&](int count, bool& ok) {
    const int i = count & 1;
    ok = come(smem_addr(&work_full[i]), static_cast<uint32_t>((count >> 1) & 1));
    Piece w{0, 0, 0, 0, 0, 0};
    if (!ok) return w;
    const int4 v = *const_cast<const int4*>(&work[i]);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&work_empty[i]));
    w.s0 = v.x, w.n = v.y, w.pair = v.z, w.h = v.w;
    w.steps0 = 2 * w.pair + 1;
    w.steps1 = (2 * w.pair + 1) * kTile < w.n ? 2 * w.pair + 2 : 0;
    return w;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
    if (warp == 10) {
      // ---------------------------------------------------------------- pieces of work
      int item = static_cast<int>(blockIdx.x), count = 0;
      uint32_t turn = 0;
      bool ok = begin, more = true;
      while (ok) {
        int4 w = make_int4(0, 0, 0, 0);
        if (more) w = find_work(p, item);
        if (more && w.y == 0) more = false;  // (pieces in front of the last sequence's end all exist)
        const int i = count & 1;
        ok = come(smem_addr(&work_empty[i]), static_cast<uint32_t>(((count >> 1) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          work[i] = w;
          mbar_arrive(smem_addr(&work_full[i]));
        }
        __syncwarp();
        ++count;
        if (!more) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(smem_addr(asked), 16);
          asm volatile(
              "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                  smem_addr(answer)),
              "r"(smem_addr(asked))
              : "memory");
        }
        __syncwarp();
        ok = come(smem_addr(asked), turn);
        if (!ok) {
          (void)mbar_wait_bounded(smem_addr(asked), turn);  // the answer lands before the shared memory goes away
          break;
        }
        turn ^= 1u;
        uint32_t got, x;
        asm volatile(
            "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\tld.shared.b128 a, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
            : "=r"(got), "=r"(x)
            : "r"(smem_addr(answer))
            : "memory");
        fence_proxy_async_smem();  // (the next answer is written over this one)
        __syncwarp();
        more = got != 0;
        item = static_cast<int>(x);
      }
      if (!ok && lane == 0) give_up();
    } else if (warp == 8) {
      // ---------------------------------------------------------------- copies
      const bool lead = elect_one();
      uint64_t pol;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
      auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
        mbar_arrive_expect_tx(bar, TL::kBytes);
#pragma unroll
        for (int i = 0; i < kHalves; ++i) tma_load_2d(dst + i * kBox, map, x + 64 * i, y, bar, pol);
      };
      int used = 0, q_used[2] = {0, 0};
      bool ok = begin;
      auto next = [&](const CUtensorMap* map, int x, int y) {
        if (!ok) return;
        const int s = used % kStages;
        ok = come(smem_addr(&empty[s]), static_cast<uint32_t>(((used / kStages) & 1) ^ 1));
        if (!ok) return;
        if (lead) load(ring + s * TL::kBytes, map, x, y, smem_addr(&full[s]));
        ++used;
      };
      auto next_q = [&](int tile, int x, int y) {
        if (!ok) return;
        ok = come(smem_addr(&q_empty[tile]), static_cast<uint32_t>((q_used[tile] & 1) ^ 1));
        if (!ok) return;
        if (lead) load(q_s + tile * TL::kBytes, &tm_q, x, y, smem_addr(&q_full[tile]));
        ++q_used[tile];
      };
      for (int count = 0; ok; ++count) {
        const Piece w = next_piece(count, ok);
        if (!ok || w.n == 0) break;
        const int hk = w.h / p.G;
        next_q(0, w.h * D, w.s0 + 2 * w.pair * kTile);
        next(&tm_k, hk * D, w.s0);
        if (w.steps1 > 0) next_q(1, w.h * D, w.s0 + (2 * w.pair + 1) * kTile);
        next(&tm_v, hk * D, w.s0);
        for (int j = 1; j < w.steps() && ok; ++j) {
          next(&tm_k, hk * D, w.s0 + j * kTile);
          next(&tm_v, hk * D, w.s0 + j * kTile);
        }
      }
      if (!ok && lane == 0) give_up();
      // the last copies land before the shared memory goes away
      for (int i = used > kStages ? used - kStages : 0; i < used; ++i)
        (void)mbar_wait_bounded(smem_addr(&full[i % kStages]), static_cast<uint32_t>((i / kStages) & 1));
      for (int i = 0; i < 2; ++i)
        if (q_used[i] > 0) (void)mbar_wait_bounded(smem_addr(&q_full[i]), static_cast<uint32_t>((q_used[i] - 1) & 1));
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMA issue
      constexpr uint32_t idesc_s = umma_idesc_bf16(kTile, kTile);
      constexpr uint32_t idesc_o = umma_idesc_bf16(kTile, D) | (1u << 16);  // V's rows run along N
      const bool lead = elect_one();
      bool ok = begin;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok) ok = come(smem_addr(bar), static_cast<uint32_t>(phase & 1));
        tmem_fence_after_sync();
      };
      // item i of the ring: K of a step, or V
      auto scores = [&](int tile, int i) {
        if (lead) {
          const uint64_t dq = umma_desc_sw128(q_s + tile * TL::kBytes), dk = umma_desc_sw128(ring + (i % kStages) * TL::kBytes);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = (k / 4) * (kBox >> 4) + (k % 4) * 2;
            umma_bf16(tmem + 128 * tile, dq + at, dk + at, idesc_s, k != 0 ? 1u : 0u);
          }
        }
        __syncwarp();
      };
      auto outputs = [&](int tile, int i, int half, bool first) {
        if (lead) {
          const uint64_t dv = umma_desc_mn_sw128(ring + (i % kStages) * TL::kBytes, kBox);
#pragma unroll
          for (int k = half * (kTile / 32); k < (half + 1) * (kTile / 32); ++k)
            umma_bf16_ts(tmem + TL::kOCol + tile * D, tmem + 128 * tile + 8 * k, dv + k * (2048 >> 4), idesc_o,
                         first && k == 0 ? 0u : 1u);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (lead) umma_commit(smem_addr(bar));
        __syncwarp();
      };
      int base = 0, q_seen[2] = {0, 0}, p_seen[2] = {0, 0};
      for (int count = 0; ok; ++count) {
        const Piece w = next_piece(count, ok);
        if (!ok || w.n == 0) break;
        const int of[2] = {w.steps0, w.steps1}, steps = w.steps();
        // (S of this piece goes over the weights that the last products of the piece before have read: in order)
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          if (of[tile] == 0) continue;
          wait(&q_full[tile], q_seen[tile]++);
          wait(&full[base % kStages], base / kStages);
          if (!ok) break;
          scores(tile, base);
          commit(&s_full[tile]);
          if (of[tile] == 1) commit(&q_empty[tile]);
        }
        if (!ok) break;
        commit(&empty[base % kStages]);
        for (int j = 0; j < steps && ok; ++j) {
          const int iv = base + 2 * j + 1, ik = iv + 1;
#pragma unroll
          for (int tile = 0; tile < 2; ++tile) {
            if (j >= of[tile] || !ok) continue;
            wait(&full[iv % kStages], iv / kStages);
            wait(&p_full[tile], p_seen[tile]);
            if (!ok) break;
            outputs(tile, iv, 0, j == 0);
            wait(&p_full[2 + tile], p_seen[tile]++);
            if (!ok) break;
            outputs(tile, iv, 1, false);
            if (j + 1 < of[tile]) {
              wait(&full[ik % kStages], ik / kStages);
              if (!ok) break;
              scores(tile, ik);
              commit(&s_full[tile]);
              if (j + 2 == of[tile]) commit(&q_empty[tile]);
            } else {
              commit(&o_full[tile]);
              if (lead) mbar_arrive(smem_addr(&o_full[tile]));  // (with it the marks that came with the weights are seen)
              __syncwarp();
            }
          }
          if (!ok) break;
          commit(&empty[iv % kStages]);
          if (j + 1 < steps) commit(&empty[ik % kStages]);
        }
        base += 2 * steps;
      }
      if (!ok && lane == 0) give_up();
      commit(done);
      (void)mbar_wait_bounded(smem_addr(done), 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------------ softmax and epilogue
    const int tile = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + 128 * tile, o_t = tmem + lanes + TL::kOCol + tile * D;
    const uint64_t c2 = f2_pack(p.c, p.c);
    int base = 0, s_seen = 0, o_seen = 0;
    bool ok = begin;
    for (int count = 0; ok; ++count) {
      const Piece w = next_piece(count, ok);
      if (!ok || w.n == 0) break;
      const int my_steps = tile == 0 ? w.steps0 : w.steps1;
      const int i0 = (2 * w.pair + tile) * kTile;  // first row of the tile in its sequence
      float m = -INFINITY, l = 0.0f;               // m in powers of two
      for (int j = 0; j < my_steps; ++j) {
        ok = come(smem_addr(&s_full[tile]), static_cast<uint32_t>(s_seen++ & 1));
        if (!ok) break;
        tmem_fence_after_sync();
        uint32_t s[kTile];
#pragma unroll
        for (int k = 0; k < kTile; k += 32) tmem_ld32_async(s_t + k, s + k);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < kTile; k += 32) tmem_arrived(s + k);
        // Blocks of 32 keys of the tile's own step that no row of the warp sees cost nothing but their zeros.
        const bool own = j == my_steps - 1;
        const int blocks = own ? (warp & 3) + 1 : 4;
        if (own) {
          // the tile's own keys: those behind the row's are not seen
#pragma unroll
          for (int k = 0; k < kTile; k += 32)
            if (k / 32 == (warp & 3)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e > (row & 31)) s[k + e] = 0xFF800000u;
            }
          // A zero weight must not carry an infinity or a NaN of a row that is not seen into the sums: rows of V
          // behind the sequence become zeros here, and so do such elements of the tile's own rows. The epilogue gives
          // them back to the rows that see them: those of this tile, and of tile 1, whose products read tile 0's rows after this.
          const int left = w.n - i0, iv = base + 2 * j + 1;
          ok = come(smem_addr(&full[iv % kStages]), static_cast<uint32_t>((iv / kStages) & 1));
          if (!ok) break;
          uint4* v = reinterpret_cast<uint4*>(smem + (2 + iv % kStages) * TL::kBytes);
          uint32_t top = 0u;
#pragma unroll
          for (int i = 0; i < 8 * kHalves; ++i) top = mag_max(top, v[row + i * kTile]);
          if (max(top & 0xFFFFu, top >> 16) >= 0x7F80u || left < kTile) {
            for (int x = row; x < kTile * 8 * kHalves; x += kTile) {
              const uint4 u = v[x];
              const uint32_t inf = nonfinite(u.x) | nonfinite(u.y) | nonfinite(u.z) | nonfinite(u.w);
              if (((x >> 3) & (kTile - 1)) >= left) {
                v[x] = make_uint4(0u, 0u, 0u, 0u);
              } else if (inf != 0u) {
                v[x] = make_uint4(u.x & ~nonfinite(u.x), u.y & ~nonfinite(u.y), u.z & ~nonfinite(u.z), u.w & ~nonfinite(u.w));
                unusual[2 * (count & 3) + tile] = count + 1;
              }
            }
            fence_proxy_async_smem();
          }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < kTile; k += 32)
          if (k / 32 < blocks) {
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(s[k + e]));
          }
        mx *= p.c;
        if (__any_sync(0xffffffffu, mx > m + 8.0f)) {
          const float to = fmaxf(m, mx);
          const float f = m == -INFINITY ? 0.0f : ex2(m - to);
          m = to;
          l *= f;
          if (j > 0) {
#pragma unroll
            for (int k = 0; k < D; k += 32) {
              uint32_t o[32];
              tmem_ld32_async(o_t + k, o);
              tmem_wait_ld();
              tmem_arrived(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_t + k, o);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.0f : m;
        const uint64_t nm = f2_pack(-ms, -ms);
        uint64_t sum = 0ull;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // (the first half's products start under the second's exponentials)
          uint32_t pw[32];
#pragma unroll
          for (int k = 0; k < 32; k += 16)
            if (half * 2 + k / 16 < blocks) {
#pragma unroll
              for (int e = k; e < k + 16; ++e) {
                const int at = half * 64 + 2 * e;
                const uint64_t y = f2_fma(f2_pack(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), c2, nm);
                const float a = ex2(f2_lo(y)), b = ex2(f2_hi(y));
                sum = f2_add(sum, f2_pack(a, b));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pw[e]) : "f"(b), "f"(a));
              }
            } else {
#pragma unroll
              for (int e = k; e < k + 16; ++e) pw[e] = 0u;
            }
          tmem_st32(s_t + 32 * half, pw);
          tmem_wait_st();
          tmem_fence_before_sync();
          mbar_arrive(smem_addr(&p_full[2 * half + tile]));
        }
        l += f2_lo(sum) + f2_hi(sum);
      }
      base += 2 * w.steps();
      if (!ok || my_steps == 0) continue;
      ok = come(smem_addr(&o_full[tile]), static_cast<uint32_t>(o_seen++ & 1));
      if (!ok) break;
      tmem_fence_after_sync();
      const bool in = i0 + row < w.n;
      const int64_t r = static_cast<int64_t>(w.s0) + i0 + row;
      const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      uint16_t* dst = p.out + r * p.ld_out + w.h * D;
      const volatile int* marks = unusual + 2 * (count & 3);
      // places in the tile of the rows whose elements were taken out and that this row sees
      const int add0 = tile == 1 && marks[0] == count + 1 ? -kTile : 0, add1 = marks[tile] == count + 1 ? row + 1 : 0;
#pragma unroll
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        __syncwarp();  // (its rows went through loops of their own lengths)
        tmem_ld32_async(o_t + k, o);
        tmem_wait_ld();
        tmem_arrived(o);
        if (in) {
          for (int x = add0; x < add1; ++x) {
            const uint16_t* v = p.v + (static_cast<int64_t>(w.s0) + i0 + x) * p.ld_v + w.h / p.G * D + k;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t u = v[e];
              if ((u & 0x7F80u) == 0x7F80u) o[e] = __float_as_uint(__uint_as_float(o[e]) + bf16_bits_to_f32(u));
            }
          }
        }
        if (in) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(x[y])
                  : "f"(__uint_as_float(o[e + 2 * y + 1]) * f), "f"(__uint_as_float(o[e + 2 * y]) * f));
            *reinterpret_cast<uint4*>(dst + k + e) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      if (in && p.lse != nullptr)
        p.lse[r * p.q_heads + w.h] = l > 0.0f || l != l ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
    }
    if (!ok && lane == 0) give_up();
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tmem_fence_after_sync();
    tmem_dealloc(tmem, kPTmemCols);
  }
}

bool encode_rows(TmapEncodeFn enc, CUtensorMap* map, const uint16_t* p, int64_t ld, int T, int columns) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, kTile}, step[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_attention_prompt(const AttentionPromptArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const TmapEncodeFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  CUtensorMap tq, tk, tv;
  if (!encode_rows(enc, &tq, a.q, a.ld_q, a.T, a.q_heads * a.D) || !encode_rows(enc, &tk, a.k, a.ld_k, a.T, a.kv_heads * a.D) ||
      !encode_rows(enc, &tv, a.v, a.ld_v, a.T, a.kv_heads * a.D))
    return cudaErrorInvalidValue;
  PromptParams p{a.v, a.ld_v, a.row_start, a.out, a.lse, a.status, a.ld_out, a.T, a.B, a.q_heads, a.q_heads / a.kv_heads, a.D,
                 a.scale * 1.44269504088896341f, stage_wait_ns()};
  // pairs of tiles: a sequence of n rows has at most n / 256 + 1
  const int64_t items = a.T / (2 * kTile) + a.B;
  void* args[] = {&tq, &tk, &tv, &p};
  if (a.D == 64)
    return launch_pdl(reinterpret_cast<const void*>(attention_prompt_kernel<64>), dim3(static_cast<unsigned>(items * a.q_heads)),
                      dim3(kPThreads), PTile<64>::kSmem, stream, args);
  return launch_pdl(reinterpret_cast<const void*>(attention_prompt_kernel<128>), dim3(static_cast<unsigned>(items * a.q_heads)),
                    dim3(kPThreads), PTile<128>::kSmem, stream, args);
}

}  // namespace mtp
