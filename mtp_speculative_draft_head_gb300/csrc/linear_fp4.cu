// Rows of activations times an FP4 weight matrix, both in four bits:
//   y[r, n] = bf16( rs_x[r] rs_w[n] sum_k (s_x code_x)[r, k] (s_w code_w)[n, k] )
//
// Kernels:
//  1. the rows of x are quantised (fp4_quantize.cu) into the workspace, their block scales already
//     in the order in which tensor memory wants them;
//  2. linear_fp4_kernel: the product on the fifth-generation tensor cores with the block scales
//     applied by the MMA itself (tcgen05.mma kind::mxf4nvf4, one E4M3 scale per 16 codes of either
//     operand, fp32 accumulation); the row scales multiply in the epilogue.
//
// The weights are the MMA's M operand (128 rows a tile) and the activation rows its N operand (16 to
// 224 a tile): one row of activations costs an eighth of a 128-row tile instead of filling one, so
// the same kernel serves a draft step's few sequences, bound by the read of the weights, and a
// prompt's thousands of rows, bound by its operands' way into the SMs. Codes arrive by 2-D TMA (256 codes = 128
// bytes a row and stage, 128-byte swizzle). The weights' scales are rows of 16 bytes a stage in the
// copy's plain layout; one warp loads them and stores the four words of a row into the four
// 32 x 16-byte blocks that tcgen05.cp spreads over tensor memory (the scales of rows r, r + 32,
// r + 64, r + 96 side by side). The activations' scales are written in that order by the quantiser
// and come by one bulk copy a stage.
//
// Schedules. Many rows: a persistent grid, one CTA per SM, two accumulators in tensor memory, so a
// tile's epilogue runs under the next tile's MMAs. Few rows (less than a wave of tiles): the k range
// is split over a cluster of 2 to 8 CTAs, whose fp32 partial sums meet in the first CTA's shared
// memory and are added in k order.
//
// Measured, 12288 -> 6144, with the rows' quantisation: 16 rows 18.0 us with the weights in L2, 20.0 out of HBM (42.5
// MB, 6.4 us at the copy rate: latencies of a short kernel, the quantiser before it and the cluster's join are the
// rest); 4096 rows 141 us, 26 of them the quantiser's. There the operands' way into the SMs bounds it: 745 cycles for a
// stage's 51 KB (69 bytes a cycle and SM, the four stages that shared memory holds all in flight); its MMAs take 318
// at the nominal rate, and their pipe counts as active for 58 % of the time, 430.
//
// Warp roles: 0 weight codes, 1 tensor-memory allocation and MMA issue, 2 weight scales, 3
// activation codes and scales, 4..7 epilogue (warp w reads
// TMEM lanes 32 (w % 4) ..). Every wait is bounded, as in context.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "linear_fp4_sched.h"
#include "tc.cuh"

namespace mtp {

namespace {

constexpr int kLThreads = 256;
constexpr int kABytes = kLM * kLK / 2;       // 16 KB of weight codes per stage
constexpr int kSfChunk = 4 * 512;            // scales of 128 rows x 256 codes: four 512-byte blocks
constexpr uint32_t kTmemCols = 512;

template <int NT>
struct LTile {
  static constexpr int kChunks = (NT + 127) / 128;             // 128-row scale blocks of the activations
  static constexpr int kBBytes = NT * kLK / 2;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfChunk * (1 + kChunks);
  static constexpr int kSfBytes = 4 * kLM * 16, kSfBufs = 2;   // a fetch of the weights' scales: four stages of them
  static constexpr int kFit = (227 * 1024 - 1024 - 512 - 16 * NT - kSfBufs * kSfBytes) / kStageBytes;
  static constexpr int kStages = kFit < 9 ? kFit : 9;
  // after the two accumulators; an MMA takes the scales from an address that is a multiple of four columns
  static constexpr uint32_t kSfaCol = 2 * NT;
  static constexpr uint32_t kSfbCol = kSfaCol + 16;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + (2 * kStages + 4) * 8 + 16 +
                                  4 * NT * 4 + kSfBufs * kSfBytes;
  static_assert(NT % 16 == 0 && NT <= 256, "N of an M = 128 MMA");
  static_assert(kSfbCol + 16 * kChunks <= kTmemCols, "tensor memory");
};

struct LinearParams {
  const uint8_t* w_bs;   // [N, kp / 16]
  const float* w_rs;     // [N]
  const uint8_t* x_sf;   // workspace: scales in operand order (fp4.h)
  const float* x_rs;     // workspace: [R]
  uint16_t* y;           // [R, N]
  int32_t* status;
  int R, N, kp;
};

// ------------------------------------------------------------------------------- PTX
// Instruction descriptor, kind::mxf4nvf4: E2M1 A and B, both K-major, E4M3 scales, M x N, K = 64.
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Descriptor of 32 rows of 16 bytes (512 contiguous bytes of shared memory): no swizzle, groups of
// eight 16-byte rows 128 bytes apart, descriptor version 1.
__device__ __forceinline__ uint64_t sf_desc(uint32_t smem) {
  return static_cast<uint64_t>((smem & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46);
}
// Those rows to four TMEM columns, repeated in all four 32-lane quarters.
__device__ __forceinline__ void tmem_copy_sf(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// A position in the ring of stages: slot and the parity of its current round.
template <int STAGES>
struct Ring {
  uint32_t s = 0, ph = 0, used = 0;
  __device__ __forceinline__ void next() {
    ++used;
    if (++s == STAGES) {
      s = 0;
      ph ^= 1u;
    }
  }
};
// The copies of a producer's last stages land before the CTA's shared memory goes away (normally the
// MMA warp has seen them all; after a timeout another role's arrival may be missing, and the waits
// end by their limit).
template <int STAGES>
__device__ __forceinline__ void drain(Ring<STAGES> r, uint64_t* full) {
  for (uint32_t i = 0; i < STAGES && i < r.used; ++i) {
    if (r.s == 0) {
      r.s = STAGES;
      r.ph ^= 1u;
    }
    --r.s;
    (void)mbar_wait_bounded(smem_addr(&full[r.s]), r.ph);
  }
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------------------- kernel
template <int NT, bool SPLIT, bool GROUP>
__global__ void __launch_bounds__(kLThreads, 1)
    linear_fp4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const LinearParams p, const LinearSched c) {
  using TL = LTile<NT>;
  constexpr int kStages = TL::kStages, kChunks = TL::kChunks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * TL::kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  float* rx_all = reinterpret_cast<float*>(tmem_slot + 4);  // [4][NT]
  uint8_t* sf_raw = reinterpret_cast<uint8_t*>(rx_all + 4 * NT);  // 16-byte aligned: all before it comes in such pieces
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's tiles t0, t0 + step, ... and its stages kb0 .. kb0 + nkb of each
  const uint32_t rank = SPLIT ? cta_rank() : 0u;
  const int t0 = SPLIT ? static_cast<int>(blockIdx.x) / c.splits : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? c.tiles : static_cast<int>(gridDim.x);
  // Tile t: every weight tile in turn for each activation tile, or (GROUP) for each kGroup activation tiles.
  auto weight_tile = [&](int t) {
    if constexpr (!GROUP) return t % c.mt;
    const int g = t / (c.mt * kGroup), left = c.tiles / c.mt - g * kGroup;
    return (t - g * c.mt * kGroup) / (left < kGroup ? left : kGroup);
  };
  auto x_tile = [&](int t) {
    if constexpr (!GROUP) return t / c.mt;
    const int g = t / (c.mt * kGroup), left = c.tiles / c.mt - g * kGroup;
    return g * kGroup + (t - g * c.mt * kGroup) % (left < kGroup ? left : kGroup);
  };
  auto tile_row = [&](int t) { return weight_tile(t) * kLM; };  // first weight row of tile t
  const int kb0 = SPLIT ? static_cast<int>(rank) * c.nkb / c.splits : 0;
  const int nkb = (SPLIT ? (static_cast<int>(rank) + 1) * c.nkb / c.splits : c.nkb) - kb0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&full[i]), 3);  // the two producers and the scale warp
      mbar_init(smem_addr(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&acc_full[i]), 1);
      mbar_init(smem_addr(&acc_empty[i]), 4);
    }
    abort_flag = 0;
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
  }
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), kTmemCols);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  auto aborted = [&] { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  auto give_up = [&] {
    store_status(p.status, MTP_ERR_TIMEOUT);
    atomicExch(&abort_flag, 1);
  };

  // The row scales of a tile's activation rows, per epilogue warp in shared memory (loaded before the
  // accumulator is waited for: read one by one between the stores, each cost an L2 round trip, 44 us a
  // tile).
  auto load_rx = [&](float* rx, int r0) {
    for (int j = lane; j < NT; j += 32) rx[j] = r0 + j < p.R ? __ldcg(p.x_rs + r0 + j) : 0.0f;
    __syncwarp();
  };
  // Sixteen columns of y from this lane's accumulator row: neighbouring lanes swap halves, so that an
  // even lane holds its own and the next weight row for one activation row, an odd lane for the next
  // one, and a warp stores 2 x 64 bytes at a time (N odd: 2-byte stores).
  auto store16 = [&](int r0, int c0, int row, const float (&v)[16], float rw, const float* rx) {
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 s = reinterpret_cast<const float2*>(rx + c0)[e];
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
          : "=r"(o[e])
          : "f"(__fmul_rn(__fmul_rn(v[2 * e + 1], rw), s.y)), "f"(__fmul_rn(__fmul_rn(v[2 * e], rw), s.x)));
    }
    if ((p.N & 1) == 0) {
      const int odd = lane & 1;
      uint16_t* dst = p.y + static_cast<size_t>(r0 + c0 + odd) * p.N + (row - odd);
      const bool in = row < p.N;  // N is even: the pair is inside or outside as a whole
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = __shfl_xor_sync(0xffffffffu, o[e], 1);
        const uint32_t d = odd ? __byte_perm(w, o[e], 0x7632) : __byte_perm(o[e], w, 0x5410);
        if (in && r0 + c0 + 2 * e + odd < p.R) *reinterpret_cast<uint32_t*>(dst + static_cast<size_t>(2 * e) * p.N) = d;
      }
    } else if (row < p.N) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (r0 + c0 + e < p.R)
          p.y[static_cast<size_t>(r0 + c0 + e) * p.N + row] = static_cast<uint16_t>(o[e >> 1] >> (16 * (e & 1)));
    }
  };

  // The roles below run as whole warps on warp-uniform values, with one elected lane issuing: a copy or
  // an MMA issued from a single-lane branch pays for moving each operand to the uniform registers,
  // ~300 cycles a stage in each role (about 1,100 cycles a stage in all against 320 of MMAs).
  if (warp == 0) {
    // ------------------------------------------------------------------ weight codes
    // They do not depend on the kernel before (the quantiser): the ring fills while it runs.
    const bool lead = elect_one();
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    Ring<kStages> r;
    bool ok = true;
    for (int t = t0; t < c.tiles && ok; t += step) {
      const int row = tile_row(t);
      for (int kb = kb0; kb < kb0 + nkb; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&empty[r.s]), r.ph ^ 1u));
        if (!ok) break;
        if (lead) {
          const uint32_t bar = smem_addr(&full[r.s]);
          mbar_arrive_expect_tx(bar, kABytes);
          tma_load_2d(smem_addr(smem) + r.s * TL::kStageBytes, &tm_w, kb * (kLK / 2), row, bar, pol);
        }
        r.next();
      }
    }
    if (!ok && lane == 0) give_up();
    drain(r, full);
  } else if (warp == 3) {
    // ------------------------------------------------------------------ activation codes and scales
    const bool lead = elect_one();
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    pdl_wait_prior_grid();  // the quantiser's
    Ring<kStages> r;
    bool ok = true;
    for (int t = t0; t < c.tiles && ok; t += step) {
      const int xt = x_tile(t);
      const uint8_t* sf = p.x_sf + (static_cast<size_t>(xt) * kChunks * (p.kp / 64) + kb0 * 4) * 512;
      for (int kb = kb0; kb < kb0 + nkb; ++kb, sf += kSfChunk) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&empty[r.s]), r.ph ^ 1u));
        if (!ok) break;
        if (lead) {
          const uint32_t bar = smem_addr(&full[r.s]);
          const uint32_t st = smem_addr(smem) + r.s * TL::kStageBytes + kABytes;
          mbar_arrive_expect_tx(bar, TL::kBBytes + kSfChunk * kChunks);
          tma_load_2d(st, &tm_x, kb * (kLK / 2), xt * NT, bar, pol);
#pragma unroll
          for (int ch = 0; ch < kChunks; ++ch)
            bulk_copy_g2s(st + TL::kBBytes + kSfChunk * (1 + ch), sf + static_cast<size_t>(ch) * (p.kp / 64) * 512, kSfChunk,
                          bar, pol);
        }
        r.next();
      }
    }
    if (!ok && lane == 0) give_up();
    drain(r, full);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue
    constexpr uint32_t idesc = idesc_fp4(kLM, NT);
    const bool lead = elect_one();
    Ring<kStages> r;
    bool ok = true;
    int n = 0;
    for (int t = t0; t < c.tiles && ok; t += step, ++n) {
      const int buf = n & 1;
      // this accumulator's previous tile must have left tensor memory
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&acc_empty[buf]), static_cast<uint32_t>(((n >> 1) & 1) ^ 1)));
      tmem_fence_after_sync();
      const uint32_t acc = tmem + static_cast<uint32_t>(buf * NT);
      for (int kb = 0; kb < nkb && ok; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&full[r.s]), r.ph));
        if (!ok) break;
        tmem_fence_after_sync();
        if (lead) {
          const uint32_t st = smem_addr(smem) + r.s * TL::kStageBytes;
          const uint32_t sf = st + kABytes + TL::kBBytes;
          const uint64_t da = umma_desc_sw128(st), db = umma_desc_sw128(st + kABytes), ds = sf_desc(sf);
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // 64 codes = 32 bytes along the swizzle row
            const uint32_t sfa = tmem + TL::kSfaCol + 4 * k, sfb = tmem + TL::kSfbCol + 4 * kChunks * k;
            tmem_copy_sf(sfa, ds + 32 * k);
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) tmem_copy_sf(sfb + 4 * ch, ds + (kSfChunk / 16) * (1 + ch) + 32 * k);
            umma_fp4(acc, da + 2 * k, db + 2 * k, idesc, sfa, sfb, (kb | k) != 0 ? 1u : 0u);
          }
          umma_commit(smem_addr(&empty[r.s]));  // the stage is free once these have read it
        }
        r.next();
      }
      if (lead) umma_commit(smem_addr(&acc_full[buf]));
      __syncwarp();
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ weight scales
    // Four stages (64 bytes a row) are fetched at a time into shared memory, four lanes a row so that each row is
    // one request, one group ahead of the stores; a group ends with its tile. For a stage lane r then takes the
    // 16 scale bytes of rows r, r + 32, r + 64, r + 96: word k of a row belongs to MMA k. (Loaded to registers,
    // 16 bytes of a row a lane, each row took two requests: 16 rows of 12288 -> 6144,
    // weights out of HBM, 23.1 us instead of 20.9.)
    // Buffer: row r's 16-byte piece g at 64 r + 16 (g ^ ((r >> 1) & 3)), so that neither side has bank conflicts.
    constexpr int kFetch = 4, kBufs = TL::kSfBufs;
    int ft = t0, frow = tile_row(t0), fkb = kb0, fb = 0;  // the next stage to fetch, and its buffer
    auto fetch = [&] {
      const int g = lane & 3;
      const bool on = ft < c.tiles && fkb + g < kb0 + nkb;
      const int row0 = on ? frow + (lane >> 2) : 0;
      const uint8_t* src = p.w_bs + (on ? static_cast<size_t>(fkb + g) * 16 : 0);
      const uint32_t dst = smem_addr(sf_raw) + fb * TL::kSfBytes;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 8 * i + (lane >> 2);
        const bool in = on && row0 + 8 * i < p.N;
        // (in: the row exists; otherwise nothing is read and the piece becomes zeros)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * 64 + ((g ^ ((r >> 1) & 3)) << 4)),
                     "l"(src + (in ? static_cast<size_t>(row0 + 8 * i) * (p.kp / 16) : 0)), "r"(in ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (++fb == kBufs) fb = 0;
      fkb += kFetch;
      if (fkb >= kb0 + nkb) {
        fkb = kb0;
        ft += step;
        if (ft < c.tiles) frow = tile_row(ft);
      }
    };
#pragma unroll
    for (int i = 0; i < kBufs - 1; ++i) fetch();
    Ring<kStages> r;
    bool ok = true;
    int ub = 0;
    for (int t = t0; t < c.tiles && ok; t += step)
      for (int kb = 0; kb < nkb && ok; kb += kFetch) {
        __syncwarp();  // the buffer that the next fetch fills has been read by every lane
        fetch();
        asm volatile("cp.async.wait_group %0;" ::"n"(kBufs - 1) : "memory");
        __syncwarp();
        const uint32_t src = smem_addr(sf_raw) + ub * TL::kSfBytes + lane * 64;
        if (++ub == kBufs) ub = 0;
#pragma unroll
        for (int g = 0; g < kFetch; ++g)
          if (kb + g < nkb && ok) {
            uint4 d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(d[j].x), "=r"(d[j].y), "=r"(d[j].z), "=r"(d[j].w)
                           : "r"(src + j * 2048 + ((g ^ ((lane >> 1) & 3)) << 4))
                           : "memory");
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&empty[r.s]), r.ph ^ 1u));
            if (ok) {
              uint4* dst = reinterpret_cast<uint4*>(smem + r.s * TL::kStageBytes + kABytes + TL::kBBytes) + lane;
              dst[0] = make_uint4(d[0].x, d[1].x, d[2].x, d[3].x);
              dst[32] = make_uint4(d[0].y, d[1].y, d[2].y, d[3].y);
              dst[64] = make_uint4(d[0].z, d[1].z, d[2].z, d[3].z);
              dst[96] = make_uint4(d[0].w, d[1].w, d[2].w, d[3].w);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&full[r.s]));
              r.next();
            }
          }
      }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) give_up();
  } else if (warp >= 4 && !SPLIT) {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;
    pdl_wait_prior_grid();  // x_rs comes from the quantiser
    int n = 0;
    for (int t = t0; t < c.tiles; t += step, ++n) {
      const int buf = n & 1;
      const int row = tile_row(t) + 32 * q + lane, r0 = x_tile(t) * NT;
      const float rw = row < p.N ? __ldg(p.w_rs + row) : 0.0f;
      float* rx = rx_all + q * NT;
      load_rx(rx, r0);
      const bool done = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&acc_full[buf]), static_cast<uint32_t>((n / 2) & 1)));
      tmem_fence_after_sync();
      if (!done || aborted()) {
        if (lane == 0) give_up();
        break;
      }
#pragma unroll
      for (int c0 = 0; c0 < NT; c0 += 16) {
        if (r0 + c0 < p.R) {
          uint32_t v[16];
          tmem_ld16(tmem + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(buf * NT + c0), v);
          float s[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = __uint_as_float(v[e]);
          store16(r0, c0, row, s, rw, rx);
        }
      }
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&acc_empty[buf]));
    }
  }

  if constexpr (SPLIT) {
    // ------------------------------------------------------------------ joining the k ranges
    // The MMAs of every CTA of the cluster are done after the first barrier, so the first CTA's ring
    // is free for the others' partial sums: slot (rank - 1)[column][128 rows].
    const int q = warp & 3;
    const bool epi = warp >= 4;
    float* slots = reinterpret_cast<float*>(smem);
    bool done = true;
    // the scales of the first CTA's epilogue, under the last MMAs
    const int row = tile_row(t0) + 32 * q + lane, r0 = x_tile(t0) * NT;
    float rw = 0.0f;
    float* rx = rx_all + q * NT;
    if (epi) {
      pdl_wait_prior_grid();
      if (rank == 0) {
        if (row < p.N) rw = __ldg(p.w_rs + row);
        load_rx(rx, r0);
      }
      done = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&acc_full[0]), 0));
      tmem_fence_after_sync();
      if (!done && lane == 0) give_up();
    }
    __syncthreads();
    cluster_barrier();
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    if (epi && rank != 0) {
      uint32_t dst;
      const float* mine = slots + static_cast<size_t>(rank - 1) * NT * kLM + 32 * q + lane;
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_addr(mine)));
#pragma unroll 1
      for (int c0 = 0; c0 < NT; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(lane_base + c0, v);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dst + (c0 + e) * kLM * 4), "r"(v[e]) : "memory");
      }
    }
    cluster_barrier();
    if (epi && rank == 0 && !aborted()) {
#pragma unroll
      for (int c0 = 0; c0 < NT; c0 += 16) {
        if (r0 + c0 < p.R) {
          uint32_t v[16];
          tmem_ld16(lane_base + c0, v);
          float s[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) s[e] = __uint_as_float(v[e]);
          for (int k = 1; k < c.splits; ++k)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              s[e] = __fadd_rn(s[e], slots[(static_cast<size_t>(k - 1) * NT + c0 + e) * kLM + 32 * q + lane]);
          store16(r0, c0, row, s, rw, rx);
        }
      }
    }
  }
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    // after a timeout the epilogue may have stopped early: tensor memory is released only once the
    // MMAs issued into it are done (normally this returns at once)
    if (lane == 0 && aborted())
      for (int b = 0; b < 2; ++b) {
        (void)mbar_wait_bounded(smem_addr(&acc_full[b]), 0);
        (void)mbar_wait_bounded(smem_addr(&acc_full[b]), 1);
      }
    __syncwarp();
    tmem_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  // (no early launch: a stage that follows may read y, as its weights, before its own wait)
}

// ------------------------------------------------------------------------------- host side
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct LinearWs {
  uint8_t* q;
  uint8_t* sf;
  float* rs;
};
// Workspace: codes [R, kp / 2], block scales, row scales [R]. The block scales take whole 128-row
// blocks per activation tile; the size allows for the tile that needs the most of them.
size_t bind(LinearWs* w, uint8_t* p, int R, int K) {
  const size_t kp = fp4_padded(K);
  uint8_t* p0 = p;
  w->q = p;
  p += round256(static_cast<size_t>(R) * kp / 2);
  w->rs = reinterpret_cast<float*>(p);
  p += round256(static_cast<size_t>(R) * 4);
  w->sf = p;
  const size_t blocks = R <= 128 ? 8 : (static_cast<size_t>(R) + 63) / 64 + 2;  // see make_sched
  p += blocks * (kp / 64) * 512;
  return static_cast<size_t>(p - p0);
}

template <int NT, bool SPLIT, bool GROUP>
cudaError_t launch_tile(const CUtensorMap& tw, const CUtensorMap& tx, const LinearParams& p, const LinearSched& c,
                        int sm_count, cudaStream_t stream) {
  static std::mutex mu;
  static bool done[64] = {};
  const void* kernel = reinterpret_cast<const void*>(linear_fp4_kernel<NT, SPLIT, GROUP>);
  constexpr size_t smem = LTile<NT>::kSmem;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (err != cudaSuccess) return err;
      done[dev] = true;
    }
  }
  CUtensorMap w = tw, x = tx;
  LinearParams pp = p;
  LinearSched cc = c;
  void* args[] = {&w, &x, &pp, &cc};
  cudaLaunchConfig_t cfg = {};
  const int cluster = SPLIT ? c.splits : 1;
  cfg.gridDim = dim3(static_cast<unsigned>(SPLIT || c.tiles < sm_count ? c.tiles * cluster : sm_count));
  cfg.blockDim = dim3(kLThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int NT>
cudaError_t launch_nt(const CUtensorMap& tw, const CUtensorMap& tx, const LinearParams& p, const LinearSched& c,
                      int sm_count, cudaStream_t stream) {
  if (c.splits > 1) return launch_tile<NT, true, false>(tw, tx, p, c, sm_count, stream);
  if constexpr (NT >= 128)
    if (c.group) return launch_tile<NT, false, true>(tw, tx, p, c, sm_count, stream);
  return launch_tile<NT, false, false>(tw, tx, p, c, sm_count, stream);
}

bool code_map(CUtensorMap* tm, const uint8_t* base, int rows, int kp, int box_rows, TmapEncodeFn enc) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kp / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kp / 2)};
  const cuuint32_t box[2] = {kLK / 2, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t fp4_linear_workspace_bytes(int R, int, int K) {
  LinearWs w;
  return bind(&w, nullptr, R, K);
}

cudaError_t launch_linear_fp4(const Fp4LinearArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const TmapEncodeFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  LinearWs w;
  bind(&w, a.ws, a.R, a.K);
  const int kp = fp4_padded(a.K);
  const LinearSched c = make_sched(a.R, a.N, kp, di.sm_count);
  CUtensorMap tw, tx;
  if (!code_map(&tw, a.w.q, a.N, kp, kLM, enc) || !code_map(&tx, w.q, a.R, kp, c.nt, enc)) return cudaErrorNotSupported;
  err = launch_fp4_quantize(a.x, w.q, w.sf, w.rs, a.status, a.valid, a.R, a.K, stream, c.nt);
  if (err != cudaSuccess) return err;
  const LinearParams p{a.w.bs, a.w.rs, w.sf, w.rs, a.y, a.status, a.R, a.N, kp};
  switch (c.nt) {
    case 16: return launch_nt<16>(tw, tx, p, c, di.sm_count, stream);
    case 32: return launch_nt<32>(tw, tx, p, c, di.sm_count, stream);
    case 64: return launch_nt<64>(tw, tx, p, c, di.sm_count, stream);
    case 128: return launch_nt<128>(tw, tx, p, c, di.sm_count, stream);
    case 192: return launch_nt<192>(tw, tx, p, c, di.sm_count, stream);
    default: return launch_nt<224>(tw, tx, p, c, di.sm_count, stream);
  }
}

}  // namespace mtp
