// Output stage over the FP4 copy of lm_head ("glm5next_mtp_head.rs", `forward_one`:
// shared_head.norm, the lm_head gemv, argmax; the copy is used for drafting only, as the source's
// FP8 copy is):  logits[b, v] = rs[v] * sum_k s[v, k/16] code[v, k] xhat[b, k],  then the argmax.
//
// Bound by the read of the copy (9/16 byte a weight: 0.54 GB at H = 6144, V = 154880, 80 us at the
// measured copy rate), with four weights to a lane's byte pair: the work per byte is what shapes the
// kernel. Codes are widened by the hardware E2M1 -> f16 conversion, multiplied by their block scale in
// f16 (exact: 6 significant bits) and fed to warp-level MMAs (m16n8k16, f16 x f16 -> fp32) as register
// operands, the batch as N = 8 or 16. Any batch size takes this path: at one sequence the MMAs are as
// few instructions as the dot products would be.
//
// Kernels:
//  1. fp4_xhat_kernel: xhat in f16, in the order of the MMA's B fragments, into the workspace;
//  2. sweep_fp4_kernel, one CTA per SM over 128-row tiles. One warp streams stages of 128 rows x 512
//     codes with their scales (2-D TMA, 36 KB a stage; 256 contiguous bytes a row, since DRAM pages
//     are left too soon with less), one the matching activations (one bulk copy a stage, from L2).
//     Sixteen consumer warps: four row quarters (two 16-row MMA tiles each, so an activation fragment
//     in registers serves 32 rows) times four quarters of a stage's columns. The column quarters' sums
//     meet in shared memory once per tile.
// Measured at H = 6144, V = 154880: one sequence 87 us (6.2 TB/s, 0.92 of the copy rate), 16 sequences 120 us.
// Up to eight sequences the read is the bound; with 16 the consumers are (82 % of the issue slots, and one MMA of
// 16 x 8 x 16 takes a scheduler's tensor pipe 8.4 cycles), which is also why twice the warps with half the rows each
// gained (141 -> 120 us).
// The tensor cores' running sum is restarted every 128 columns and added in fp32.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "tc.cuh"

namespace mtp {

namespace {

// Workspace: the output stage's header (finished-CTA counter and running picks, common.cuh), the
// activations' unscale factors [16] fp32, then xhat in f16 for 8 or 16 sequences, in fragment order:
// per 32 columns and 8 sequences 512 bytes, 16 for each lane (g, t4) of an MMA's B operand -- columns
// 8 t4 .. 8 t4 + 7 of sequence g.
constexpr int kUnscaleOffset = kWsBytes;
constexpr int kXhatOffset = kWsBytes + 256;
constexpr int kStageK = 512;  // codes per row and stage
__host__ __device__ constexpr int stage_padded(int h) { return (h + kStageK - 1) / kStageK * kStageK; }

constexpr int kNormThreads = 320;

// A load that stays in front of what follows.
__device__ __forceinline__ uint4 ld_now(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// xhat_b = shared_head.norm(x_b) in BF16 (the exact rounding of the other kernels), stored as f16
// times a power of two that puts the largest element just under 2^15: exact down to 2^-29 of it,
// and below that within 2^-40 of it. One CTA per activation row; rows past B and columns past H
// become zeros.
__global__ void __launch_bounds__(kNormThreads) fp4_xhat_kernel(const Fp4SweepArgs a) {
  __shared__ DF part[kNormThreads / 32];
  __shared__ float pmax[kNormThreads / 32], pval[kNormThreads / 32];
  __shared__ float fac[3];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.H, kp = stage_padded(H), nt = a.B <= 8 ? 1 : 2;
  // columns 8 v .. 8 v + 7 of this sequence
  auto piece = [&](int v) {
    return reinterpret_cast<uint4*>(a.ws + kXhatOffset) + (static_cast<size_t>(v >> 2) * nt + (b >> 3)) * 32 + (b & 7) * 4 + (v & 3);
  };
  pdl_wait_prior_grid();
  // This row's first pieces are asked for before the sweep's weight stream can get in front of them.
  constexpr int kHeld = 3;
  uint4 hx[kHeld], hw[kHeld];
  const bool vec = H % 8 == 0;  // rows of whole 16-byte pieces are read a piece at a time
  const uint16_t* x = a.x + static_cast<size_t>(b < a.B ? b : 0) * H;
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  const uint4* wv = reinterpret_cast<const uint4*>(a.final_norm_w);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int v = tid + i * kNormThreads;
    hx[i] = hw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (vec && b < a.B && v < H / 8) {
      hx[i] = ld_now(xv + v);
      hw[i] = ld_now(wv + v);
    }
  }
  // The sweep may launch now: it reads the copy before its own wait (written, if it was, before this
  // grid's wait ended), and the activations after it.
  pdl_launch_dependents();
  if (b >= a.B) {
    for (int v = tid; v < kp / 8; v += kNormThreads) *piece(v) = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) reinterpret_cast<float*>(a.ws + kUnscaleOffset)[b] = 0.0f;
    return;
  }
  // sum of squares (double-float), max |x w| and max |x| of the row times sc, a power of two: 1, or what
  // brings the row near one when its squares leave the fp32 range
  float sc = 1.0f;
  auto sums = [&](float& biggest) {
    DF2 acc{0ull, 0ull};
    float mx = 0.0f, mv = 0.0f;
    auto add = [&](float v0, float v1, float w0, float w1) {
      v0 = __fmul_rn(v0, sc);
      v1 = __fmul_rn(v1, sc);
      const uint64_t v = f2_pack(v0, v1);
      df2_add(acc, f2_mul(v, v));
      mx = fmaxf(mx, fmaxf(fabsf(__fmul_rn(v0, w0)), fabsf(__fmul_rn(v1, w1))));
      mv = fmaxf(mv, fmaxf(fabsf(v0), fabsf(v1)));
    };
    auto add8 = [&](const uint4& q, const uint4& wq) {
      const uint32_t u[4] = {q.x, q.y, q.z, q.w}, w4[4] = {wq.x, wq.y, wq.z, wq.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) add(bf16_lo(u[i]), bf16_hi(u[i]), bf16_lo(w4[i]), bf16_hi(w4[i]));
    };
    if (vec) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) add8(hx[i], hw[i]);  // (zeros past the row)
      for (int v = tid + kHeld * kNormThreads; v < H / 8; v += kNormThreads) add8(xv[v], wv[v]);
    } else {
      for (int k = tid; k < H; k += kNormThreads) add(bf16_bits_to_f32(x[k]), 0.0f, bf16_bits_to_f32(a.final_norm_w[k]), 0.0f);
    }
    DF sum = df_add(df2_x(acc), df2_y(acc));
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      sum = df_add(sum, shfl_xor_df(sum, m));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, m));
    }
    __syncthreads();  // the previous call's partials are read
    if (lane == 0) {
      part[warp] = sum;
      pmax[warp] = mx;
      pval[warp] = mv;
    }
    __syncthreads();
    DF tot = part[0];
    biggest = pmax[0];
    for (int i = 1; i < kNormThreads / 32; ++i) {
      tot = df_add(tot, part[i]);
      biggest = fmaxf(biggest, pmax[i]);
    }
    return tot;
  };
  float m;
  DF tot = sums(m);
  if (!(tot.hi >= 1e-24f && tot.hi <= 1e37f && m <= 1e37f)) {  // the same for every thread
    float mv = 0.0f;
    for (int i = 0; i < kNormThreads / 32; ++i) mv = fmaxf(mv, pval[i]);
    int e = 0;
    if (mv > 0.0f && mv <= 3.4e38f) (void)frexpf(mv, &e);
    sc = ldexpf(1.0f, e < -120 ? 120 : -e);
    tot = sums(m);
  }
  if (tid == 0) {
    const double ms = (static_cast<double>(tot.hi) + static_cast<double>(tot.lo)) / static_cast<double>(H);
    const double r = rsqrt(ms + static_cast<double>(a.eps) * static_cast<double>(sc) * static_cast<double>(sc));
    const float rh = static_cast<float>(r), rl = static_cast<float>(r - static_cast<double>(rh));
    fac[0] = rh;
    fac[1] = rl;
    // the largest |xhat| (rounding is monotonic, so it is the rounded maximum)
    const float yh = __fmul_rn(m, rh);
    const float big = bf16_bits_to_f32(bf16_rne_df(yh, __fmaf_rn(m, rl, __fmaf_rn(m, rh, -yh))));
    int e = 15;
    if (big > 0.0f && big <= 3.0e38f) (void)frexpf(big, &e);
    if (e < -100) e = -100;  // 2^(15 - e) stays in the fp32 range
    fac[2] = ldexpf(1.0f, 15 - e);
    reinterpret_cast<float*>(a.ws + kUnscaleOffset)[b] = ldexpf(1.0f, e - 15);
  }
  __syncthreads();
  const float rh = fac[0], rl = fac[1], xs = fac[2];
#pragma unroll 1
  for (int v = tid; v < kp / 8; v += kNormThreads) {
    uint32_t xu[4] = {0u, 0u, 0u, 0u}, wu[4] = {0u, 0u, 0u, 0u};
    if (vec) {
      if (8 * v < H) {
        const uint4 q = xv[v], wq = wv[v];  // from L1
        xu[0] = q.x, xu[1] = q.y, xu[2] = q.z, xu[3] = q.w;
        wu[0] = wq.x, wu[1] = wq.y, wu[2] = wq.z, wu[3] = wq.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * v + i < H) {
          xu[i >> 1] |= static_cast<uint32_t>(x[8 * v + i]) << (16 * (i & 1));
          wu[i >> 1] |= static_cast<uint32_t>(a.final_norm_w[8 * v + i]) << (16 * (i & 1));
        }
    }
    uint32_t o[4];
    if (sc == 1.0f) {
      const float wf[8] = {bf16_lo(wu[0]), bf16_hi(wu[0]), bf16_lo(wu[1]), bf16_hi(wu[1]),
                           bf16_lo(wu[2]), bf16_hi(wu[2]), bf16_lo(wu[3]), bf16_hi(wu[3])};
      const uint4 y = bf16x8_scaled_rne(xu, wf, rh, rl);
      o[0] = y.x, o[1] = y.y, o[2] = y.z, o[3] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = bf16_scaled_rne(__fmul_rn(__fmul_rn(bf16_lo(xu[i]), sc), bf16_lo(wu[i])), rh, rl) |
               (bf16_scaled_rne(__fmul_rn(__fmul_rn(bf16_hi(xu[i]), sc), bf16_hi(wu[i])), rh, rl) << 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f16x2_bits(__fmul_rn(bf16_lo(o[i]), xs), __fmul_rn(bf16_hi(o[i]), xs));
    *piece(v) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

constexpr int kRows = 128;             // rows per tile
constexpr int kConsumers = 16;         // warps: four row quarters x four column quarters
constexpr int kMT = kRows / 4 / 16;    // 16-row MMA tiles per warp
constexpr int kSThreads = (kConsumers + 2) * 32;
constexpr int kCodeBytes = kRows * kStageK / 2;    // 32 KB: two swizzled boxes of 128 bytes a row
constexpr int kScaleBytes = kRows * kStageK / 16;  // 4 KB
constexpr int kStageBytes = kCodeBytes + kScaleBytes;

template <int NT>
struct SweepCfg {
  static constexpr int kStages = NT == 1 ? 5 : 4;
  static constexpr int kXBytes = NT * (kStageK / 32) * 512;  // activations of a stage
  static constexpr int kXStages = 3;
  static constexpr int kPartBytes = 4 * 8 * NT * kRows * 4;  // [column quarter][sequence][row] fp32
  static constexpr size_t kSmem =
      1024 + static_cast<size_t>(kStages) * kStageBytes + kXStages * kXBytes + kPartBytes + 2 * (kStages + kXStages) * 8 + kConsumers * 2 * NT * sizeof(ArgBest);
  static_assert(kSmem <= 226 * 1024, "shared memory");
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// A load that stays where it is written (an ordinary one was moved to its use, after the column loop,
// and every tile then waited ~3,000 cycles for it).
__device__ __forceinline__ float ldg_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
// Whether ok holds for every consumer thread (named barrier 1).
__device__ __forceinline__ bool consumers_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(kConsumers * 32)
      : "memory");
  return r != 0;
}

template <int NT>
__global__ void __launch_bounds__(kSThreads, 1)
    sweep_fp4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_s,
                     const Fp4SweepArgs a, unsigned long long wait_ns) {
  using C = SweepCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* xring = smem + C::kStages * kStageBytes;
  float* part = reinterpret_cast<float*>(xring + C::kXStages * C::kXBytes);
  uint64_t* afull = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(part) + C::kPartBytes);
  uint64_t* aempty = afull + C::kStages;
  uint64_t* xfull = aempty + C::kStages;
  uint64_t* xempty = xfull + C::kXStages;
  ArgBest* wbest = reinterpret_cast<ArgBest*>(xempty + C::kXStages);  // [warp][2 NT]
  __shared__ int is_last;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t V = a.V;
  const int KP = stage_padded(a.H) / kStageK;
  const int T = static_cast<int>((V + kRows - 1) / kRows);
  const int t0 = static_cast<int>(static_cast<int64_t>(T) * blockIdx.x / gridDim.x);
  const int t1 = static_cast<int>(static_cast<int64_t>(T) * (blockIdx.x + 1) / gridDim.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_addr(&afull[i]), 1);
      mbar_init(smem_addr(&aempty[i]), kConsumers);
    }
    for (int i = 0; i < C::kXStages; ++i) {
      mbar_init(smem_addr(&xfull[i]), 1);
      mbar_init(smem_addr(&xempty[i]), kConsumers);
    }
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_s)) : "memory");
  }
  __syncthreads();

  if (warp == kConsumers) {
    // ------------------------------------------------------------------ the copy
    // It does not depend on the kernels before: the stream starts at once.
    const bool lead = elect_one();
    const uint64_t pol = l2_evict_first_policy();
    uint64_t pol_s;  // a 32-byte piece of a row's scales shares its DRAM burst with the next stages'
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol_s));
    int slot = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int t = t0; t < t1 && ok; ++t) {
      for (int kp = 0; kp < KP; ++kp) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&aempty[slot]), ph, wait_ns));
        if (!ok) break;
        if (lead) {
          const uint32_t bar = smem_addr(&afull[slot]);
          const uint32_t dst = smem_addr(smem) + slot * kStageBytes;
          mbar_arrive_expect_tx(bar, kStageBytes);
          // (past the end of a row the second box is zeros)
          tma_load_2d(dst, &tm_q, kp * (kStageK / 2), t * kRows, bar, pol);
          tma_load_2d(dst + kCodeBytes / 2, &tm_q, kp * (kStageK / 2) + 128, t * kRows, bar, pol);
          tma_load_2d(dst + kCodeBytes, &tm_s, kp * (kStageK / 16), t * kRows, bar, pol_s);
        }
        ++issued;
        if (++slot == C::kStages) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) store_status(a.status, MTP_ERR_TIMEOUT);
    // every copy issued must land before the CTA's shared memory goes away
    for (int s = 0; s < C::kStages && s < issued; ++s)
      (void)mbar_wait_bounded(smem_addr(&afull[s]), static_cast<uint32_t>(((issued - s + C::kStages - 1) / C::kStages - 1) & 1));
  } else if (warp == kConsumers + 1) {
    // ------------------------------------------------------------------ activations
    const bool lead = elect_one();
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    pdl_wait_prior_grid();  // the activations come from the preceding kernel
    int slot = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int t = t0; t < t1 && ok; ++t) {
      for (int kp = 0; kp < KP; ++kp) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&xempty[slot]), ph, wait_ns));
        if (!ok) break;
        if (lead) {
          const uint32_t bar = smem_addr(&xfull[slot]);
          mbar_arrive_expect_tx(bar, C::kXBytes);
          bulk_copy_g2s(smem_addr(xring) + slot * C::kXBytes, a.ws + kXhatOffset + static_cast<size_t>(kp) * C::kXBytes,
                        C::kXBytes, bar, pol);
        }
        ++issued;
        if (++slot == C::kXStages) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) store_status(a.status, MTP_ERR_TIMEOUT);
    for (int s = 0; s < C::kXStages && s < issued; ++s)
      (void)mbar_wait_bounded(smem_addr(&xfull[s]), static_cast<uint32_t>(((issued - s + C::kXStages - 1) / C::kXStages - 1) & 1));
  } else {
    // ------------------------------------------------------------------ consumers
    const int g = lane >> 2, t4 = lane & 3;
    const int rq = warp >> 2, quarter = warp & 3;  // rows 32 rq .., columns 128 quarter .. of a stage
    // this warp's 64 bytes of a row's codes: box quarter / 2, 16-byte chunks 4 (quarter % 2) ..
    const uint32_t box = static_cast<uint32_t>(quarter >> 1) * (kCodeBytes / 2);
    const int chunk0 = 4 * (quarter & 1);
    const uint32_t pick = (t4 >> 1) ? 0x5531u : 0x4420u;  // bytes 2 c + (t4 / 2) of a word, c = 0, 1
    // In the epilogue a thread finishes row `er` of the tile for sequences eq, eq + 4, ...
    const int er = threadIdx.x & (kRows - 1), eq = threadIdx.x / kRows;
    ArgBest best[2 * NT];
    float us[2 * NT];  // unscale factors of those sequences
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) best[i] = ArgBest{0.0f, -1};
    int aslot = 0, xslot = 0;
    uint32_t ap = 0, xp = 0;
    bool ok = true;
    bool waited = false;
    for (int t = t0; t < t1; ++t) {
      float acc[kMT][NT][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int jn = 0; jn < NT; ++jn) acc[mt][jn][0] = acc[mt][jn][1] = acc[mt][jn][2] = acc[mt][jn][3] = 0.0f;
      const int64_t row = static_cast<int64_t>(t) * kRows + er;
      float rs = 0.0f;  // the row scale, ahead of the epilogue
      if (row < V) rs = ldg_now(a.w.rs + row);
      for (int kp = 0; kp < KP; ++kp) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&xfull[xslot]), xp, wait_ns) &&
                                         mbar_wait_bounded(smem_addr(&afull[aslot]), ap, wait_ns));
        if (!ok) break;
        const uint32_t st = smem_addr(smem) + aslot * kStageBytes;
        const uint32_t xs = smem_addr(xring) + xslot * C::kXBytes + (4 * quarter * NT * 32 + lane) * 16;
        uint32_t sc[kMT][2][2];  // f16 scale pairs of rows g, g + 8: chunks 0, 1 and 2, 3
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w0, w1;
            lds_v2(w0, w1, st + kCodeBytes + (32 * rq + 16 * mt + g + 8 * h) * (kStageK / 16) + 8 * quarter);
            sc[mt][h][0] = e4m3x2_to_f16x2(__byte_perm(w0, 0u, pick));
            sc[mt][h][1] = e4m3x2_to_f16x2(__byte_perm(w1, 0u, pick));
          }
        float c4[kMT][NT][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int jn = 0; jn < NT; ++jn) c4[mt][jn][0] = c4[mt][jn][1] = c4[mt][jn][2] = c4[mt][jn][3] = 0.0f;
#pragma unroll
        for (int cc = 0; cc < 4; cc += 2) {
          uint32_t r[kMT][4];  // rows g, g + 8 of chunk cc, then of chunk cc + 1
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
            ldmatrix_x4(r[mt], st + box + swz(32 * rq + 16 * mt + (lane & 15), chunk0 + cc + (lane >> 4)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 x[NT];  // B fragments of the chunk's two k16 steps
#pragma unroll
            for (int jn = 0; jn < NT; ++jn) x[jn] = lds128(xs + ((cc + i) * NT + jn) * 512);
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              uint32_t va[4], vb[4];
              e2m1x8_to_f16x2x4(r[mt][2 * i], va);
              e2m1x8_to_f16x2x4(r[mt][2 * i + 1], vb);
              const uint32_t sa = __byte_perm(sc[mt][0][cc >> 1], 0u, i == 0 ? 0x1010u : 0x3232u);
              const uint32_t sb = __byte_perm(sc[mt][1][cc >> 1], 0u, i == 0 ? 0x1010u : 0x3232u);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t f[4] = {f16x2_mul(va[2 * h], sa), f16x2_mul(vb[2 * h], sb),
                                       f16x2_mul(va[2 * h + 1], sa), f16x2_mul(vb[2 * h + 1], sb)};
#pragma unroll
                for (int jn = 0; jn < NT; ++jn)
                  mma_f16(c4[mt][jn], f, h == 0 ? x[jn].x : x[jn].z, h == 0 ? x[jn].y : x[jn].w);
              }
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
          for (int jn = 0; jn < NT; ++jn)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][jn][i] = __fadd_rn(acc[mt][jn][i], c4[mt][jn][i]);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_addr(&aempty[aslot]));
          mbar_arrive(smem_addr(&xempty[xslot]));
        }
        if (++aslot == C::kStages) {
          aslot = 0;
          ap ^= 1u;
        }
        if (++xslot == C::kXStages) {
          xslot = 0;
          xp ^= 1u;
        }
      }
      // a consumer that gave up takes the others with it, so that all meet at the barriers below (and the
      // previous tile's partial sums have been read)
      ok = consumers_all(ok);
      if (!ok) break;
      if (!waited) {
        pdl_wait_prior_grid();  // the unscale factors come from the preceding kernel
        waited = true;
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) us[i] = __ldcg(reinterpret_cast<const float*>(a.ws + kUnscaleOffset) + eq + 4 * i);
      }
      // ---- the column quarters' sums, rows swizzled by the sequence so that neither the fragments'
      // stores nor the rows' loads conflict. The epilogue is short and its stores are whole 128-byte
      // lines: straight from the fragments (unrolled, 32 bytes of a row at a time, on a quarter of the
      // warps) it held the stages back for 7,500 cycles a tile at 16 sequences.
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int jn = 0; jn < NT; ++jn)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            part[((quarter * 8 * NT + 8 * jn + 2 * t4 + (i & 1)) * kRows) + ((32 * rq + 16 * mt + g + 8 * (i >> 1)) ^ (t4 << 3))] =
                acc[mt][jn][i];
      named_barrier_sync(1, kConsumers * 32);
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int n = eq + 4 * i;
        if (n < a.B && row < V) {
          const float* src = part + n * kRows + (er ^ (((n >> 1) & 3) << 3));
          float s = src[0];
#pragma unroll
          for (int q = 1; q < 4; ++q) s = __fadd_rn(s, src[q * 8 * NT * kRows]);
          const float v = __fmul_rn(__fmul_rn(s, us[i]), rs);
          if (a.logits != nullptr) __stcs(a.logits + static_cast<int64_t>(n) * V + row, v);
          // rows come in ascending order: a later one wins only by a larger value
          if (v > best[i].v || (best[i].i < 0 && v == v)) best[i] = ArgBest{v, static_cast<int32_t>(row)};
        }
      }
    }
    if (!ok && lane == 0) store_status(a.status, MTP_ERR_TIMEOUT);
    // the warp's best of its rows, per sequence
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      ArgBest b = best[i];
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) {
        const float v = __shfl_xor_sync(0xffffffffu, b.v, m);
        const int32_t j = __shfl_xor_sync(0xffffffffu, b.i, m);
        if (j >= 0) arg_update(b, v, j);
      }
      if (lane == 0) wbest[warp * 2 * NT + i] = b;
    }
  }
  __syncthreads();
  pdl_wait_prior_grid();  // the workspace may still be read by the kernel before (no-op if done)
  if (threadIdx.x < a.B) {
    ArgBest c{0.0f, -1};
    const int eq = threadIdx.x & 3;  // the four warps that held this sequence
    for (int w = 4 * eq; w < 4 * eq + 4; ++w) {
      const ArgBest o = wbest[w * 2 * NT + (threadIdx.x >> 2)];
      if (o.i >= 0) arg_update(c, o.v, o.i);
    }
    pick_publish(a.ws, threadIdx.x, c.v, c.i, 0);
    __threadfence();
  }
  __syncthreads();
  unsigned int* counter = reinterpret_cast<unsigned int*>(a.ws);
  if (threadIdx.x == 0) is_last = (atomicAdd(counter, 1u) == gridDim.x - 1) ? 1 : 0;
  __syncthreads();
  if (is_last) {
    __threadfence();
    if (threadIdx.x < a.B) pick_finish(a.ws, threadIdx.x, a.draft, nullptr);
    if (threadIdx.x == 0) atomicExch(counter, 0u);
  }
}

template <int NT>
cudaError_t launch_nt(const CUtensorMap& tq, const CUtensorMap& ts, const Fp4SweepArgs& in, unsigned grid,
                      const DeviceInfo& di, cudaStream_t stream) {
  if (SweepCfg<NT>::kSmem > static_cast<size_t>(di.smem_optin)) return cudaErrorNotSupported;
  CUtensorMap q = tq, s = ts;
  Fp4SweepArgs a = in;
  unsigned long long wait_ns = stage_wait_ns();
  void* args[] = {&q, &s, &a, &wait_ns};
  return launch_pdl(reinterpret_cast<const void*>(sweep_fp4_kernel<NT>), dim3(grid), dim3(kSThreads),
                    SweepCfg<NT>::kSmem, stream, args);
}

bool row_map(CUtensorMap* tm, const uint8_t* base, int64_t rows, int row_bytes, int box_bytes, CUtensorMapSwizzle swizzle,
             TmapEncodeFn enc) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes), kRows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t fp4_sweep_workspace_bytes(int B, int H) {
  return kXhatOffset + static_cast<size_t>(B <= 8 ? 8 : 16) * stage_padded(H) * 2;
}

cudaError_t launch_sweep_fp4(const Fp4SweepArgs& in, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  const TmapEncodeFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  const int kp = fp4_padded(in.H);
  CUtensorMap tq, ts;
  if (!row_map(&tq, in.w.q, in.V, kp / 2, 128, CU_TENSOR_MAP_SWIZZLE_128B, enc) ||
      !row_map(&ts, in.w.bs, in.V, kp / kFp4Block, kStageK / kFp4Block, CU_TENSOR_MAP_SWIZZLE_NONE, enc))
    return cudaErrorNotSupported;
  Fp4SweepArgs a = in;
  void* args[] = {&a};
  err = launch_pdl(reinterpret_cast<const void*>(fp4_xhat_kernel), dim3(a.B <= 8 ? 8 : 16), dim3(kNormThreads), 0,
                   stream, args);
  if (err != cudaSuccess) return err;
  const int64_t T = (static_cast<int64_t>(a.V) + kRows - 1) / kRows;
  const unsigned grid = static_cast<unsigned>(T < di.sm_count ? T : di.sm_count);
  return a.B <= 8 ? launch_nt<1>(tq, ts, a, grid, di, stream) : launch_nt<2>(tq, ts, a, grid, di, stream);
}

}  // namespace mtp
