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
//     are left too soon with less), one the matching activations (one bulk copy a stage, shared by a
//     group of row tiles). Eight consumer warps: two halves of the rows (four 16-row MMA tiles each, so
//     an activation fragment in registers serves 64 rows) times four quarters of a stage's columns.
//     The quarters' sums meet in shared memory once per tile.
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

// Small enough (with 32 registers a thread) to sit on an SM beside a sweep CTA.
constexpr int kNormThreads = 320;

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
  // The sweep may launch at once: it reads the copy before its own wait (written, if it was, before this
  // grid's wait ended), and the activations after it.
  pdl_launch_dependents();
  if (b >= a.B) {
    for (int v = tid; v < kp / 8; v += kNormThreads) *piece(v) = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) reinterpret_cast<float*>(a.ws + kUnscaleOffset)[b] = 0.0f;
    return;
  }
  const uint16_t* x = a.x + static_cast<size_t>(b) * H;
  // sum of squares (double-float) and max |x w| of the row times sc, a power of two: 1, or what brings
  // the row near one when its squares leave the fp32 range
  float sc = 1.0f;
  auto sums = [&](float& biggest) {
    DF acc{0.0f, 0.0f};
    float mx = 0.0f, mv = 0.0f;
    for (int k = tid; k < H; k += kNormThreads) {
      const float v = __fmul_rn(bf16_bits_to_f32(x[k]), sc);
      df_add(acc, __fmul_rn(v, v));
      mx = fmaxf(mx, fabsf(__fmul_rn(v, bf16_bits_to_f32(a.final_norm_w[k]))));
      mv = fmaxf(mv, fabsf(v));
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      acc = df_add(acc, shfl_xor_df(acc, m));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, m));
    }
    __syncthreads();  // the previous call's partials are read
    if (lane == 0) {
      part[warp] = acc;
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
  for (int v = tid; v < kp / 8; v += kNormThreads) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 8 * v + 2 * i + j;
        y[j] = 0.0f;
        if (k < H)
          y[j] = __fmul_rn(bf16_bits_to_f32(bf16_scaled_rne(
                               __fmul_rn(__fmul_rn(bf16_bits_to_f32(x[k]), sc), bf16_bits_to_f32(a.final_norm_w[k])), rh, rl)),
                           xs);
      }
      o[i] = f16x2_bits(y[0], y[1]);
    }
    *piece(v) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

constexpr int kRows = 128;             // rows per tile
constexpr int kConsumers = 8;          // warps
constexpr int kSThreads = (kConsumers + 2) * 32;
constexpr int kGroup = 2;              // row tiles that share an activation stage
constexpr int kCodeBytes = kRows * kStageK / 2;    // 32 KB: two swizzled boxes of 128 bytes a row
constexpr int kScaleBytes = kRows * kStageK / 16;  // 4 KB
constexpr int kStageBytes = kCodeBytes + kScaleBytes;

template <int NT>
struct SweepCfg {
  static constexpr int kStages = NT == 1 ? 5 : 4;
  static constexpr int kXBytes = NT * (kStageK / 32) * 512;  // activations of a stage
  static constexpr int kXStages = 3;
  static constexpr int kPartBytes = 2 * 4 * 3 * 32 * NT * 16;  // [half][MMA tile][other quarter][lane][NT] float4
  static constexpr size_t kSmem =
      1024 + static_cast<size_t>(kStages) * kStageBytes + kXStages * kXBytes + kPartBytes + 2 * (kStages + kXStages) * 8 + kConsumers * 8 * NT * sizeof(ArgBest);
  static_assert(kSmem <= 226 * 1024, "shared memory");
};

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
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
  float4* part = reinterpret_cast<float4*>(xring + C::kXStages * C::kXBytes);
  uint64_t* afull = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(part) + C::kPartBytes);
  uint64_t* aempty = afull + C::kStages;
  uint64_t* xfull = aempty + C::kStages;
  uint64_t* xempty = xfull + C::kXStages;
  ArgBest* wbest = reinterpret_cast<ArgBest*>(xempty + C::kXStages);  // [warp][8 NT]
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
  for (int i = threadIdx.x; i < kConsumers * 8 * NT; i += kSThreads) wbest[i] = ArgBest{0.0f, -1};
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
    for (int gt = t0; gt < t1 && ok; gt += kGroup) {
      const int nt = t1 - gt < kGroup ? t1 - gt : kGroup;
      for (int kp = 0; kp < KP && ok; ++kp) {
        for (int j = 0; j < nt; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&aempty[slot]), ph, wait_ns));
          if (!ok) break;
          if (lead) {
            const uint32_t bar = smem_addr(&afull[slot]);
            const uint32_t dst = smem_addr(smem) + slot * kStageBytes;
            const int row = (gt + j) * kRows;
            mbar_arrive_expect_tx(bar, kStageBytes);
            // (past the end of a row both boxes are zeros)
            tma_load_2d(dst, &tm_q, kp * (kStageK / 2), row, bar, pol);
            tma_load_2d(dst + kCodeBytes / 2, &tm_q, kp * (kStageK / 2) + 128, row, bar, pol);
            tma_load_2d(dst + kCodeBytes, &tm_s, kp * (kStageK / 16), row, bar, pol_s);
          }
          ++issued;
          if (++slot == C::kStages) {
            slot = 0;
            ph ^= 1u;
          }
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
    for (int gt = t0; gt < t1 && ok; gt += kGroup) {
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
    const int half = warp >> 2, quarter = warp & 3;
    // this warp's 64 bytes of a row's codes: box quarter / 2, 16-byte chunks 4 (quarter % 2) ..
    const uint32_t box = static_cast<uint32_t>(quarter >> 1) * (kCodeBytes / 2);
    const int chunk0 = 4 * (quarter & 1);
    const uint32_t pick = (t4 >> 1) ? 0x5531u : 0x4420u;  // bytes 2 c + (t4 / 2) of a word, c = 0, 1
    ArgBest best[NT][2];
#pragma unroll
    for (int jn = 0; jn < NT; ++jn) best[jn][0] = best[jn][1] = ArgBest{0.0f, -1};
    int aslot = 0, xslot = 0;
    uint32_t ap = 0, xp = 0;
    bool ok = true;
    bool waited = false;
    for (int gt = t0; gt < t1; gt += kGroup) {
      const int ntile = t1 - gt < kGroup ? t1 - gt : kGroup;
      float acc[kGroup][4][NT][4];
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int jn = 0; jn < NT; ++jn) acc[j][mt][jn][0] = acc[j][mt][jn][1] = acc[j][mt][jn][2] = acc[j][mt][jn][3] = 0.0f;
      for (int kp = 0; kp < KP && ok; ++kp) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&xfull[xslot]), xp, wait_ns))) {
          ok = false;
          break;
        }
        uint4 x[4][NT];  // B fragments of this warp's 128 columns: two k16 steps a chunk
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int jn = 0; jn < NT; ++jn)
            x[c][jn] = lds128(smem_addr(xring) + xslot * C::kXBytes + (((4 * quarter + c) * NT + jn) * 32 + lane) * 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&xempty[xslot]));
        if (++xslot == C::kXStages) {
          xslot = 0;
          xp ^= 1u;
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          if (j < ntile && ok) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_addr(&afull[aslot]), ap, wait_ns))) {
              ok = false;
            } else {
              const uint32_t st = smem_addr(smem) + aslot * kStageBytes;
#pragma unroll
              for (int mt = 0; mt < 4; ++mt) {
                const int r0 = 64 * half + 16 * mt;
                uint32_t sc[2][2];  // f16 scale pairs of rows g, g + 8: chunks 0, 1 and 2, 3
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint32_t w0, w1;
                  lds_v2(w0, w1, st + kCodeBytes + (r0 + g + 8 * h) * (kStageK / 16) + 8 * quarter);
                  sc[h][0] = e4m3x2_to_f16x2(__byte_perm(w0, 0u, pick));
                  sc[h][1] = e4m3x2_to_f16x2(__byte_perm(w1, 0u, pick));
                }
                float c4[NT][4];
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) c4[jn][0] = c4[jn][1] = c4[jn][2] = c4[jn][3] = 0.0f;
#pragma unroll
                for (int cc = 0; cc < 4; cc += 2) {
                  uint32_t r[4];  // rows g, g + 8 of chunk cc, then of chunk cc + 1
                  ldmatrix_x4(r, st + box + swz(r0 + (lane & 15), chunk0 + cc + (lane >> 4)));
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t va[4], vb[4];
                    e2m1x8_to_f16x2x4(r[2 * i], va);
                    e2m1x8_to_f16x2x4(r[2 * i + 1], vb);
                    const uint32_t sa = __byte_perm(sc[0][cc >> 1], 0u, i == 0 ? 0x1010u : 0x3232u);
                    const uint32_t sb = __byte_perm(sc[1][cc >> 1], 0u, i == 0 ? 0x1010u : 0x3232u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const uint32_t f[4] = {f16x2_mul(va[2 * h], sa), f16x2_mul(vb[2 * h], sb),
                                             f16x2_mul(va[2 * h + 1], sa), f16x2_mul(vb[2 * h + 1], sb)};
#pragma unroll
                      for (int jn = 0; jn < NT; ++jn)
                        mma_f16(c4[jn], f, h == 0 ? x[cc + i][jn].x : x[cc + i][jn].z,
                                h == 0 ? x[cc + i][jn].y : x[cc + i][jn].w);
                    }
                  }
                }
#pragma unroll
                for (int jn = 0; jn < NT; ++jn)
#pragma unroll
                  for (int i = 0; i < 4; ++i) acc[j][mt][jn][i] = __fadd_rn(acc[j][mt][jn][i], c4[jn][i]);
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&aempty[aslot]));
              if (++aslot == C::kStages) {
                aslot = 0;
                ap ^= 1u;
              }
            }
          }
        }
      }
      // a consumer that gave up takes the others with it, so that all meet at the barriers below
      ok = consumers_all(ok);
      if (!ok) break;
      if (!waited) {
        pdl_wait_prior_grid();  // the unscale factors come from the preceding kernel
        waited = true;
      }
      // ---- the quarters' sums of each tile: a warp finishes the MMA tile of its quarter's number
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (j < ntile) {  // the same for every consumer
          named_barrier_sync(1, kConsumers * 32);  // the previous tile's sums are read
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
            if (mt != quarter)
#pragma unroll
              for (int jn = 0; jn < NT; ++jn)
                part[(((half * 4 + mt) * 3 + (quarter < mt ? quarter : quarter - 1)) * 32 + lane) * NT + jn] =
                    make_float4(acc[j][mt][jn][0], acc[j][mt][jn][1], acc[j][mt][jn][2], acc[j][mt][jn][3]);
          named_barrier_sync(1, kConsumers * 32);
          const int64_t rbase = static_cast<int64_t>(gt + j) * kRows + 64 * half + 16 * quarter + g;
          float rs[2];
          rs[0] = rbase < V ? __ldg(a.w.rs + rbase) : 0.0f;
          rs[1] = rbase + 8 < V ? __ldg(a.w.rs + rbase + 8) : 0.0f;
#pragma unroll
          for (int jn = 0; jn < NT; ++jn) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
              if (mt == quarter)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = acc[j][mt][jn][i];
#pragma unroll
            for (int o = 0; o < 3; ++o) {
              const float4 v = part[(((half * 4 + quarter) * 3 + o) * 32 + lane) * NT + jn];
              s[0] = __fadd_rn(s[0], v.x);
              s[1] = __fadd_rn(s[1], v.y);
              s[2] = __fadd_rn(s[2], v.z);
              s[3] = __fadd_rn(s[3], v.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = 8 * jn + 2 * t4 + (i & 1);
              const int64_t row = rbase + 8 * (i >> 1);
              if (n < a.B && row < V) {
                const float us = __ldcg(reinterpret_cast<const float*>(a.ws + kUnscaleOffset) + n);
                const float v = __fmul_rn(__fmul_rn(s[i], us), rs[i >> 1]);
                if (a.logits != nullptr) a.logits[static_cast<int64_t>(n) * V + row] = v;
                arg_update(best[jn][i & 1], v, static_cast<int32_t>(row));
              }
            }
          }
        }
      }
    }
    if (!ok && lane == 0) store_status(a.status, MTP_ERR_TIMEOUT);
    // combine lanes that hold the same sequences (same t4), then publish per warp
#pragma unroll
    for (int jn = 0; jn < NT; ++jn)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        ArgBest b = best[jn][hh];
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
          const float v = __shfl_xor_sync(0xffffffffu, b.v, m);
          const int32_t i = __shfl_xor_sync(0xffffffffu, b.i, m);
          if (i >= 0) arg_update(b, v, i);
        }
        const int n = 8 * jn + 2 * t4 + hh;
        if (g == 0 && n < a.B) wbest[warp * 8 * NT + n] = b;
      }
  }
  __syncthreads();
  pdl_wait_prior_grid();  // the workspace may still be read by the kernel before (no-op if done)
  if (threadIdx.x < a.B) {
    ArgBest c{0.0f, -1};
    for (int w = 0; w < kConsumers; ++w) {
      const ArgBest o = wbest[w * 8 * NT + threadIdx.x];
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
