// Output stage over the FP4 copy of lm_head ("glm5next_mtp_head.rs", `forward_one`:
// shared_head.norm, the lm_head gemv, argmax; the copy is used for drafting only, as the source's
// FP8 copy is):  logits[b, v] = rs[v] * sum_k s[v, k/16] code[v, k] xhat[b, k],  then the argmax.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "fp4_dot.cuh"
#include "internal.h"

namespace mtp {

namespace {

// Workspace: the output stage's header (finished-CTA counter and running picks, common.cuh), the
// activations' unscale factors [16] fp32, then xhat in f16 [8 or 16, fp4_padded(H)].
constexpr int kUnscaleOffset = kWsBytes;
constexpr int kXhatOffset = kWsBytes + 256;

constexpr int kNormThreads = 512;

// xhat_b = shared_head.norm(x_b) in BF16 (the exact rounding of the other kernels), stored as f16
// times a power of two that puts the largest element just under 2^15: exact down to 2^-29 of it,
// and below that within 2^-40 of it. One CTA per activation row; rows past B and columns past H
// become zeros.
__global__ void __launch_bounds__(kNormThreads) fp4_xhat_kernel(const Fp4SweepArgs a) {
  __shared__ DF part[kNormThreads / 32];
  __shared__ float pmax[kNormThreads / 32], pval[kNormThreads / 32];
  __shared__ float fac[3];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.H, kp = fp4_padded(H);
  uint16_t* out = reinterpret_cast<uint16_t*>(a.ws + kXhatOffset) + static_cast<size_t>(b) * kp;
  pdl_wait_prior_grid();
  if (b >= a.B) {
    for (int k = tid; k < kp; k += kNormThreads) out[k] = 0;
    if (tid == 0) reinterpret_cast<float*>(a.ws + kUnscaleOffset)[b] = 0.0f;
    pdl_launch_dependents();
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
  for (int k = tid; k < kp; k += kNormThreads) {
    float y = 0.0f;
    if (k < H)
      y = __fmul_rn(bf16_bits_to_f32(bf16_scaled_rne(
                        __fmul_rn(__fmul_rn(bf16_bits_to_f32(x[k]), sc), bf16_bits_to_f32(a.final_norm_w[k])), rh, rl)),
                    xs);
    out[k] = static_cast<uint16_t>(f16x2_bits(y, 0.0f));
  }
  pdl_launch_dependents();
}

constexpr int kWarpsPerCta = 4;

__global__ void __launch_bounds__(kWarpsPerCta * 32) sweep_fp4_kernel(const Fp4SweepArgs a) {
  __shared__ ArgBest best[kWarpsPerCta][16];
  __shared__ int is_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int kp = fp4_padded(a.H);
  const int64_t V = a.V;
  for (int i = threadIdx.x; i < kWarpsPerCta * 16; i += blockDim.x) best[i >> 4][i & 15] = ArgBest{0.0f, -1};
  __syncthreads();
  pdl_wait_prior_grid();
  const uint16_t* xh = reinterpret_cast<const uint16_t*>(a.ws + kXhatOffset);
  const float* us = reinterpret_cast<const float*>(a.ws + kUnscaleOffset);
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + warp) * 16; r0 < V;
       r0 += static_cast<int64_t>(gridDim.x) * kWarpsPerCta * 16) {
    for (int n0 = 0; n0 < a.B; n0 += 8) {
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      fp4_dot_16x8(a.w.q, a.w.bs, r0, V, kp, xh + static_cast<size_t>(n0) * kp, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 2 * t4 + (i & 1);
        const int64_t row = r0 + g + 8 * (i >> 1);
        ArgBest c{0.0f, -1};
        if (n < a.B && row < V) {
          const float v = __fmul_rn(__fmul_rn(d[i], us[n]), a.w.rs[row]);
          if (a.logits != nullptr) a.logits[static_cast<int64_t>(n) * V + row] = v;
          arg_update(c, v, static_cast<int32_t>(row));
        }
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
          const float v = __shfl_xor_sync(0xffffffffu, c.v, m);
          const int32_t j = __shfl_xor_sync(0xffffffffu, c.i, m);
          if (j >= 0) arg_update(c, v, j);
        }
        if (g == 0 && n < a.B && c.i >= 0) arg_update(best[warp][n], c.v, c.i);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < a.B) {
    ArgBest c{0.0f, -1};
    for (int w = 0; w < kWarpsPerCta; ++w)
      if (best[w][threadIdx.x].i >= 0) arg_update(c, best[w][threadIdx.x].v, best[w][threadIdx.x].i);
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

}  // namespace

size_t fp4_sweep_workspace_bytes(int B, int H) {
  return kXhatOffset + static_cast<size_t>(B <= 8 ? 8 : 16) * fp4_padded(H) * 2;
}

cudaError_t launch_sweep_fp4(const Fp4SweepArgs& in, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t err = device_info(&di);
  if (err != cudaSuccess) return err;
  Fp4SweepArgs a = in;
  void* args[] = {&a};
  err = launch_pdl(reinterpret_cast<const void*>(fp4_xhat_kernel), dim3(a.B <= 8 ? 8 : 16), dim3(kNormThreads), 0,
                   stream, args);
  if (err != cudaSuccess) return err;
  int64_t grid = (static_cast<int64_t>(a.V) + kWarpsPerCta * 16 - 1) / (kWarpsPerCta * 16);
  if (grid > 4 * di.sm_count) grid = 4 * di.sm_count;
  return launch_pdl(reinterpret_cast<const void*>(sweep_fp4_kernel), dim3(static_cast<unsigned>(grid)),
                    dim3(kWarpsPerCta * 32), 0, stream, args);
}

}  // namespace mtp
