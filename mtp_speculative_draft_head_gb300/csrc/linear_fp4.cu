// Rows of activations times an FP4 weight matrix, both in four bits:
//   y[r, n] = bf16( rs_x[r] rs_w[n] sum_k (s_x code_x)[r, k] (s_w code_w)[n, k] )
// The rows of x are quantised on the way (fp4_quantize.cu) into the workspace.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "fp4_dot.cuh"
#include "internal.h"

namespace mtp {

namespace {

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct LinearWs {
  uint8_t* q;
  uint8_t* bs;
  float* rs;
  uint16_t* xh;
};
size_t bind(LinearWs* w, uint8_t* p, int R, int K) {
  const size_t kp = fp4_padded(K), rp = (static_cast<size_t>(R) + 7) / 8 * 8;
  uint8_t* p0 = p;
  w->q = p;
  p += round256(R * kp / 2);
  w->bs = p;
  p += round256(R * kp / 16);
  w->rs = reinterpret_cast<float*>(p);
  p += round256(static_cast<size_t>(R) * 4);
  w->xh = reinterpret_cast<uint16_t*>(p);
  p += rp * kp * 2;
  return static_cast<size_t>(p - p0);
}

// code * s of the quantised activations in f16 (exact); rows past R become zeros.
__global__ void __launch_bounds__(256) fp4_expand_kernel(const Fp4Matrix m, uint16_t* xh, int R, int rp, int kp) {
  const int64_t total = static_cast<int64_t>(rp) * (kp / 8);
  pdl_wait_prior_grid();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / (kp / 8);
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (row < R) {
      const uint32_t s2 = e4m3x2_to_f16x2(m.bs[i / 2] * 0x0101u);
      e2m1x8_to_f16x2x4(reinterpret_cast<const uint32_t*>(m.q)[i], v);
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = f16x2_mul(v[t], s2);
    }
    reinterpret_cast<uint4*>(xh)[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
  pdl_launch_dependents();
}

constexpr int kWarpsPerCta = 8;

__global__ void __launch_bounds__(kWarpsPerCta * 32) linear_fp4_kernel(const Fp4Matrix w, const uint16_t* xh,
                                                                       const float* rs_x, uint16_t* y, int R, int N,
                                                                       int kp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  pdl_wait_prior_grid();
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + warp) * 16;
  const int t0 = blockIdx.y * 8;
  if (r0 < N) {
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    fp4_dot_16x8(w.q, w.bs, r0, N, kp, xh + static_cast<size_t>(t0) * kp, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 2 * t4 + (i & 1);
      const int64_t n = r0 + g + 8 * (i >> 1);
      if (t < R && n < N)
        y[static_cast<int64_t>(t) * N + n] =
            static_cast<uint16_t>(bf16_bits_rn(__fmul_rn(__fmul_rn(d[i], w.rs[n]), rs_x[t])));
    }
  }
  pdl_launch_dependents();
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
  LinearWs w;
  bind(&w, a.ws, a.R, a.K);
  err = launch_fp4_quantize(a.x, w.q, w.bs, w.rs, a.status, a.valid, a.R, a.K, stream);
  if (err != cudaSuccess) return err;
  int kp = fp4_padded(a.K), R = a.R, N = a.N, rp = (a.R + 7) / 8 * 8;
  {
    Fp4Matrix m{w.q, w.bs, w.rs};
    void* args[] = {&m, &w.xh, &R, &rp, &kp};
    err = launch_pdl(reinterpret_cast<const void*>(fp4_expand_kernel), dim3(4 * di.sm_count), dim3(256), 0, stream, args);
    if (err != cudaSuccess) return err;
  }
  Fp4Matrix m = a.w;
  uint16_t* y = a.y;
  void* args[] = {&m, &w.xh, &w.rs, &y, &R, &N, &kp};
  return launch_pdl(reinterpret_cast<const void*>(linear_fp4_kernel),
                    dim3((N + kWarpsPerCta * 16 - 1) / (kWarpsPerCta * 16), rp / 8), dim3(kWarpsPerCta * 32), 0, stream,
                    args);
}

}  // namespace mtp
