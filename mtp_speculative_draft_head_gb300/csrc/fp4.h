// Host-side declarations of the FP4 operators (kernels in fp4_quantize.cu, sweep_fp4.cu,
// linear_fp4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mtp {

constexpr int kFp4Block = 16;   // codes that share a block scale
constexpr int kFp4Row = 256;    // rows are padded to a multiple of this many codes
constexpr int kMaxH = 65536;    // longest head row
constexpr int kMaxFp4K = 2 * kMaxH;  // longest row of an FP4 copy (an eh_proj row of the longest head)
constexpr int kMaxLinearRows = 65536;

// Padded length of a row of k codes: whole 128-byte lines of codes and 16-byte pieces of scales,
// so that every row (and every tile of 256 codes) can be fetched by TMA whatever k is.
constexpr int fp4_padded(int k) { return (k + kFp4Row - 1) / kFp4Row * kFp4Row; }

// An FP4 copy of a [rows, k] matrix: codes [rows, fp4_padded(k) / 2] (the code of column 2i in the
// low half of byte i), block scales [rows, fp4_padded(k) / 16] (E4M3), row scales [rows].
struct Fp4Matrix {
  const uint8_t* q;
  const uint8_t* bs;
  const float* rs;
};

// w [rows, k] BF16 (row stride k) -> q, bs, rs. Rows whose valid flag (optional) is 0 become zeros.
// tile = 0: bs in the layout of a copy. tile > 0: in the order of the linear's operand, for tiles of
// `tile` rows -- per tile, per 128 rows of it (the last one may be partial), per 64 columns, 512
// bytes: scale i (0..3) of row r + 32 j (r < 32, j < 4) at 16 r + 4 j + i.
cudaError_t launch_fp4_quantize(const uint16_t* w, uint8_t* q, uint8_t* bs, float* rs, int32_t* status,
                                const int32_t* valid, int rows, int k, cudaStream_t stream, int tile = 0);
cudaError_t launch_fp4_dequantize(const Fp4Matrix& m, uint16_t* w, int rows, int k, cudaStream_t stream);

struct Fp4SweepArgs {
  const uint16_t* x;
  const uint16_t* final_norm_w;
  Fp4Matrix w;
  float* logits;  // may be nullptr
  int32_t* draft;
  int32_t* status;
  uint8_t* ws;
  int B, H, V;
  float eps;
};
size_t fp4_sweep_workspace_bytes(int B, int H);
cudaError_t launch_sweep_fp4(const Fp4SweepArgs& a, cudaStream_t stream);

struct Fp4LinearArgs {
  const uint16_t* x;      // [R, K] BF16
  const int32_t* valid;   // [R] optional: 0 makes that row of y zeros
  Fp4Matrix w;            // [N, K]
  uint16_t* y;            // [R, N] BF16
  int32_t* status;
  uint8_t* ws;
  int R, N, K;
};
size_t fp4_linear_workspace_bytes(int R, int N, int K);
cudaError_t launch_linear_fp4(const Fp4LinearArgs& a, cudaStream_t stream);

}  // namespace mtp
