// Host-side declarations of the sampling operators (sample.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mtp {

struct SampleArgs {
  const void* logits;        // [R, ld] fp32 or BF16
  const float* temperature;  // [R] or nullptr (1)
  const int32_t* top_k;      // [R] or nullptr (off)
  const float* top_p;        // [R] or nullptr (off)
  const float* min_p;        // [R] or nullptr (off)
  const float* u;            // [R]; nullptr only without token and prob
  int32_t* token;            // [R] or nullptr
  float* prob;               // [R] or nullptr
  float* probs;              // [R, V] or nullptr
  int32_t* status;
  int64_t ld;
  int R, V;
  bool bf16;
  int list_k;                // set by launch_sample
};
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream);

struct VerifyArgs {
  const float* target_probs;   // [B, D + 1, V]
  const float* draft_probs;    // [B, D, V] or nullptr (greedy drafts)
  const int32_t* draft_tokens; // [B, D]
  const int32_t* draft_len;    // [B] or nullptr (D)
  const float* u;              // [B, D + 1]
  int32_t* tokens;             // [B, D + 1]
  int32_t* accepted;           // [B]
  float* prob;                 // [B] or nullptr
  int32_t* status;
  int B, D, V;
};
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);

}  // namespace mtp
