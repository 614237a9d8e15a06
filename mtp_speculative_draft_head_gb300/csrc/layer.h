// Host-side declarations of the operators of a draft layer's attention half (kernels in
// norm_residual.cu, cache_fp4.cu, attention_fp4.cu, attention_prompt.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mtp {

constexpr int kNormGroup = 128;  // columns that share a scale of the norm's 8-bit copy (or the whole row)

struct NormResidualArgs {
  const uint16_t* x;
  const uint16_t* delta;  // may be nullptr
  const uint16_t* w;
  uint16_t* total;        // may be nullptr
  uint16_t* y;            // may be nullptr
  uint8_t* q;             // may be nullptr
  float* q_scale;
  int32_t* status;
  int R, H, group;        // group: 0 (a scale per row) or kNormGroup
  float eps;
  double inv_h;
};
cudaError_t launch_norm_residual(const NormResidualArgs& a, cudaStream_t stream);

// The paged FP4 cache: pages of `page` tokens; of each page the keys, then the values, of every head.
//   q [pages, 2, heads, page, D / 2], bs [pages, 2, heads, page, D / 16], rs [pages, 2, heads, page]
// A row (a token's key or value of one head) is an FP4 row of D columns in the format of fp4.cuh.
struct CacheFp4 {
  uint8_t* q;
  uint8_t* bs;
  float* rs;
  int pages, page, heads, D;
};
inline bool cache_dim_ok(int D) { return D == 64 || D == 128; }
inline bool cache_page_ok(int page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }

struct CacheRowsArgs {
  CacheFp4 c;
  const uint16_t *k_in, *v_in;  // write
  uint16_t *k_out, *v_out;      // read
  int64_t ld_k, ld_v;           // elements from a row of k (v) to the next
  const int32_t* row_start;     // [B + 1]
  const int32_t* position;      // [B]
  const int32_t* table;         // [B, max_pages]
  int32_t* status;
  int T, B, max_pages;
};
cudaError_t launch_cache_write(const CacheRowsArgs& a, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t stream);

struct AttentionFp4Args {
  CacheFp4 c;
  const uint16_t* query;  // [B, Q, q_heads, D], a row's heads dense
  int64_t ld_q;           // elements from one (b, i) row to the next
  const int32_t* table;   // [B, max_pages]
  const int32_t* length;  // [B]
  const int32_t* rows;    // [B] or nullptr
  uint16_t* out;          // [B, Q, q_heads, D]
  int64_t ld_out;
  float* lse;             // [B, Q, q_heads] or nullptr
  int32_t* status;
  uint8_t* ws;
  size_t ws_bytes;
  int B, Q, q_heads, max_pages;
  float scale;
};
size_t attention_fp4_workspace_bytes(int B, int Q, int q_heads, int kv_heads, int D, int64_t max_len);
cudaError_t launch_attention_fp4(const AttentionFp4Args& a, cudaStream_t stream);

struct AttentionPromptArgs {
  const uint16_t *q, *k, *v;    // [T, heads, D], a row's heads dense
  int64_t ld_q, ld_k, ld_v;     // elements from a row to the next
  const int32_t* row_start;     // [B + 1]
  uint16_t* out;                // [T, q_heads, D]
  int64_t ld_out;
  float* lse;                   // [T, q_heads] or nullptr
  int32_t* status;
  int T, B, q_heads, kv_heads, D;
  float scale;
};
cudaError_t launch_attention_prompt(const AttentionPromptArgs& a, cudaStream_t stream);

}  // namespace mtp
