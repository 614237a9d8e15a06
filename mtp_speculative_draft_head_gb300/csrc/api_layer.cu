// extern "C" entry points of the operators of a draft layer's attention half (declared and documented in
// include/mtp_head.h). Every argument is checked on the host before anything touches the GPU.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "checks.h"
#include "common.cuh"
#include "fp4.h"
#include "layer.h"

namespace {

using namespace mtp;

constexpr int kMaxRows = 65536;        // rows of the norm
constexpr int kMaxTokens = 1 << 22;    // packed rows
constexpr int kMaxSequences = 65536;
constexpr int kMaxHeads = 1024;
constexpr int kMaxQueryRows = 1024;    // of a sequence over the cache
constexpr int64_t kMaxLength = 1 << 30;

bool bad4(const void* p) { return p && !aligned(p, 4); }
// A row stride: dense heads fit, and rows start on 16-byte boundaries.
bool bad_ld(int64_t ld, int64_t row) { return ld < row || ld > (static_cast<int64_t>(1) << 40); }
size_t strided(int64_t rows, int64_t ld, int64_t row) { return (static_cast<size_t>(rows - 1) * ld + row) * 2; }
// With log2(e) and, over the cache, half of a query row's power of two (2^60 at most) it stays a number: an infinite factor
// would make NaN of scores that are zero.
constexpr float kMaxScale = 0x1p60f;
bool bad_scale(float s) { return !(s > 0.0f && s <= kMaxScale); }

int check_cache(const void* q, const void* bs, const void* rs, int heads, int D, int pages, int page, int max_pages) {
  if (!q || !bs || !rs) return MTP_ERR_ARG;
  if (heads < 1 || heads > kMaxHeads || pages < 1 || max_pages < 1 || !cache_page_ok(page) ||
      static_cast<int64_t>(max_pages) * page > kMaxLength)
    return MTP_ERR_SHAPE;
  if (D < 1) return MTP_ERR_SHAPE;
  if (!cache_dim_ok(D)) return MTP_ERR_NOT_IMPLEMENTED;
  if (!aligned(q, 16) || !aligned(bs, 16) || !aligned(rs, 16)) return MTP_ERR_ALIGN;
  return MTP_OK;
}
struct CacheSpans {
  Span q, bs, rs;
  CacheSpans(const void* qp, const void* bp, const void* rp, int heads, int D, int pages, int page) {
    const size_t rows = static_cast<size_t>(pages) * 2 * heads * page;
    q = {qp, rows * (D / 2)};
    bs = {bp, rows * (D / kFp4Block)};
    rs = {rp, rows * 4};
  }
};

int cache_rows(bool write, const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, const int32_t* row_start,
               const int32_t* position, const int32_t* block_table, uint8_t* q, uint8_t* bs, float* rs, int32_t* status,
               int T, int B, int heads, int D, int pages, int page, int max_pages, void* stream) {
  if (!k || !v || !row_start || !position || !block_table) return MTP_ERR_ARG;
  const int c = check_cache(q, bs, rs, heads, D, pages, page, max_pages);
  if (c != MTP_OK) return c;
  const int64_t row = static_cast<int64_t>(heads) * D;
  if (T < 1 || T > kMaxTokens || B < 1 || B > kMaxSequences || bad_ld(ld_k, row) || bad_ld(ld_v, row)) return MTP_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || ld_k % 8 != 0 || ld_v % 8 != 0 || bad4(row_start) || bad4(position) ||
      bad4(block_table) || bad4(status))
    return MTP_ERR_ALIGN;
  if (static_cast<int64_t>(T) * 2 * heads * (D / kFp4Block) > (static_cast<int64_t>(1) << 38)) return MTP_ERR_SHAPE;
  const CacheSpans cs(q, bs, rs, heads, D, pages, page);
  const size_t b = static_cast<size_t>(B);
  const Span rk{k, strided(T, ld_k, row)}, rv{v, strided(T, ld_v, row)};
  const Span ints[] = {{row_start, (b + 1) * 4}, {position, b * 4}, {block_table, b * max_pages * 4}};
  const Span st{status, 4};
  if (write) {
    const Span outs[] = {cs.q, cs.bs, cs.rs, st}, ins[] = {rk, rv, ints[0], ints[1], ints[2]};
    if (outputs_overlap(outs, ins)) return MTP_ERR_ARG;
  } else {
    // k and v of one projection's rows lie side by side: their spans interleave, their rows do not
    const bool side_by_side = ld_k == ld_v && ld_k >= 2 * row &&
                              (k < v ? v - k : k - v) >= row && (k < v ? v - k : k - v) <= ld_k - row;
    if (!side_by_side && overlap(rk.p, rk.bytes, rv.p, rv.bytes)) return MTP_ERR_ARG;
    const Span ins[] = {cs.q, cs.bs, cs.rs, ints[0], ints[1], ints[2]};
    const Span k_out[] = {rk, st}, v_out[] = {rv, st};
    if (outputs_overlap(k_out, ins) || outputs_overlap(v_out, ins)) return MTP_ERR_ARG;
  }
  return guarded([&] {
    CacheRowsArgs a{};
    a.c = CacheFp4{q, bs, rs, pages, page, heads, D};
    if (write) {
      a.k_in = k;
      a.v_in = v;
    } else {
      a.k_out = const_cast<uint16_t*>(k);
      a.v_out = const_cast<uint16_t*>(v);
    }
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.row_start = row_start;
    a.position = position;
    a.table = block_table;
    a.status = status;
    a.T = T;
    a.B = B;
    a.max_pages = max_pages;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return map_cuda(write ? launch_cache_write(a, st) : launch_cache_read(a, st));
  });
}

bool bad_attention(int B, int Q, int q_heads, int kv_heads, int64_t max_len) {
  if (B < 1 || B > kMaxSequences || Q < 1 || Q > kMaxQueryRows || kv_heads < 1 || kv_heads > kMaxHeads || q_heads < 1 ||
      q_heads > kMaxHeads || q_heads % kv_heads != 0 || max_len < 1 || max_len > kMaxLength)
    return true;
  // pieces of work, counted in 32 bits: rounds of 128 tokens for each (sequence, key head, 16 rows)
  const int64_t groups = (static_cast<int64_t>(Q) * (q_heads / kv_heads) + 15) / 16, rounds = (max_len + 127) / 128;
  const int64_t pairs = static_cast<int64_t>(B) * kv_heads * groups;
  return pairs > (1 << 23) || pairs * rounds > (static_cast<int64_t>(1) << 31);
}

}  // namespace

extern "C" {

int mtp_head_norm_residual(const uint16_t* x, const uint16_t* delta, const uint16_t* w, uint16_t* total, uint16_t* y,
                           uint8_t* q, float* q_scale, int32_t* status, int R, int H, int group, float eps,
                           void* stream) {
  if (!x || !w || (!total && !y && !q) || (q && (!q_scale || !status))) return MTP_ERR_ARG;
  if (check_eps(eps) != MTP_OK || (group != 0 && group != kNormGroup)) return MTP_ERR_ARG;
  if (R < 1 || R > kMaxRows || H < 1 || H > kMaxH) return MTP_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(w, 16) || (delta && !aligned(delta, 16)) || (total && !aligned(total, 16)) ||
      (y && !aligned(y, 16)) || (q && !aligned(q, 16)) || bad4(q_scale) || bad4(status))
    return MTP_ERR_ALIGN;
  const size_t n = static_cast<size_t>(R) * H;
  const size_t scales = static_cast<size_t>(R) * (group == 0 ? 1 : (H + group - 1) / group);
  const Span outs[] = {{total, n * 2}, {y, n * 2}, {q, n}, {q ? q_scale : nullptr, scales * 4}, {status, 4}};
  const Span ws[] = {{w, static_cast<size_t>(H) * 2}};
  if (outputs_overlap(outs, ws)) return MTP_ERR_ARG;
  // total and y may take exactly the place of x or delta: a row is read whole before it is written
  for (const uint16_t* in : {x, delta})
    for (const Span& o : outs) {
      const bool in_place = o.p == in && (o.p == total || o.p == y);
      if (!in_place && overlap(o.p, o.bytes, in, n * 2)) return MTP_ERR_ARG;
    }
  return guarded([&] {
    NormResidualArgs a{x, delta, w, total, y, q, q_scale, status, R, H, group, eps, 1.0 / static_cast<double>(H)};
    return map_cuda(launch_norm_residual(a, static_cast<cudaStream_t>(stream)));
  });
}

int mtp_head_cache_write_fp4(const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, const int32_t* row_start,
                             const int32_t* position, const int32_t* block_table, uint8_t* q, uint8_t* block_scale,
                             float* row_scale, int32_t* status, int T, int B, int heads, int D, int pages, int page,
                             int max_pages, void* stream) {
  return cache_rows(true, k, ld_k, v, ld_v, row_start, position, block_table, q, block_scale, row_scale, status, T, B,
                    heads, D, pages, page, max_pages, stream);
}

int mtp_head_cache_read_fp4(const uint8_t* q, const uint8_t* block_scale, const float* row_scale,
                            const int32_t* row_start, const int32_t* position, const int32_t* block_table, uint16_t* k,
                            int64_t ld_k, uint16_t* v, int64_t ld_v, int32_t* status, int T, int B, int heads, int D,
                            int pages, int page, int max_pages, void* stream) {
  return cache_rows(false, k, ld_k, v, ld_v, row_start, position, block_table, const_cast<uint8_t*>(q),
                    const_cast<uint8_t*>(block_scale), const_cast<float*>(row_scale), status, T, B, heads, D, pages, page,
                    max_pages, stream);
}

size_t mtp_head_attention_fp4_workspace_bytes(int B, int Q, int q_heads, int kv_heads, int D, int64_t max_len) {
  if (bad_attention(B, Q, q_heads, kv_heads, max_len) || !cache_dim_ok(D)) return 0;
  return attention_fp4_workspace_bytes(B, Q, q_heads, kv_heads, D, max_len);
}

int mtp_head_attention_fp4(const uint16_t* query, int64_t ld_q, const uint8_t* q, const uint8_t* block_scale,
                           const float* row_scale, const int32_t* block_table, const int32_t* length, const int32_t* rows,
                           uint16_t* out, int64_t ld_out, float* lse, int32_t* status, void* workspace,
                           size_t workspace_bytes, int B, int Q, int q_heads, int kv_heads, int D, int pages, int page,
                           int max_pages, float scale, void* stream) {
  if (!query || !block_table || !length || !out || bad_scale(scale)) return MTP_ERR_ARG;
  const int c = check_cache(q, block_scale, row_scale, kv_heads, D, pages, page, max_pages);
  if (c != MTP_OK) return c;
  const int64_t max_len = static_cast<int64_t>(max_pages) * page, row = static_cast<int64_t>(q_heads) * D;
  if (bad_attention(B, Q, q_heads, kv_heads, max_len) || bad_ld(ld_q, row) || bad_ld(ld_out, row)) return MTP_ERR_SHAPE;
  if (!aligned(query, 16) || ld_q % 8 != 0 || !aligned(out, 16) || ld_out % 8 != 0 || bad4(block_table) || bad4(length) ||
      bad4(rows) || bad4(lse) || bad4(status) || (workspace && !aligned(workspace, 16)))
    return MTP_ERR_ALIGN;
  const size_t need = attention_fp4_workspace_bytes(B, Q, q_heads, kv_heads, D, max_len);
  if (!workspace || workspace_bytes < need) return MTP_ERR_WORKSPACE;
  const CacheSpans cs(q, block_scale, row_scale, kv_heads, D, pages, page);
  const size_t b = static_cast<size_t>(B), n = b * Q;
  const Span outs[] = {{out, strided(static_cast<int64_t>(n), ld_out, row)}, {lse, n * q_heads * 4}, {status, 4}, {workspace, workspace_bytes}};
  const Span ins[] = {{query, strided(static_cast<int64_t>(n), ld_q, row)}, cs.q, cs.bs, cs.rs, {block_table, b * max_pages * 4},
                      {length, b * 4}, {rows, b * 4}};
  if (outputs_overlap(outs, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    AttentionFp4Args a{};
    a.c = CacheFp4{const_cast<uint8_t*>(q), const_cast<uint8_t*>(block_scale), const_cast<float*>(row_scale), pages, page,
                   kv_heads, D};
    a.query = query;
    a.ld_q = ld_q;
    a.table = block_table;
    a.length = length;
    a.rows = rows;
    a.out = out;
    a.ld_out = ld_out;
    a.lse = lse;
    a.status = status;
    a.ws = static_cast<uint8_t*>(workspace);
    a.ws_bytes = workspace_bytes;
    a.B = B;
    a.Q = Q;
    a.q_heads = q_heads;
    a.max_pages = max_pages;
    a.scale = scale;
    return map_cuda(launch_attention_fp4(a, static_cast<cudaStream_t>(stream)));
  });
}

int mtp_head_attention_prompt(const uint16_t* q, int64_t ld_q, const uint16_t* k, int64_t ld_k, const uint16_t* v,
                              int64_t ld_v, const int32_t* row_start, uint16_t* out, int64_t ld_out, float* lse,
                              int32_t* status, int T, int B, int q_heads, int kv_heads, int D, float scale,
                              void* stream) {
  if (!q || !k || !v || !row_start || !out || bad_scale(scale)) return MTP_ERR_ARG;
  if (T < 1 || T > kMaxTokens || B < 1 || B > kMaxSequences || kv_heads < 1 || kv_heads > kMaxHeads || q_heads < 1 ||
      q_heads > kMaxHeads || q_heads % kv_heads != 0 || D < 1)
    return MTP_ERR_SHAPE;
  if (!cache_dim_ok(D)) return MTP_ERR_NOT_IMPLEMENTED;
  const int64_t qr = static_cast<int64_t>(q_heads) * D, kr = static_cast<int64_t>(kv_heads) * D;
  if (bad_ld(ld_q, qr) || bad_ld(ld_k, kr) || bad_ld(ld_v, kr) || bad_ld(ld_out, qr)) return MTP_ERR_SHAPE;
  if (static_cast<int64_t>(T / 256 + B) * q_heads > 0x7FFFFFFF) return MTP_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || ld_q % 8 != 0 || ld_k % 8 != 0 ||
      ld_v % 8 != 0 || ld_out % 8 != 0 || bad4(row_start) || bad4(lse) || bad4(status))
    return MTP_ERR_ALIGN;
  const Span outs[] = {{out, strided(T, ld_out, qr)}, {lse, static_cast<size_t>(T) * q_heads * 4}, {status, 4}};
  const Span ins[] = {{q, strided(T, ld_q, qr)}, {k, strided(T, ld_k, kr)}, {v, strided(T, ld_v, kr)},
                      {row_start, (static_cast<size_t>(B) + 1) * 4}};
  if (outputs_overlap(outs, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    AttentionPromptArgs a{q, k, v, ld_q, ld_k, ld_v, row_start, out, ld_out, lse, status, T, B, q_heads, kv_heads, D, scale};
    return map_cuda(launch_attention_prompt(a, static_cast<cudaStream_t>(stream)));
  });
}

}  // extern "C"
