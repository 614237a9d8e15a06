// extern "C" entry points of the FP4 operators (declared and documented in include/mtp_head.h).
// Every argument is checked on the host before anything touches the GPU.
#include <cuda_runtime.h>
#include <stdint.h>

#include "checks.h"
#include "common.cuh"
#include "fp4.h"
#include "internal.h"

namespace {

using namespace mtp;

constexpr int kMaxRows = kMaxLinearRows;

bool bad_fp4(const uint8_t* q, const uint8_t* bs, const float* rs) {
  return !aligned(q, 16) || !aligned(bs, 16) || !aligned(rs, 4);
}

// The arrays of a copy of [rows, k].
struct CopySpans {
  Span q, bs, rs;
  CopySpans(const uint8_t* qp, const uint8_t* bp, const float* rp, int rows, int k)
      : q{qp, static_cast<size_t>(rows) * (fp4_padded(k) / 2)},
        bs{bp, static_cast<size_t>(rows) * (fp4_padded(k) / kFp4Block)},
        rs{rp, static_cast<size_t>(rows) * 4} {}
};
Span bf16_span(const uint16_t* p, int rows, int k) { return {p, static_cast<size_t>(rows) * k * 2}; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the context-row path: the concat [R, 2H] BF16, the row flags, then the linear's.
size_t context_head_bytes(int R, int H) {
  return round256(static_cast<size_t>(R) * 2 * H * 2) + round256(static_cast<size_t>(R) * 4);
}

}  // namespace

extern "C" {

int mtp_head_fp4_padded(int K) { return K < 1 || K > kMaxFp4K ? 0 : fp4_padded(K); }

int mtp_head_quantize_fp4(const uint16_t* w, uint8_t* q, uint8_t* block_scale, float* row_scale, int32_t* status,
                          int V, int H, void* stream) {
  if (!w || !q || !block_scale || !row_scale || !status) return MTP_ERR_ARG;
  if (V < 1 || H < 1 || H > kMaxFp4K) return MTP_ERR_SHAPE;
  if (!aligned(w, 16) || bad_fp4(q, block_scale, row_scale) || !aligned(status, 4)) return MTP_ERR_ALIGN;
  const CopySpans c(q, block_scale, row_scale, V, H);
  const Span outs[] = {c.q, c.bs, c.rs, {status, 4}}, ins[] = {bf16_span(w, V, H)};
  if (outputs_overlap(outs, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    return map_cuda(launch_fp4_quantize(w, q, block_scale, row_scale, status, nullptr, V, H,
                                        static_cast<cudaStream_t>(stream)));
  });
}

int mtp_head_dequantize_fp4(const uint8_t* q, const uint8_t* block_scale, const float* row_scale, uint16_t* w, int V,
                            int H, void* stream) {
  if (!w || !q || !block_scale || !row_scale) return MTP_ERR_ARG;
  if (V < 1 || H < 1 || H > kMaxFp4K) return MTP_ERR_SHAPE;
  if (!aligned(w, 16) || bad_fp4(q, block_scale, row_scale)) return MTP_ERR_ALIGN;
  const CopySpans c(q, block_scale, row_scale, V, H);
  const Span outs[] = {bf16_span(w, V, H)}, ins[] = {c.q, c.bs, c.rs};
  if (outputs_overlap(outs, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    return map_cuda(launch_fp4_dequantize(Fp4Matrix{q, block_scale, row_scale}, w, V, H,
                                          static_cast<cudaStream_t>(stream)));
  });
}

size_t mtp_head_fp4_workspace_bytes(int B, int H, int V) {
  if (B < 1 || B > kMaxB || H < 1 || H > kMaxH || V < 1) return 0;
  return fp4_sweep_workspace_bytes(B, H);
}

int mtp_head_logits_argmax_fp4(const uint16_t* x, const uint16_t* final_norm_w, const uint8_t* q,
                               const uint8_t* block_scale, const float* row_scale, float* logits, int32_t* draft,
                               int32_t* status, void* workspace, size_t workspace_bytes, int B, int H, int V,
                               float eps, void* stream) {
  if (!x || !final_norm_w || !q || !block_scale || !row_scale || !draft) return MTP_ERR_ARG;
  if (check_eps(eps) != MTP_OK) return MTP_ERR_ARG;
  if (B < 1 || B > kMaxB || H < 1 || H > kMaxH || V < 1) return MTP_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(final_norm_w, 16) || bad_fp4(q, block_scale, row_scale) ||
      (logits && !aligned(logits, 4)) || !aligned(draft, 4) || (status && !aligned(status, 4)) ||
      (workspace && !aligned(workspace, 16)))
    return MTP_ERR_ALIGN;
  if (!workspace || workspace_bytes < fp4_sweep_workspace_bytes(B, H)) return MTP_ERR_WORKSPACE;
  const CopySpans c(q, block_scale, row_scale, V, H);
  const Span ws[] = {{workspace, fp4_sweep_workspace_bytes(B, H)}};
  const Span outs[] = {{logits, static_cast<size_t>(B) * V * 4}, {draft, static_cast<size_t>(B) * 4}, {status, 4}, ws[0]};
  const Span copy[] = {c.q, c.bs, c.rs}, ins[] = {bf16_span(x, B, H), bf16_span(final_norm_w, 1, H)};
  if (outputs_overlap(outs, copy) || outputs_overlap(ws, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    Fp4SweepArgs a{x, final_norm_w, Fp4Matrix{q, block_scale, row_scale}, logits, draft, status,
                   static_cast<uint8_t*>(workspace), B, H, V, eps};
    return map_cuda(launch_sweep_fp4(a, static_cast<cudaStream_t>(stream)));
  });
}

size_t mtp_head_linear_fp4_workspace_bytes(int R, int N, int K) {
  if (R < 1 || R > kMaxRows || N < 1 || K < 1 || K > kMaxFp4K) return 0;
  return fp4_linear_workspace_bytes(R, N, K);
}

int mtp_head_linear_fp4(const uint16_t* x, const uint8_t* q, const uint8_t* block_scale, const float* row_scale,
                        uint16_t* y, int32_t* status, void* workspace, size_t workspace_bytes, int R, int N, int K,
                        void* stream) {
  if (!x || !q || !block_scale || !row_scale || !y) return MTP_ERR_ARG;
  if (R < 1 || R > kMaxRows || N < 1 || K < 1 || K > kMaxFp4K) return MTP_ERR_SHAPE;
  if (!aligned(x, 16) || bad_fp4(q, block_scale, row_scale) || !aligned(y, 16) || (status && !aligned(status, 4)) ||
      (workspace && !aligned(workspace, 16)))
    return MTP_ERR_ALIGN;
  if (!workspace || workspace_bytes < fp4_linear_workspace_bytes(R, N, K)) return MTP_ERR_WORKSPACE;
  const CopySpans c(q, block_scale, row_scale, N, K);
  const Span side[] = {{status, 4}, {workspace, fp4_linear_workspace_bytes(R, N, K)}};
  const Span outs[] = {bf16_span(y, R, N), side[0], side[1]}, copy[] = {c.q, c.bs, c.rs}, ins[] = {bf16_span(x, R, K)};
  // (y on x is fine: x has been quantised when the first row of y is written)
  if (outputs_overlap(outs, copy) || outputs_overlap(side, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    Fp4LinearArgs a{x, nullptr, Fp4Matrix{q, block_scale, row_scale}, y, status, static_cast<uint8_t*>(workspace),
                    R, N, K};
    return map_cuda(launch_linear_fp4(a, static_cast<cudaStream_t>(stream)));
  });
}

size_t mtp_head_context_fp4_workspace_bytes(int R, int H) {
  if (R < 1 || R > kMaxRows || H < 1 || H > kMaxH || H % 8 != 0) return 0;
  return context_head_bytes(R, H) + fp4_linear_workspace_bytes(R, H, 2 * H);
}

int mtp_head_context_rows_fp4(const uint16_t* embed, const uint16_t* enorm_w, const uint16_t* hnorm_w,
                              const uint8_t* eh_q, const uint8_t* eh_block_scale, const float* eh_row_scale,
                              const int32_t* tokens, const uint16_t* target_hidden, uint16_t* x_out, int32_t* status,
                              void* workspace, size_t workspace_bytes, int R, int H, int V, float eps, void* stream) {
  if (!embed || !enorm_w || !hnorm_w || !eh_q || !eh_block_scale || !eh_row_scale || !tokens || !target_hidden || !x_out)
    return MTP_ERR_ARG;
  if (check_eps(eps) != MTP_OK) return MTP_ERR_ARG;
  if (R < 1 || R > kMaxRows || H < 1 || H > kMaxH || V < 1) return MTP_ERR_SHAPE;
  if (!aligned(embed, 16) || !aligned(enorm_w, 16) || !aligned(hnorm_w, 16) ||
      bad_fp4(eh_q, eh_block_scale, eh_row_scale) || !aligned(tokens, 4) || !aligned(target_hidden, 16) ||
      !aligned(x_out, 16) || (status && !aligned(status, 4)) || (workspace && !aligned(workspace, 16)))
    return MTP_ERR_ALIGN;
  if (H % 8 != 0) return MTP_ERR_NOT_IMPLEMENTED;
  if (!workspace || workspace_bytes < mtp_head_context_fp4_workspace_bytes(R, H)) return MTP_ERR_WORKSPACE;
  {
    const CopySpans c(eh_q, eh_block_scale, eh_row_scale, H, 2 * H);
    const Span side[] = {{status, 4}, {workspace, mtp_head_context_fp4_workspace_bytes(R, H)}};
    const Span outs[] = {bf16_span(x_out, R, H), side[0], side[1]}, copy[] = {c.q, c.bs, c.rs};
    const Span ins[] = {bf16_span(embed, V, H), bf16_span(enorm_w, 1, H), bf16_span(hnorm_w, 1, H),
                        {tokens, static_cast<size_t>(R) * 4}, bf16_span(target_hidden, R, H)};
    // (x_out on target_hidden is fine: the concat rows are made when the first row of x_out is written)
    if (outputs_overlap(outs, copy) || outputs_overlap(side, ins)) return MTP_ERR_ARG;
  }
  return guarded([&] {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    ContextArgs c{};
    c.embed = embed;
    c.enorm_w = enorm_w;
    c.hnorm_w = hnorm_w;
    c.tokens = tokens;
    c.hidden = target_hidden;
    c.status = status;
    c.concat = reinterpret_cast<uint16_t*>(ws);
    c.valid = reinterpret_cast<int32_t*>(ws + round256(static_cast<size_t>(R) * 2 * H * 2));
    c.R = R;
    c.H = H;
    c.V = V;
    c.eps = eps;
    c.inv_h = 1.0 / static_cast<double>(H);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = launch_context_concat(c, st);
    if (err != cudaSuccess) return map_cuda(err);
    Fp4LinearArgs a{c.concat, c.valid, Fp4Matrix{eh_q, eh_block_scale, eh_row_scale}, x_out, status,
                    ws + context_head_bytes(R, H), R, H, 2 * H};
    return map_cuda(launch_linear_fp4(a, st));
  });
}

}  // extern "C"
