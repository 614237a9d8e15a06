// extern "C" entry points of sampling and of the acceptance of drafts (declared and documented in
// include/mtp_head.h). Every argument is checked on the host before anything touches the GPU.
#include <cuda_runtime.h>
#include <stdint.h>

#include "checks.h"
#include "sample.h"

namespace {

using namespace mtp;

constexpr int kMaxRows = 65536;
constexpr int kMaxDrafts = 1024;

bool bad4(const void* p) { return p && !aligned(p, 4); }

}  // namespace

extern "C" {

int mtp_head_sample(const void* logits, int logits_dtype, int64_t ld, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, const float* u, int32_t* token, float* prob, float* probs,
                    int32_t* status, int R, int V, void* stream) {
  if (!logits || (!token && !prob && !probs) || ((token || prob) && !u)) return MTP_ERR_ARG;
  if (logits_dtype != MTP_LOGITS_FP32 && logits_dtype != MTP_LOGITS_BF16) return MTP_ERR_ARG;
  if (R < 1 || R > kMaxRows || V < 1 || ld < V) return MTP_ERR_SHAPE;
  if (!aligned(logits, logits_dtype == MTP_LOGITS_FP32 ? 4 : 2) || bad4(temperature) || bad4(top_k) || bad4(top_p) ||
      bad4(min_p) || bad4(u) || bad4(token) || bad4(prob) || bad4(probs) || bad4(status))
    return MTP_ERR_ALIGN;
  // The rows of logits are read more than once; a row's parameters by its own CTAs alone, before anything is written,
  // so token and prob may take exactly the place of one.
  const size_t item = logits_dtype == MTP_LOGITS_FP32 ? 4 : 2, r = static_cast<size_t>(R);
  const Span outs[] = {{token, r * 4}, {prob, r * 4}, {probs, r * V * 4}, {status, 4}};
  const Span row[] = {{logits, (static_cast<size_t>(R - 1) * ld + V) * item}};
  if (outputs_overlap(outs, row)) return MTP_ERR_ARG;
  for (const void* in : {static_cast<const void*>(temperature), static_cast<const void*>(top_k), static_cast<const void*>(top_p),
                         static_cast<const void*>(min_p), static_cast<const void*>(u)})
    for (const Span& o : outs)
      if ((o.p != in || o.bytes != r * 4 || o.p == status) && overlap(o.p, o.bytes, in, r * 4)) return MTP_ERR_ARG;
  return guarded([&] {
    SampleArgs a{logits, temperature, top_k, top_p, min_p, u, token, prob, probs, status, ld, R, V,
                 logits_dtype == MTP_LOGITS_BF16};
    return map_cuda(launch_sample(a, static_cast<cudaStream_t>(stream)));
  });
}

int mtp_head_verify(const float* target_probs, const float* draft_probs, const int32_t* draft_tokens,
                    const int32_t* draft_len, const float* u, int32_t* tokens, int32_t* accepted, float* prob,
                    int32_t* status, int B, int D, int V, void* stream) {
  if (!target_probs || !draft_tokens || !u || !tokens || !accepted) return MTP_ERR_ARG;
  if (B < 1 || B > kMaxRows || D < 1 || D > kMaxDrafts || V < 1) return MTP_ERR_SHAPE;
  if (!aligned(target_probs, 4) || bad4(draft_probs) || !aligned(draft_tokens, 4) || bad4(draft_len) ||
      !aligned(u, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) || bad4(prob) || bad4(status))
    return MTP_ERR_ALIGN;
  // (the CTAs of a sequence read its length, its numbers and its drafts in their own time: one that found another's
  // result in their place would take part in other exchanges than its peers)
  const size_t b = static_cast<size_t>(B), d = static_cast<size_t>(D), v = static_cast<size_t>(V);
  const Span outs[] = {{tokens, b * (d + 1) * 4}, {accepted, b * 4}, {prob, b * 4}, {status, 4}};
  const Span ins[] = {{target_probs, b * (d + 1) * v * 4}, {draft_probs, b * d * v * 4}, {draft_tokens, b * d * 4},
                      {draft_len, b * 4}, {u, b * (d + 1) * 4}};
  if (outputs_overlap(outs, ins)) return MTP_ERR_ARG;
  return guarded([&] {
    VerifyArgs a{target_probs, draft_probs, draft_tokens, draft_len, u, tokens, accepted, prob, status, B, D, V};
    return map_cuda(launch_verify(a, static_cast<cudaStream_t>(stream)));
  });
}

}  // extern "C"
