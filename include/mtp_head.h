/*
 * mtp_head.h -- C ABI of libmtphead.so, the GB300 (sm_103a) hot path of the GLM-5.3 MTP
 * speculative draft head (the `Glm5NextMtpHead::forward_one` draft step).
 *
 * What it computes, for each of B independent sequences b (the decoder layer between the two
 * stages is the identity here; the source pages: "metrale_model_arch / glm5next_mtp_head.rs",
 * module doc math summary and `forward_one`):
 *
 *   input stage   c_b    = [ enorm(embed[token_b, :]) | hnorm(target_hidden_b) ]   [2H] BF16
 *                 x_b    = bf16( eh_proj . c_b )                                     [H]  BF16
 *   output stage  xhat_b = shared_head.norm(x_b)                                     [H]  BF16
 *                 logit_b[v] = lm_head[v, :] . xhat_b   (BF16 head, or the FP8 E4M3 copy
 *                              with per-row scale: s[v] * sum_k e4m3(Q[v, k]) * xhat_b[k])
 *                 draft_b = lowest v with logit_b[v] == max_u logit_b[u]
 *
 *   norm(x; w) = rms_norm_vanilla = bf16( x * w / sqrt(mean(x^2) + eps) )  -- never 1 + w
 *   ("metrale_model_arch / glm5next_layer / mod.rs", module doc invariant).
 *
 * Conventions for every entry point
 *   - Pointers are DEVICE pointers unless the argument says "host". The caller owns every
 *     buffer (weights, activations, outputs, workspace). The library allocates nothing and
 *     keeps no state beyond cached device attributes, with two stated exceptions: the pinned
 *     staging buffers and recorded graphs of mtp_head_forward_host, and the fixed workspace
 *     array of mtp_head_logits_argmax_batched_noalloc.
 *   - BF16 values are passed as uint16_t bit patterns, FP8 E4M3 codes as uint8_t (OCP E4M3
 *     "fn": bias 7, subnormals, max 448, no infinities). All matrices are row-major and dense.
 *   - Base pointers of matrices and vectors must be 16-byte aligned (every cudaMalloc /
 *     PyTorch allocation is); int32/float pointers 4-byte aligned. Misalignment returns
 *     MTP_ERR_ALIGN before anything is launched.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) and the
 *     call returns without waiting, except mtp_head_forward_host, which is synchronous.
 *   - The return value reports host-checkable errors (arguments, shapes, alignment,
 *     workspace size) and launch failures (MTP_ERR_CUDA). Nothing is launched when it is not
 *     MTP_OK. Data-dependent errors (a token outside [0, V), a NaN/Inf weight handed to the
 *     quantiser, a kernel-side wait that gave up) are written by the kernels to the optional
 *     device word `status`: the first error stored wins; the caller zeroes it and reads it
 *     after synchronising. The library never clears it.
 *   - Shapes: 1 <= B <= 16, 1 <= H <= 65536, 1 <= V < 2^31, eps finite and >= 0.
 *   - Programmatic dependent launch: the input stage and the output stage are launched so that
 *     they may start streaming their weight matrix (eh_proj / lm_head) before the previous
 *     kernel on the stream has finished; the FP4 output stage and the FP4 linear do so with their
 *     copies. They read tokens, target_hidden, x, the norm weights
 *     and the workspace only after it has finished. Do not write those weight matrices in
 *     a kernel that itself triggers early launch of its dependents.
 */
#ifndef MTP_HEAD_H
#define MTP_HEAD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MTP_OK = 0,
    MTP_ERR_ARG = -1,             /* null pointer, bad enum, eps not finite or negative */
    MTP_ERR_SHAPE = -2,           /* B, H or V outside the supported range */
    MTP_ERR_ALIGN = -3,           /* a pointer is not aligned as stated above */
    MTP_ERR_WORKSPACE = -4,       /* workspace NULL or smaller than mtp_head_workspace_bytes */
    MTP_ERR_CUDA = -5,            /* a CUDA runtime call or launch failed */
    MTP_ERR_NONFINITE = -6,       /* (device status) the quantiser met a NaN or Inf weight */
    MTP_ERR_TOKEN_RANGE = -7,     /* (device status) a token outside [0, V) */
    MTP_ERR_NOT_IMPLEMENTED = -8, /* shape combination without a kernel in this build */
    MTP_ERR_TIMEOUT = -9          /* (device status) a kernel-side wait ran out of time */
} mtp_status;

enum { MTP_W_BF16 = 0, MTP_W_FP8_E4M3 = 1 };

/* ------------------------------------------------------------------------------------------
 * Input stage ("glm5next_mtp_head.rs", `forward_one`: the embedding row read by pointer at
 * token*hidden, `norm` with enorm into concat[0:H] and hnorm into concat[H:2H], then the
 * `eh_proj` dense gemv with n = H, k = 2H). One fused kernel per call.
 *
 *   embed          [V, H]  BF16   token embedding table (row token_b is gathered)
 *   enorm_w        [H]     BF16   enorm weight
 *   hnorm_w        [H]     BF16   hnorm weight
 *   eh_proj        [H, 2H] BF16   projection; row n is output n, columns [0:H) meet the enorm
 *                                 half of the concat, [H:2H) the hnorm half
 *   tokens         [B]     int32  device-resident tokens (a graph replay or a draft chain
 *                                 can feed the previous draft straight back in)
 *   target_hidden  [B, H]  BF16   the target model's hidden state for each sequence
 *   x_out          [B, H]  BF16   output: the block input x
 *   status         [1]     int32  optional (may be NULL); MTP_ERR_TOKEN_RANGE if some token is
 *                                 outside [0, V): that sequence's x row is written as zeros and
 *                                 the embedding table is not read for it
 * ---------------------------------------------------------------------------------------- */
int mtp_head_input_batched(const uint16_t* embed, const uint16_t* enorm_w,
                           const uint16_t* hnorm_w, const uint16_t* eh_proj,
                           const int32_t* tokens, const uint16_t* target_hidden,
                           uint16_t* x_out, int32_t* status, int B, int H, int V, float eps,
                           void* stream);

/* Same, B = 1. */
int mtp_head_input(const uint16_t* embed, const uint16_t* enorm_w, const uint16_t* hnorm_w,
                   const uint16_t* eh_proj, const int32_t* token, const uint16_t* target_hidden,
                   uint16_t* x_out, int32_t* status, int H, int V, float eps, void* stream);

/* ------------------------------------------------------------------------------------------
 * Context-row input stage ("glm5next_mtp_head.rs", `rows_impl`: for every context row r, the
 * embedding row of tokens[r] and target_hidden row r go through enorm / hnorm, the concat and
 * eh_proj -- the input stage of `forward_one` per row; the source loops over the rows on the
 * host, here all R rows run at once).
 *
 *   embed, enorm_w, hnorm_w, eh_proj  as for mtp_head_input_batched
 *   tokens         [R]     int32  device-resident tokens; tokens[r] is the token row r pairs
 *                                 with (the source pairs hidden row r with the token after it,
 *                                 so a caller passes its token array shifted by one)
 *   target_hidden  [R, H]  BF16
 *   x_out          [R, H]  BF16   output; a row whose token is outside [0, V) is zeros and
 *                                 status (optional) gets MTP_ERR_TOKEN_RANGE
 *   workspace             device scratch of at least mtp_head_context_workspace_bytes(R, H)
 *                         bytes (no initialisation needed; may be NULL when R <= 16, in which
 *                         case the batched input stage normalises the rows in every CTA)
 *   R              1 .. 65536 rows
 *
 * With the workspace (and H a multiple of 32, R >= 2) two kernels run: the normalised concat of
 * every row into the workspace (the same correctly rounded BF16 values as the input stage), then
 * x = concat . eh_proj^T as a tiled GEMM on the tcgen05 tensor cores with FP32 accumulation --
 * the source's eh_proj precision, so x is the BF16 rounding of an FP32-accumulated sum -- plus,
 * when the GEMM splits its tiles along k, a kernel that adds their partial sums in k order.
 * R <= 16 without the workspace (or with H not a multiple of 32, or R = 1) runs the input stage
 * of mtp_head_input_batched instead. H must be a multiple of 32 for R > 16
 * (MTP_ERR_NOT_IMPLEMENTED otherwise).
 * ---------------------------------------------------------------------------------------- */
int mtp_head_context_rows(const uint16_t* embed, const uint16_t* enorm_w, const uint16_t* hnorm_w,
                          const uint16_t* eh_proj, const int32_t* tokens, const uint16_t* target_hidden,
                          uint16_t* x_out, int32_t* status, void* workspace, size_t workspace_bytes,
                          int R, int H, int V, float eps, void* stream);

/* Bytes of workspace mtp_head_context_rows needs for R rows (0 for invalid shapes). */
size_t mtp_head_context_workspace_bytes(int R, int H);

/* ------------------------------------------------------------------------------------------
 * Output stage ("glm5next_mtp_head.rs", `forward_one`: `shared_head.norm` in place, then the
 * `lm_head` dense gemv -- or `dense_gemv_fp8w` over the FP8 copy described in the `head_fp8`
 * doc -- then `argmax_bf16`; here the sweep covers the whole vocabulary on one GPU and the
 * argmax is fused into it). One sweep kernel per call, which reads lm_head once for all B
 * sequences; for B = 2..16 a small kernel before it sums the squares of x's rows (for the norm).
 *
 *   x              [B, H]  BF16   block output
 *   final_norm_w   [H]     BF16   shared_head.norm weight
 *   lm_head        [V, H]  BF16 (w_dtype MTP_W_BF16) or E4M3 codes (MTP_W_FP8_E4M3)
 *   row_scale      [V]     fp32   per-row scale of the FP8 copy; NULL for BF16
 *   logits         [B, V]  fp32   optional output (NULL = not stored). Kept in fp32, not BF16.
 *   draft          [B]     int32  output: lowest index of the maximum logit; NaN never wins;
 *                                 -1 if every logit of that sequence is NaN
 *   status         [1]     int32  optional (may be NULL); MTP_ERR_TIMEOUT on a kernel-side wait
 *   workspace             device scratch of at least mtp_head_workspace_bytes(B, H, V)
 *                         bytes, zero-filled once before its first use. The kernels return
 *                         its counters to zero themselves, so it stays valid across calls and
 *                         CUDA-graph replays. Two calls that may run at the same time
 *                         (different streams) need different workspaces.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_logits_argmax_batched(const uint16_t* x, const uint16_t* final_norm_w,
                                   const void* lm_head, const float* row_scale, int w_dtype,
                                   float* logits, int32_t* draft, int32_t* status,
                                   void* workspace, size_t workspace_bytes, int B, int H, int V,
                                   float eps, void* stream);

/* Same, B = 1. */
int mtp_head_logits_argmax(const uint16_t* x, const uint16_t* final_norm_w, const void* lm_head,
                           const float* row_scale, int w_dtype, float* logits, int32_t* draft,
                           int32_t* status, void* workspace, size_t workspace_bytes, int H,
                           int V, float eps, void* stream);

/* ------------------------------------------------------------------------------------------
 * Output stage over one vocabulary shard ("glm5next_mtp_head.rs": the vocab-shard geometry
 * `head_rank` / `head_v0` / `head_n` -- a rank sweeps rows [head_v0, head_v0 + head_n) of the
 * shared lm_head, and its FP8 copy covers that shard only -- and `forward_one`'s sharded branch
 * with its cross-rank pick). The same kernels as mtp_head_logits_argmax_batched, over the n rows
 * that start at global row v0:
 *
 *   lm_head_shard    [n, H]  BF16 or E4M3 codes: the shard's rows (row v0 of the full matrix;
 *                            16-byte aligned, as for the output stage)
 *   row_scale_shard  [n]     fp32 scales of those rows (FP8), NULL for BF16
 *   v0, n                    the shard's first global row and its row count; 0 <= v0,
 *                            1 <= n, v0 + n <= 2^31 - 1 (else MTP_ERR_SHAPE)
 *   logits           [B, n]  fp32, optional: the shard's logits (column j is global row v0 + j)
 *   pick             [B]     int64 output, 8-byte aligned: each sequence's exchange key of its
 *                            (max logit, lowest global index) over the shard -- see below
 *   draft            [B]     int32, optional: the shard's own draft as a global index
 *   x, final_norm_w, status, workspace, B, H, eps, stream   as for the output stage
 *
 * Exchange key. One int64 per sequence whose signed order is the argmax order: the larger FP32
 * value first, then the lower global index (-0 counts as +0). The pick over any set of shards is
 * therefore the plain maximum of their keys -- mtp_head_pick_combine on one GPU, or a MAX
 * all-reduce of the [B] keys between ranks -- exact and for any number of shards. The source
 * exchanges BF16 lanes (each rank's max logit and three base-256 digits of its index) through a
 * SUM all-reduce, because its all-reduce sums BF16 elements; with FP32 logits a BF16 lane would
 * round two close maxima to one value, so the key carries the FP32 value whole. A shard whose
 * logits are all NaN gives the empty key INT64_MIN, below every other key.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_logits_argmax_shard(const uint16_t* x, const uint16_t* final_norm_w,
                                 const void* lm_head_shard, const float* row_scale_shard,
                                 int w_dtype, int v0, int n, float* logits, int64_t* pick,
                                 int32_t* draft, int32_t* status, void* workspace,
                                 size_t workspace_bytes, int B, int H, float eps, void* stream);

/* The pick over R shards: picks [R, B] int64 (row r = shard r's keys, 8-byte aligned) ->
 * draft [B] int32 (the global index of the largest key; -1 when every key of that sequence is
 * empty) and value [B] fp32 (optional, may be NULL: the winning logit). One small kernel on
 * `stream`; 1 <= R <= 65536, 1 <= B <= 16. After a MAX all-reduce between ranks, R = 1 decodes. */
int mtp_head_pick_combine(const int64_t* picks, int R, int B, int32_t* draft, float* value,
                          void* stream);

/* The exchange key on the host (no GPU involved): the key of (value, global index), and its
 * index and value back. mtp_head_pick_key returns INT64_MIN for index < 0 or a NaN value;
 * mtp_head_pick_index returns -1 and mtp_head_pick_value NaN for that key. */
int64_t mtp_head_pick_key(float value, int32_t index);
int32_t mtp_head_pick_index(int64_t key);
float mtp_head_pick_value(int64_t key);

/* ------------------------------------------------------------------------------------------
 * Output stage without a caller-provided workspace. The source pages have no counterpart: this
 * entry point exists for callers of this library that cannot allocate device memory -- e.g. a
 * plug-in that only receives the buffers its host framework hands it and has no allocator of
 * its own, or a process whose device memory was all claimed up front by another allocator.
 * It computes exactly what mtp_head_logits_argmax_batched computes (same kernels, same
 * arguments minus workspace / workspace_bytes) and allocates nothing: the workspace is a fixed
 * device array inside the library, 2,304 bytes, enough for any batch (B <= 16);
 * every GPU that loads the library holds it until the process exits. B outside 1..16 returns
 * MTP_ERR_SHAPE before anything runs.
 *   - The first call on a device looks up that array's device address (once per device, with
 *     the device current). Make that first call before any stream capture on the device. The
 *     address is kept for the life of the process: after cudaDeviceReset (or any reset of the
 *     device's primary context) the library's device array is a new one and the kept address is
 *     stale, so do not call this entry point on a device after resetting it.
 *   - All calls share the one array. The call clears its counter on `stream` before launching,
 *     so it never depends on what a previous call left there, but calls that may run at the
 *     same time on the GPU (different streams, or different host threads) race on it: order
 *     them on one stream or use mtp_head_logits_argmax_batched with separate workspaces. The
 *     clearing is a memset between the preceding kernel and the sweep, so unlike the workspace
 *     entry point the sweep cannot start its weight stream before the preceding kernel ends.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_logits_argmax_batched_noalloc(const uint16_t* x, const uint16_t* final_norm_w,
                                           const void* lm_head, const float* row_scale,
                                           int w_dtype, float* logits, int32_t* draft,
                                           int32_t* status, int B, int H, int V, float eps,
                                           void* stream);

/* Bytes of workspace for the output stage and the whole-step entry points (no device query; 0
 * for invalid shapes): the output stage's part (the first 2304 bytes for any B, which must be
 * zero-filled once), then, 256-byte aligned, room for the context-row path's workspace of B rows
 * (mtp_head_context_workspace_bytes(B, H): concat, row flags and FP32 partial sums; no
 * initialisation needed). The output stage alone accepts any workspace of at least its own part.
 * mtp_head_forward_batched / _host given a workspace of the full size run the input stage of
 * 2..16 sequences at H a multiple of 32 through the context-row path (mtp_head_context_rows:
 * concat kernel + tcgen05 GEMM; x then carries the GEMM's FP32 accumulation); otherwise they run
 * the input stage of mtp_head_input_batched. */
size_t mtp_head_workspace_bytes(int B, int H, int V);

/* ------------------------------------------------------------------------------------------
 * Whole draft step, device buffers: the input stage into x, then the output stage from x.
 * Exactly mtp_head_input_batched followed by mtp_head_logits_argmax_batched on one stream.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_forward_batched(const uint16_t* embed, const uint16_t* enorm_w,
                             const uint16_t* hnorm_w, const uint16_t* eh_proj,
                             const uint16_t* final_norm_w, const void* lm_head,
                             const float* row_scale, int w_dtype, const int32_t* tokens,
                             const uint16_t* target_hidden, uint16_t* x, float* logits,
                             int32_t* draft, int32_t* status, void* workspace,
                             size_t workspace_bytes, int B, int H, int V, float eps,
                             void* stream);

/* ------------------------------------------------------------------------------------------
 * Whole draft step from HOST buffers, synchronous: the shape of the source's
 * `forward_one(token, hidden_in, ...) -> u32`, which synchronises and copies the draft to the
 * host. Copies tokens_host [B] and hidden_host [B, H] into the caller's device buffers
 * tokens_dev / hidden_dev, runs mtp_head_forward_batched, copies draft back into
 * draft_host [B] and waits for the stream. Host buffers should be pinned for asynchronous
 * copies. The device `status` word, if given, is read back too and returned when nonzero.
 *
 * On a stream other than the legacy default stream (and not under the caller's own capture),
 * the first call for a given set of device buffers, shapes, eps and stream runs operation by
 * operation and then records the step in a CUDA graph around small mapped pinned staging
 * buffers (held by the library, at most 8 such steps, least recently used replaced). Later calls
 * with the same set copy the host inputs into the staging buffers, launch the graph once, wait,
 * and copy the draft out: the same work, without a launch per operation. Inside the graph the
 * moves between the staging buffers and tokens_dev / hidden_dev / draft_dev are small kernels
 * on the mapped memory (when B * H is a multiple of 8; copy operations otherwise). The host buffers may
 * differ from call to call. Calls from several threads are safe; calls sharing a recorded
 * step are serialised. On that recorded path the call returns as soon as the step's last kernel
 * has written the draft and status to the staging memory and set a completion word there (the
 * host polls it, asking the stream now and then so that a failed launch returns MTP_ERR_CUDA),
 * which spares the wake-up of a stream synchronisation; the stream may then still be retiring
 * that kernel, so work on another stream that must follow this step should wait on `stream`.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_forward_host(const uint16_t* embed, const uint16_t* enorm_w,
                          const uint16_t* hnorm_w, const uint16_t* eh_proj,
                          const uint16_t* final_norm_w, const void* lm_head,
                          const float* row_scale, int w_dtype,
                          const int32_t* tokens_host, const uint16_t* hidden_host,
                          int32_t* tokens_dev, uint16_t* hidden_dev, uint16_t* x_dev,
                          int32_t* draft_dev, int32_t* draft_host, int32_t* status,
                          void* workspace, size_t workspace_bytes, int B, int H, int V,
                          float eps, void* stream);

/* ------------------------------------------------------------------------------------------
 * The same step with the arguments that stay fixed from call to call gathered in one struct
 * (no counterpart on the source pages, like mtp_head_forward_host itself, whose shape is
 * `forward_one`'s). For a caller that makes the same draft step over and over through a costly
 * call boundary -- a language binding marshals 23 arguments per call, ~3 us from Python --
 * a step then passes four. The fields mean what the parameters of mtp_head_forward_host of the
 * same names mean; mtp_head_forward_host_args(a, tokens_host, hidden_host, draft_host) is
 * exactly mtp_head_forward_host(a->embed, ..., tokens_host, hidden_host, a->tokens_dev, ...,
 * draft_host, a->status, ..., a->stream): the same work, results and status codes, plus
 * MTP_ERR_ARG for a NULL `a`. The struct is read during the call only.
 * ---------------------------------------------------------------------------------------- */
typedef struct mtp_host_step_args {
  const uint16_t* embed;
  const uint16_t* enorm_w;
  const uint16_t* hnorm_w;
  const uint16_t* eh_proj;
  const uint16_t* final_norm_w;
  const void* lm_head;
  const float* row_scale;
  int w_dtype;
  int32_t* tokens_dev;
  uint16_t* hidden_dev;
  uint16_t* x_dev;
  int32_t* draft_dev;
  int32_t* status;
  void* workspace;
  size_t workspace_bytes;
  int B;
  int H;
  int V;
  float eps;
  void* stream;
} mtp_host_step_args;

int mtp_head_forward_host_args(const mtp_host_step_args* a, const int32_t* tokens_host,
                               const uint16_t* hidden_host, int32_t* draft_host);

/* ------------------------------------------------------------------------------------------
 * FP8 E4M3 copy of a [V, H] BF16 matrix ("glm5next_mtp_head.rs", `head_fp8` doc: an E4M3
 * copy of lm_head used for drafting only). Per row v:
 *   row_scale[v] = fp32( max_k |w[v, k]| / 448 )
 *   q[v, k]      = e4m3_rne_satfinite( fp32( w[v, k] / row_scale[v] ) )
 * An all-zero row gives scale 0 and zero codes. A NaN or Inf weight stores
 * MTP_ERR_NONFINITE in `status` (required here) and that row's codes and scale as zeros; the
 * copy must then not be used (the source's "quantisation fails" case).
 *   w [V, H] BF16 -> q [V, H] uint8 (E4M3 codes), row_scale [V] fp32
 * ---------------------------------------------------------------------------------------- */
int mtp_head_quantize_fp8(const uint16_t* w, uint8_t* q, float* row_scale, int32_t* status,
                          int V, int H, void* stream);

/* ------------------------------------------------------------------------------------------
 * FP4 copies ("glm5next_mtp_head.rs", `head_fp8` doc: a low-precision copy of lm_head used for
 * drafting only; the pages stop at FP8). A [V, H] BF16 matrix becomes three arrays, with
 * Hp = mtp_head_fp4_padded(H) (H rounded up to a multiple of 256):
 *
 *   q            [V, Hp/2]   uint8  E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; bit 3
 *                                   is the sign), column 2i in the low half of byte i
 *   block_scale  [V, Hp/16]  uint8  E4M3 scale of each 16 columns (non-negative)
 *   row_scale    [V]         fp32
 *
 *   row_scale[v]      = fp32( max_k |w[v, k]| / 2688 )                            (2688 = 6 * 448)
 *   block_scale[v, j] = e4m3( max_{k in block j} |w[v, k]| / (6 row_scale[v]) )
 *   q[v, k]           = e2m1( w[v, k] / (block_scale[v, k/16] row_scale[v]) )
 *
 * where e4m3 and e2m1 round the real quotient once, to nearest even, and saturate; columns from H
 * to Hp are zeros. An all-zero row (or one so small that row_scale rounds to 0) gives zeros, and so
 * does an all-zero block. A NaN or Inf weight stores MTP_ERR_NONFINITE in `status` (required here)
 * and makes that row zeros. 1 <= H <= 131072 (an eh_proj row of the longest head). q and
 * block_scale must be 16-byte aligned. In this and the next four calls an output or a workspace on an
 * input that is still read, or on another output, is MTP_ERR_ARG.
 * mtp_head_dequantize_fp4 writes the BF16 matrix that a copy stands for:
 *   w[v, k] = bf16( fp32( q * block_scale * row_scale ) ), w [V, H] BF16.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_fp4_padded(int H); /* 0 for H outside the range */

int mtp_head_quantize_fp4(const uint16_t* w, uint8_t* q, uint8_t* block_scale, float* row_scale,
                          int32_t* status, int V, int H, void* stream);

int mtp_head_dequantize_fp4(const uint8_t* q, const uint8_t* block_scale, const float* row_scale,
                            uint16_t* w, int V, int H, void* stream);

/* ------------------------------------------------------------------------------------------
 * Output stage over an FP4 copy of lm_head: mtp_head_logits_argmax_batched with
 *   logit_b[v] = row_scale[v] * sum_k block_scale[v, k/16] q[v, k] xhat_b[k],
 * xhat_b the BF16 output of shared_head.norm as there; the sum in fp32. logits (optional), draft,
 * status, B (1..16), H, V and eps as there. Two kernels: the normalised rows into the workspace,
 * then one sweep over the copy.
 *   workspace   device scratch of at least mtp_head_fp4_workspace_bytes(B, H, V) bytes, its first
 *               2304 bytes zero-filled once before its first use (the kernels leave them zero). Two
 *               calls that may run at the same time need different workspaces; one workspace serves
 *               every B up to the one it was sized for.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_logits_argmax_fp4(const uint16_t* x, const uint16_t* final_norm_w, const uint8_t* q,
                               const uint8_t* block_scale, const float* row_scale, float* logits,
                               int32_t* draft, int32_t* status, void* workspace,
                               size_t workspace_bytes, int B, int H, int V, float eps, void* stream);

size_t mtp_head_fp4_workspace_bytes(int B, int H, int V); /* 0 for invalid shapes */

/* ------------------------------------------------------------------------------------------
 * Rows of activations times an FP4 weight matrix, both operands in four bits. The rows of x are
 * quantised as by mtp_head_quantize_fp4 (into the workspace), then
 *   y[r, n] = bf16( sum_k value(Q(x))[r, k] * value(q)[n, k] ),   fp32 accumulation,
 * where value is code * block scale * row scale.
 *   x [R, K] BF16, q / block_scale / row_scale the FP4 copy of a [N, K] matrix, y [R, N] BF16
 *   status      optional: MTP_ERR_NONFINITE when a row of x holds a NaN or Inf (its y row is zeros)
 *   workspace   at least mtp_head_linear_fp4_workspace_bytes(R, N, K) bytes, no initialisation
 *               needed; calls that may run at the same time need different ones
 *   1 <= R <= 65536, 1 <= N, 1 <= K <= 131072; y may take the place of x
 * ---------------------------------------------------------------------------------------- */
int mtp_head_linear_fp4(const uint16_t* x, const uint8_t* q, const uint8_t* block_scale,
                        const float* row_scale, uint16_t* y, int32_t* status, void* workspace,
                        size_t workspace_bytes, int R, int N, int K, void* stream);

size_t mtp_head_linear_fp4_workspace_bytes(int R, int N, int K); /* 0 for invalid shapes */

/* Context-row input stage (mtp_head_context_rows) with an FP4 copy of eh_proj ([H, 2H]): the
 * normalised concat rows, then mtp_head_linear_fp4 over them. A row whose token is outside [0, V)
 * is zeros and status (optional) gets MTP_ERR_TOKEN_RANGE. 1 <= R <= 65536 rows (a draft step's
 * sequences or a prompt's rows alike); H a multiple of 8 (MTP_ERR_NOT_IMPLEMENTED otherwise). x_out
 * may take the place of target_hidden.
 * workspace: at least mtp_head_context_fp4_workspace_bytes(R, H) bytes, no initialisation. */
int mtp_head_context_rows_fp4(const uint16_t* embed, const uint16_t* enorm_w,
                              const uint16_t* hnorm_w, const uint8_t* eh_q,
                              const uint8_t* eh_block_scale, const float* eh_row_scale,
                              const int32_t* tokens, const uint16_t* target_hidden,
                              uint16_t* x_out, int32_t* status, void* workspace,
                              size_t workspace_bytes, int R, int H, int V, float eps,
                              void* stream);

size_t mtp_head_context_fp4_workspace_bytes(int R, int H); /* 0 for invalid shapes */

/* ------------------------------------------------------------------------------------------
 * Sampling: one token per row of logits from a given uniform random number (the source drafts
 * greedily, `argmax_bf16`; speculative decoding at a temperature needs drafts drawn from the
 * drafter's distribution, and that distribution for the acceptance).
 *
 *   logits       [R, ld]  fp32 (MTP_LOGITS_FP32) or BF16 (MTP_LOGITS_BF16); ld >= V elements
 *   temperature  [R] fp32  optional (NULL: 1); 0 takes the largest logit (lowest index of a tie)
 *   top_k        [R] int32 optional (NULL, <= 0 or >= V: off)
 *   top_p        [R] fp32  optional (NULL or >= 1: off)
 *   min_p        [R] fp32  optional (NULL or 0: off)
 *   u            [R] fp32  in [0, 1); may be NULL when only probs is asked for
 *   token        [R] int32 optional output
 *   prob         [R] fp32  optional output: the token's probability in the restricted distribution
 *   probs        [R, V] fp32 optional output: that distribution
 *   status       [1] int32 optional; MTP_ERR_ARG if a row's parameters are out of range
 *                (temperature negative or not finite, top_p negative or NaN, min_p outside [0, 1], u
 *                outside [0, 1)): that row's token is -1, its prob and probs are 0
 *
 * With m = max_i l_i: w_i = exp((l_i - m) / temperature), and 1 where l_i = m (several +Inf share
 * alike). NaN counts as -Inf; -Inf is never drawn; a row of nothing else gives token -1, prob and
 * probs 0 (no error). In the order (logit descending, index ascending) the tokens kept are a
 * prefix: the first top_k; of those, the ones whose preceding mass is less than top_p times the mass
 * of all of those; of those, the ones with l_i >= m + temperature * ln(min_p). At least one is
 * kept. The token is the lowest index whose cumulative kept mass, in index order, exceeds u times
 * the whole. Masses are summed in 64-bit fixed point: results do not vary from run to run, and the
 * roundings of a row's masses together stay below 2^-22 of its whole. (A distance m - l_i, or a
 * reciprocal of the temperature, beyond the fp32 range counts as infinite.)
 * 1 <= R <= 65536, 1 <= V < 2^31. No workspace. logits and probs need their elements' alignment only.
 * No output may overlap an input or another output (MTP_ERR_ARG), but token and prob may take the place
 * of a row parameter or of u.
 * ---------------------------------------------------------------------------------------- */
enum { MTP_LOGITS_FP32 = 0, MTP_LOGITS_BF16 = 1 };

int mtp_head_sample(const void* logits, int logits_dtype, int64_t ld, const float* temperature,
                    const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                    int32_t* token, float* prob, float* probs, int32_t* status, int R, int V,
                    void* stream);

/* ------------------------------------------------------------------------------------------
 * Acceptance of drafts by rejection sampling: the emitted tokens are distributed as if each had
 * been drawn from the target -- when the numbers in u are independent of the ones that drew the
 * drafts (with u[b, i] used for both, an accepted token comes up too often or too rarely).
 *
 *   target_probs  [B, D + 1, V] fp32  the target's distribution at each draft position and after
 *   draft_probs   [B, D, V]     fp32  the distributions that the drafts were drawn from; NULL for
 *                                     greedy drafts (each distribution is its token alone)
 *   draft_tokens  [B, D]        int32
 *   draft_len     [B]           int32 optional: drafts of each sequence, 0..D (NULL: D each)
 *   u             [B, D + 1]    fp32  uniform in [0, 1): u[b, i] decides draft i, u[b, D] draws the
 *                                     token after the accepted ones
 *   tokens        [B, D + 1]    int32 output: the accepted drafts, the drawn token, then -1
 *   accepted      [B]           int32 output: how many drafts were accepted
 *   prob          [B]           fp32  optional output: the drawn token's probability in the
 *                                     distribution that it was drawn from
 *   status        [1]           int32 optional; see below
 *
 * With n = draft_len[b], p_i = target_probs[b, i], q_i = draft_probs[b, i], x_i = draft_tokens[b, i]:
 * draft i is accepted while u_i q_i(x_i) < p_i(x_i). After a accepted drafts the next token comes from
 * max(p_a - q_a, 0) when a < n (from p_a itself if that has no mass), from p_n when all are
 * accepted: the lowest index whose cumulative mass exceeds u_D times the whole. Probabilities are
 * taken into [0, 1] (NaN as 0), for the acceptance too, and need not sum to one; a draft whose
 * q_i(x_i) is NaN is rejected. A distribution without mass gives token -1 and prob 0; any mass, down
 * to a subnormal number, is drawn from (the roundings of a row's masses together stay below 2^-22 of
 * its whole). A draft outside [0, V) that is reached is rejected (MTP_ERR_TOKEN_RANGE); a sequence
 * with draft_len outside 0..D, or u outside [0, 1) at any i < n or at D, gives accepted 0, tokens -1
 * and prob 0 (MTP_ERR_ARG).
 * 1 <= B <= 65536, 1 <= D <= 1024, 1 <= V < 2^31. No workspace. No output may overlap an input or
 * another output (MTP_ERR_ARG): accepted in the place of draft_len, for one, is refused.
 * ---------------------------------------------------------------------------------------- */
int mtp_head_verify(const float* target_probs, const float* draft_probs,
                    const int32_t* draft_tokens, const int32_t* draft_len, const float* u,
                    int32_t* tokens, int32_t* accepted, float* prob, int32_t* status, int B, int D,
                    int V, void* stream);

/* ------------------------------------------------------------------------------------------
 * Give-up time of the kernels' stage waits (no counterpart on the source pages, which have no
 * device-side waits: this library's kernels wait on shared-memory barriers for their weight
 * copies and for each other's stages, and every such wait is bounded so that a stalled copy can
 * never hang the GPU). Past the limit the kernel stores MTP_ERR_TIMEOUT in `status`, lets its own
 * copies in flight land, and returns; the draft and logits of that call are then undefined, and
 * the workspace is left ready for the next call. Default 2 s (2000000000 ns), far above any
 * real wait. The limit applies to the output-stage kernels (every batch size) and to the
 * single-sequence input stage, launched after this call (a CUDA graph keeps the limit it was
 * recorded with); the batched input stage, the context-row kernels and the FP4 linear always use 2 s, and so
 * does every wait for a kernel's own copies before it exits. Process-wide; returns the previous
 * limit. A short limit (a few ns: the device clock it is compared with advances about once a
 * microsecond) makes the waits that find their data missing run out; ns = 0 makes every stage
 * wait give up at once, whatever the data. Both put the error path within reach of a test.
 * ---------------------------------------------------------------------------------------- */
unsigned long long mtp_head_set_wait_limit_ns(unsigned long long ns);

/* Static description of a status code (never NULL). */
const char* mtp_head_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* MTP_HEAD_H */
