/*
 * qsmoe: the quantized sparse mixture-of-experts FFN layer of a
 * Qwen3.6-35B-A3B-style model, as a C ABI over hand-written CUDA kernels
 * for sm_103a (GB300).
 *
 * The layer, in the terms of the pages it follows:
 *   "Optimizing on-device inference for Apple Silicon" (Perplexity, 2026),
 *     section "Qwen creates three distinct workload shapes": a router scores
 *     256 experts per token and selects eight, next to a shared expert that
 *     processes every token;
 *     section "Keeping expert routing on the GPU": a histogram of the
 *     assignments per expert, a prefix scan into start offsets, a scatter
 *     of the rows into their expert groups and a block map of fixed-size
 *     row blocks, all without a host round trip;
 *     section "Dequantizing weights during matrix multiplication": 4-bit
 *     affine weights in groups of 64 with a scale and a bias, expanded on
 *     chip tile by tile, fp32 accumulation;
 *     section "Reducing intermediate and state traffic": the two input
 *     projections fused with their gated activation, and the output
 *     projection fused with its routing score and the shared expert;
 *   "oMLX MoE gate/up 融合优化：qwen35_moe_gate_up 实现剖析", section
 *     "融合原理": gate and up weights concatenated along the output axis in
 *     [gate, up] order, one quantized matmul, per-row bit-identical results;
 *   "Ember: packed Q8 decode" (voidwest.dev): the Q8_0 row format, 32 int8
 *     codes with one fp16 scale.
 *
 * Conventions (every entry point):
 *  - Pointers named in the argument lists are DEVICE pointers unless said
 *    otherwise; all arrays are dense row-major.  bf16 and fp16 values are
 *    passed as their 16-bit patterns (uint16_t).
 *  - The caller owns every buffer, including workspaces, and the stream.
 *    The library allocates nothing, never synchronises the stream and never
 *    reads device data on the host: every call only enqueues work on
 *    `stream` (stream-ordered, capturable into a CUDA graph).
 *  - The return value reports argument errors, found synchronously before
 *    anything is enqueued, and launch errors.  Problems only visible on the
 *    device (an expert id out of range, a non-finite logit, an fp16 operand
 *    out of range) are OR-ed into *dev_status as QSM_DEV_* bits; the kernels
 *    then skip the offending item and never trap.  *dev_status is never
 *    cleared by the library; the caller zeroes it and reads it after the
 *    stream has synchronised.
 *  - Pointers must be 16-byte aligned, except dev_status and logit_bias
 *    (4-byte).
 */
#ifndef QSMOE_H
#define QSMOE_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QSM_ABI_VERSION 4

#if defined(__GNUC__)
#define QSM_API __attribute__((visibility("default")))
#else
#define QSM_API
#endif

typedef enum {
  QSM_OK = 0,
  QSM_ERR_INVALID_ARGUMENT = 1, /* null / misaligned pointer, bad size */
  QSM_ERR_UNSUPPORTED = 2,      /* valid but not implemented (shape, type) */
  QSM_ERR_WORKSPACE_TOO_SMALL = 3,
  QSM_ERR_CUDA = 4              /* a CUDA launch or runtime call failed */
} qsm_status;

/* Bits of the device status word. */
#define QSM_DEV_BAD_EXPERT_ID 1 /* topk_idx entry outside [0, E) */
#define QSM_DEV_NONFINITE 2     /* non-finite router logit */
#define QSM_DEV_FP16_RANGE 4    /* a value staged in fp16 overflowed */
#define QSM_DEV_TIMEOUT 8       /* a bounded wait (on a copy, or on the
                                   tagged logits or h of
                                   moe_decode_layer) ran out: the kernel
                                   returned, its results are invalid */
#define QSM_DEV_BAD_ADAPTER_ID 16 /* an adapter id of n or more */

typedef enum { QSM_Q8_0 = 0, QSM_AFFINE4_G64 = 1 } qsm_qtype;

/* A quantized weight tensor of shape [experts, rows, cols], rows = outputs,
 * cols = inputs (reduction axis).
 *  QSM_Q8_0:        codes int8 [experts, rows, cols]; scales fp16
 *                   [experts, rows, cols/32]; weight = code * scale of its
 *                   block of 32 inputs.  biases must be NULL.
 *  QSM_AFFINE4_G64: codes uint32 [experts, rows, cols/8], input c stored in
 *                   bits 4*(c%8)..4*(c%8)+3 of word c/8; scales and biases
 *                   fp16 [experts, rows, cols/64]; weight = scale*code + bias
 *                   for its group of 64 inputs. */
typedef struct {
  int32_t qtype;
  int32_t experts, rows, cols;
  const void* codes;
  const uint16_t* scales;
  const uint16_t* biases;
} qsm_qweights;

/* One MoE FFN layer: hidden size H, expert (and shared expert) intermediate
 * size I, E routed experts of which each token uses k.
 *   gate_up        [E, 2I, H]  rows 0..I-1 gate, rows I..2I-1 up
 *   down           [E, H, I]
 *   shared_gate_up [1, 2I, H], shared_down [1, H, I]
 *   shared_gate    [H] fp32, or NULL: the shared expert's output of token t
 *                  is scaled by sigmoid(x[t] . shared_gate) (a gated shared
 *                  expert); NULL keeps weight 1 (the pages' shared expert).
 * All four tensors must share one qtype.  Requires H % 64 == 0,
 * I % 64 == 0, 1 <= k <= E <= 1024, shared_gate 16-byte aligned. */
typedef struct {
  int32_t H, I, E, k;
  qsm_qweights gate_up, down, shared_gate_up, shared_down;
  const float* shared_gate;
} qsm_moe_layer;

/* The token grouping produced by moe_group_tokens (all device arrays).
 * Assignment a = t*k + j is token t's j-th selected expert.
 *   counts   [E]     assignments per expert
 *   offsets  [E+1]   exclusive prefix sum of counts (offsets[E] = T*k when
 *                    every expert id is valid)
 *   perm     [T*k]   assignment at each sorted position, sorted by
 *                    (expert, assignment id): stable
 *   inv_perm [T*k]   sorted position of each assignment, -1 if its expert
 *                    id is invalid
 *   tile_map [2*max_tiles]  (expert, first sorted row) of every block of at
 *                    most tile_rows rows of one expert, experts ascending;
 *                    entries n_tiles .. max_tiles-1 are set to (-1, -1)
 *   n_tiles  [1]     number of blocks written (stays on the device)
 * tile_rows and max_tiles are host values chosen by the caller:
 * max_tiles >= moe_group_max_tiles(T, k, E, tile_rows), tile_rows as
 * returned by moe_ffn_tile_rows() when the grouping feeds moe_ffn_forward. */
typedef struct {
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv_perm;
  int32_t* tile_map;
  int32_t* n_tiles;
  int32_t tile_rows;
  int32_t max_tiles;
} qsm_grouping;

/* ----------------------------------------------------------------- router */

/* Bytes of workspace moe_route needs for T tokens, hidden size H and E
 * experts, whatever k is. */
QSM_API size_t moe_route_workspace_bytes(int32_t T, int32_t H, int32_t E);

/* Route flags (the `renormalize` argument of the routing calls). */
#define QSM_ROUTE_RENORMALIZE 1      /* weights: softmax over the selection */
#define QSM_ROUTE_BIAS_SELECT_ONLY 2 /* logit_bias picks experts, not weights */

/* Router: logits l[t,e] = sum_h x[t,h] * w_router[e,h] (fp32 accumulation)
 * and selection logits s[t,e] = l[t,e] + logit_bias[e]; per token the k
 * largest s (ties to the lower expert index) in descending order, and their
 * weights from w = s, or w = l with QSM_ROUTE_BIAS_SELECT_ONLY:
 *   QSM_ROUTE_RENORMALIZE set:   softmax of w over the k selected experts;
 *   QSM_ROUTE_RENORMALIZE clear: softmax of w over all E, at the selected.
 * (`renormalize` is these flags; 0 and 1 keep their old meaning.)
 * [Perplexity page, "Qwen creates three distinct workload shapes".]
 *   x          [T, H] bf16
 *   w_router   [E, H] fp32
 *   logit_bias [E] fp32 or NULL (added to the logits before selection)
 *   topk_idx   [T, k] int32 (out), topk_w [T, k] fp32 (out)
 *   workspace  >= moe_route_workspace_bytes(T, H, E) bytes.  It must hold
 *              zeros before its first use; every call leaves it fit for the
 *              next, of any T, E and k that it is large enough for.
 * Few tokens run on CUDA cores (fp32 FMA); many tokens (T > 64, E a multiple
 * of 16 up to 256, k <= 8) run one tcgen05 GEMM over an exact three-way
 * bf16 split of w_router, which keeps fp32-accurate logits.
 * Requires H % 64 == 0, 1 <= k <= min(E, 32), E <= 1024, T >= 0, no flag
 * bits beyond the two above.  A non-finite logit sets QSM_DEV_NONFINITE. */
QSM_API qsm_status moe_route(const uint16_t* x, const float* w_router,
                     const float* logit_bias, int32_t T, int32_t H, int32_t E,
                     int32_t k, int32_t renormalize, int32_t* topk_idx,
                     float* topk_w, void* workspace, size_t workspace_bytes,
                     int32_t* dev_status, cudaStream_t stream);

/* Scores of moe_route_scores: softmax over all experts, or a sigmoid of each. */
typedef enum { QSM_SCORE_SOFTMAX = 0, QSM_SCORE_SIGMOID = 1 } qsm_score;

/* A router by scores: H, E, k as a layer's;
 *   score  qsm_score
 *   groups, groups_kept, group_best  the experts lie in `groups` equal groups
 *       (e / (E / groups)); a group is worth the sum of its group_best (1 or 2)
 *       largest biased scores, the groups_kept best groups stay; 1, 1, 1: no groups
 *   renormalize  1: the weights are divided by their sum
 *   scale  factor of the weights, finite
 *   w_split  the weights as moe_router_split writes them (for this H and E)
 *   bias  [E] fp32 or NULL, added to the scores for the choice only.  -infinity
 *       closes an expert: it is taken after all others, with weight 0. */
typedef struct {
  int32_t H, E, k, score;
  int32_t groups, groups_kept, group_best, renormalize;
  float scale;
  const uint16_t* w_split;
  const float* bias;
} qsm_router;

/* Bytes of w_split (0: not supported), and the exact split of w_router [E, H]
 * fp32 into three bf16 parts, in the order that the kernel reads (once per weight).
 * H a multiple of 64, E <= 512; both 16-byte aligned, without a byte in common. */
QSM_API size_t moe_router_split_bytes(int32_t E, int32_t H);
QSM_API qsm_status moe_router_split(const float* w_router, int32_t E, int32_t H, uint16_t* w_split,
                                    cudaStream_t stream);

/* Routing by scores, for any number of tokens in one launch: logits l = x W^T
 * with fp32 accuracy, scores s = softmax(l) or sigmoid(l), biased scores
 * c = s + bias; of the kept groups' experts the k with the largest c (ties,
 * of groups too, to the lower index) in descending c, weighted with s.
 *   x [T, H] bf16, ldx elements from row to row (a multiple of 8, at least H);
 *   topk_idx [T, k] int32, topk_w [T, k] fp32 (out), as moe_group_tokens,
 *   moe_ffn_forward and moe_mx4_experts take them; they may overlap neither each
 *   other nor x, w_split or bias (QSM_ERR_INVALID_ARGUMENT).
 * Needs no workspace.  A logit that is not finite closes its expert, and so
 * does a bias of +infinity or NaN; either sets QSM_DEV_NONFINITE.  Where the taken
 * weights sum to 0 they are 0.  Scores are fp32 numbers: experts whose scores round to
 * the same one tie (a sigmoid is 1 from logits of 17 on, and 0 below -87).
 * Requires H % 64 == 0, E <= 512, k <= 32 and <= the kept groups' experts,
 * groups <= 32 dividing E. */
QSM_API qsm_status moe_route_scores(const qsm_router* r, const uint16_t* x, int64_t ldx, int32_t T,
                                    int32_t* topk_idx, float* topk_w, int32_t* dev_status,
                                    cudaStream_t stream);

/* --------------------------------------------------------------- grouping */

/* Upper bound on the number of blocks of tile_rows rows over any routing:
 * n + floor((T*k - n) / tile_rows) with n = min(E, T*k). */
QSM_API int32_t moe_group_max_tiles(int32_t T, int32_t k, int32_t E,
                            int32_t tile_rows);

/* Histogram, exclusive scan, stable scatter and block map of the
 * assignments [Perplexity page, "Keeping expert routing on the GPU"]; see
 * qsm_grouping for the outputs.  An expert id outside [0, E) sets
 * QSM_DEV_BAD_EXPERT_ID; that assignment is left out of every group
 * (inv_perm = -1) and the FFN skips it.
 * Requires 1 <= k, E <= 1024, tile_rows >= 1, T*k <= 2^24. */
QSM_API qsm_status moe_group_tokens(const int32_t* topk_idx, int32_t T, int32_t k,
                            int32_t E, const qsm_grouping* g,
                            int32_t* dev_status, cudaStream_t stream);

/* moe_route followed by moe_group_tokens in one launch, for a few tokens
 * (decode): topk_idx, topk_w and every array of g are the same bits as the
 * two calls give.  The router's CTAs split the experts as in moe_route; the
 * CTA that finishes last selects the top k and then builds the grouping of
 * the T*k assignments from the ids it holds in shared memory
 * [Perplexity page, "Qwen creates three distinct workload shapes" and
 * "Keeping expert routing on the GPU"].
 *   workspace  as for moe_route (moe_route_workspace_bytes(T, H, E)).
 * Supported: 1 <= T <= 8, H % 64 == 0, 1 <= E <= 256, 1 <= k <= min(E, 32);
 * otherwise returns QSM_ERR_UNSUPPORTED and enqueues nothing (use the two
 * calls).  Argument errors as for the two calls. */
QSM_API qsm_status moe_route_group(const uint16_t* x, const float* w_router,
                                   const float* logit_bias, int32_t T, int32_t H,
                                   int32_t E, int32_t k, int32_t renormalize,
                                   int32_t* topk_idx, float* topk_w,
                                   const qsm_grouping* g, void* workspace,
                                   size_t workspace_bytes, int32_t* dev_status,
                                   cudaStream_t stream);

/* -------------------------------------------------------------------- FFN */

/* The tile_rows moe_ffn_forward expects in its grouping for T tokens. */
QSM_API int32_t moe_ffn_tile_rows(int32_t T);

/* Bytes of workspace moe_ffn_forward needs for layer L and T tokens. */
QSM_API size_t moe_ffn_workspace_bytes(const qsm_moe_layer* L, int32_t T);

/* The expert FFNs and the combine:
 *   for every assignment (t, j) with expert e = topk_idx[t, j]:
 *     gu = W_gate_up[e] x[t]            (one fused quantized matmul)
 *     h  = silu(gu[:I]) * gu[I:]        (SwiGLU, silu(g) = g / (1 + e^-g))
 *     o  = W_down[e] h
 *   the same for the shared expert, then
 *     y[t] = sum_j topk_w[t, j] * o(t, j) + o_shared(t)
 * [Perplexity page, "Reducing intermediate and state traffic"; oMLX page,
 * "融合原理" and "前向传播补丁"].
 *   x          [T, H] bf16;  y [T, H] bf16 (out, round-to-nearest-even of
 *              the fp32 result);  y_f32 [T, H] fp32 (out, optional: the
 *              same result before rounding, for parity checks) or NULL
 *   topk_idx, topk_w  as written by moe_route;  g as written by
 *              moe_group_tokens for the same topk_idx, with tile_rows ==
 *              moe_ffn_tile_rows(T)
 *   workspace  >= moe_ffn_workspace_bytes(L, T) bytes, no initial content.
 * T <= 64 runs the decode kernels (weight streaming GEMV), larger T the
 * grouped-GEMM prefill kernels (tcgen05, weights of either type expanded to
 * fp16 tile by tile on chip; they need H % 256 == 0 and I % 128 == 0, else
 * QSM_ERR_UNSUPPORTED). */
QSM_API qsm_status moe_ffn_forward(const qsm_moe_layer* L, const uint16_t* x,
                           int32_t T, const int32_t* topk_idx,
                           const float* topk_w, const qsm_grouping* g,
                           uint16_t* y, float* y_f32, void* workspace,
                           size_t workspace_bytes, int32_t* dev_status,
                           cudaStream_t stream);

/* ------------------------------------------------------------ whole layer */

/* Bytes of workspace moe_layer_forward needs for T tokens in chunks of at
 * most `chunk` tokens (sized for one chunk: the router's, the grouping's
 * and the FFN's workspaces of the largest chunk).  0 if the layer is
 * unsupported or an argument is invalid. */
QSM_API size_t moe_layer_workspace_bytes(const qsm_moe_layer* L, int32_t T,
                                         int32_t chunk);

/* The whole layer: moe_route -> moe_group_tokens -> moe_ffn_forward over the
 * tokens in consecutive chunks of at most `chunk` tokens, all enqueued on
 * `stream` [Perplexity page, "Qwen creates three distinct workload shapes"
 * (long prompts in chunks) and "Keeping expert routing on the GPU"].  A
 * token's routing does not depend on the chunking; its output differs
 * between chunkings at most by the order of the prefill combine's fp32
 * additions (or by the decode / prefill kernel choice of its chunk's size).
 *   x [T, H] bf16;  w_router [E, H] fp32;  logit_bias [E] fp32 or NULL;
 *   topk_idx [T, k] int32 and topk_w [T, k] fp32 (out);  y [T, H] bf16 (out);
 *   y_f32 [T, H] fp32 (out) or NULL;
 *   workspace  >= moe_layer_workspace_bytes(L, T, chunk) bytes; it must hold
 *              zeros before its first use, and every call leaves it so.
 * Errors as for the three calls. */
QSM_API qsm_status moe_layer_forward(const qsm_moe_layer* L, const uint16_t* x,
                                     int32_t T, int32_t chunk,
                                     const float* w_router,
                                     const float* logit_bias, int32_t renormalize,
                                     int32_t* topk_idx, float* topk_w,
                                     uint16_t* y, float* y_f32, void* workspace,
                                     size_t workspace_bytes, int32_t* dev_status,
                                     cudaStream_t stream);

/* The whole layer for a few tokens (1 <= T <= 8) in one launch: router,
 * selection, gate_up + SwiGLU, down + combine, separated by grid-wide
 * exchanges of call-tagged words (the logits, then h between gate_up and
 * down), instead of three dependent launches
 * [Perplexity page, "Keeping expert routing on the GPU", "Reducing
 * intermediate and state traffic", "Overlapping independent GPU work"].  Results: topk_idx and topk_w
 * bit-identical to moe_route's; y the layer output as moe_ffn_forward
 * computes it (same arithmetic per product; the combine's fp32 additions in
 * another order).
 *   Arguments as for moe_layer_forward, without a chunk size.
 *   Supported: Q8_0 or affine-4 (all four weight planes alike), H % 256 ==
 *   0, H / 16 <= the device's SM count (a CTA per SM, at least one per 16
 *   output rows, all resident for the two exchanges),
 *   I % 128 == 0 (Q8_0) or % 256 == 0
 *   (affine-4), E <= 1024, k <= 32; all pointers 16-byte aligned except
 *   topk_idx, topk_w, y, y_f32 and logit_bias (4 bytes).  Otherwise
 *   QSM_ERR_UNSUPPORTED (moe_layer_forward serves every shape).
 *   workspace  >= moe_decode_layer_workspace_bytes(L, T) bytes, zeros before
 *              its first use.  Its first 8 bytes count calls (one arrival
 *              per CTA): the calls that share a workspace must have the
 *              same layer shape (H, I, E, k), and after a
 *              QSM_DEV_TIMEOUT it must be zeroed again.
 *              From byte 256: the tagged logits [8, E] (64-bit words, the
 *              call's tag in the high half), then h as 64-bit words (tag,
 *              two fp16 values).
 * Every wait in the kernel is bounded: an exchange or copy that
 * does not complete sets QSM_DEV_TIMEOUT and the call's results are
 * invalid. */
QSM_API size_t moe_decode_layer_workspace_bytes(const qsm_moe_layer* L, int32_t T);

/* The check moe_decode_layer makes before it launches, with the device's
 * figures passed in: 1 when the layer and T are supported on a device of
 * `sm_count` SMs and the kernel's whole grid (one CTA per SM, at least one
 * per 16 rows of y) can be resident at once with `blocks_per_sm` CTAs per
 * SM, else 0.  moe_decode_layer takes sm_count from the current device and
 * blocks_per_sm from the occupancy calculator at the call's shared-memory
 * size; when the check fails it returns QSM_ERR_UNSUPPORTED (and
 * moe_decode_layer_workspace_bytes returns 0), so that callers take the
 * route / group / FFN launches instead.  The check cannot see SMs that other
 * work holds while the kernel runs (another stream, MPS limits): there the
 * bounded waits run out and the call reports QSM_DEV_TIMEOUT with invalid
 * results.  Pure host logic; needs no GPU. */
QSM_API int32_t qsm_decode_layer_fits(const qsm_moe_layer* L, int32_t T, int32_t sm_count,
                                      int32_t blocks_per_sm);
QSM_API qsm_status moe_decode_layer(const qsm_moe_layer* L, const uint16_t* x, int32_t T,
                                    const float* w_router, const float* logit_bias,
                                    int32_t flags, int32_t* topk_idx, float* topk_w,
                                    uint16_t* y, float* y_f32, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_status,
                                    cudaStream_t stream);

/* moe_ffn_forward without a workspace argument, for callers that cannot
 * allocate device memory (code running inside another runtime's memory
 * pool, latency-critical threads where an allocation and the device
 * synchronisation it may cause are not allowed, hosts that own only the
 * activations and the stream).  The pages have no counterpart: this is an
 * interface convenience of this library, not a step of the method.
 *   Arguments and results are those of moe_ffn_forward.  The scratch comes
 *   from an array inside the library (1 MiB per device, held by every GPU
 *   that loads the library until the process exits), so T must be <= 64 and
 *   the scratch that moe_ffn_forward would need for this call
 *   (moe_ffn_workspace_bytes(L, T) on the path in force: the decode path's
 *   h, (T*k + T) * I * 2 bytes, and T fp32 shared-expert gates) must fit in
 *   1 MiB; otherwise QSM_ERR_UNSUPPORTED is returned and nothing is
 *   enqueued.  T < 0 is QSM_ERR_INVALID_ARGUMENT; T == 0 enqueues nothing.
 *   The call allocates nothing.  `stream` must belong to the current
 *   device (else QSM_ERR_INVALID_ARGUMENT): the scratch used is that
 *   device's copy.  The first call on each device looks up that device's
 *   copy of the array; make that first call before any stream capture.  The
 *   address found stays in use for the life of the device's context: calls
 *   after cudaDeviceReset are not supported.  All calls on a device share
 *   the one array and it keeps the last call's contents (no value has to
 *   start at zero); calls whose work overlaps on the GPU (different
 *   streams, or different threads without ordering) race on it and must be
 *   serialised by the caller. */
QSM_API qsm_status moe_ffn_forward_noalloc(const qsm_moe_layer* L,
                                           const uint16_t* x, int32_t T,
                                           const int32_t* topk_idx,
                                           const float* topk_w,
                                           const qsm_grouping* g, uint16_t* y,
                                           float* y_f32, int32_t* dev_status,
                                           cudaStream_t stream);

/* ------------------------------------------------------------ dense GEMV */

/* Batch-1 Q8_0 projection y[n] = sum_c q[n,c] * d[n, c/32] * x[c]
 * [Perplexity page, "Optimizing the single-row weight path"; Ember page,
 * Q8_0 rows].
 *   x [K] bf16;  q [N, K] int8;  d [N, K/32] fp16;  y [N] bf16 (out).
 * Requires K % 64 == 0, 64 <= K <= 16384, N >= 1; x, q, d, y 16-byte
 * aligned.  With K % 256 == 0 the weight tiles arrive by TMA copies whose
 * waits are bounded: a copy that never completes sets QSM_DEV_TIMEOUT in
 * *dev_status (which may be NULL: nothing is reported then).  A row's
 * result does not depend on N (K is summed in fixed 512-wide segments, in
 * segment order). */
QSM_API qsm_status q8_gemv(const uint16_t* x, const int8_t* q, const uint16_t* d,
                   int32_t N, int32_t K, uint16_t* y, int32_t* dev_status,
                   cudaStream_t stream);

/* Int8-activation mode of the Q8_0 GEMV ["Ember: packed Q8 decode": the
 * projections that read one activation share its quantization, and the dot
 * products run on 8-bit groups].  Reading: blocks of 32 inputs, per block
 * an fp32 scale dx = max|x| / 127 and codes qx = round-half-away(x / dx)
 * clamped to [-127, 127] (fp32 arithmetic; an all-zero block has dx = 0).
 *   q8_quantize_x:  x [K] bf16 -> qx [K] int8 (out), dx [K/32] fp32 (out);
 *                   K % 32 == 0.
 *   q8_gemv_i8:     y[n] = sum_b d[n,b] * dx[b] * sum_{c in b} q[n,c] * qx[c]
 *                   (each block's integer dot product exact, the rest fp32),
 *                   y [N] bf16 (out); N >= 1, K % 64 == 0, K <= 16384, qx,
 *                   q, d, y 16-byte aligned.  A row's result does not depend
 *                   on N.
 * This changes the numerics against q8_gemv by the activation's rounding
 * (at most half a step dx/2 per input). */
QSM_API qsm_status q8_quantize_x(const uint16_t* x, int32_t K, int8_t* qx, float* dx,
                                 int32_t* dev_status, cudaStream_t stream);
QSM_API qsm_status q8_gemv_i8(const int8_t* qx, const float* dx, const int8_t* q,
                              const uint16_t* d, int32_t N, int32_t K, uint16_t* y,
                              int32_t* dev_status, cudaStream_t stream);

/* ----------------------------------------------------------------- MXFP4 */

/* Element types of dense matrices in the MXFP4 calls. */
typedef enum { QSM_BF16 = 0, QSM_FP16 = 1, QSM_FP32 = 2 } qsm_dtype;

/* MXFP4 matrices [experts, rows, cols], cols a multiple of 32: 4-bit
 * floating-point codes (e2m1: sign, two exponent bits, one mantissa bit; 0,
 * 0.5, 1, 1.5, 2, 3, 4, 6) and one scale 2^(s - 127) (e8m0) per block of 32
 * columns; value = code * scale.  s = 255 makes its block not a number.
 *   codes   [experts, rows, cols / 2] bytes, column 2c in the low nibble of
 *           byte c
 *   scales  per expert mx4_scale_bytes(rows, cols) bytes: tiles of 128 rows
 *           x 4 blocks, 512 bytes each, in order [row tile][column tile];
 *           byte 16 (r % 32) + 4 (r / 32) + b of a tile is the scale of its
 *           row r, block b.  Rows and blocks past the matrix hold 0.
 * Both 16-byte aligned. */
typedef struct {
  int32_t experts, rows, cols;
  const uint8_t* codes;
  const uint8_t* scales;
} qsm_mx4;

/* Bytes of the scale tiles of one [rows, cols] matrix. */
QSM_API size_t mx4_scale_bytes(int32_t rows, int32_t cols);

/* x [rows, cols] -> codes and scale tiles (padding included):
 *   s = max(floor(log2 max|x in the block|) + 125, 0), 0 for a block of zeros;
 *   code = the value nearest to x / 2^(s - 127), ties to the even code,
 *   magnitudes over 6 become 6.
 * A block that holds an infinity or a NaN gets s = 255 and sets
 * QSM_DEV_NONFINITE.
 *   x  of type dtype (qsm_dtype), row_stride elements from row to row (a
 *      multiple of 8, at least cols), 16-byte aligned
 * Requires rows >= 0, cols >= 32 and a multiple of 32. */
QSM_API qsm_status mx4_quantize(const void* x, int32_t dtype, int64_t row_stride, int32_t rows,
                                int32_t cols, uint8_t* codes, uint8_t* scales,
                                int32_t* dev_status, cudaStream_t stream);

/* y [experts, rows, cols] (dtype, dense, 16-byte aligned) = the values that
 * a stands for, rounded to dtype (fp16: beyond 65504 infinite). */
QSM_API qsm_status mx4_dequantize(const qsm_mx4* a, int32_t dtype, void* y, cudaStream_t stream);

/* y[m, n] = sum_c a[m, c] * w[n, c], products exact, fp32 accumulation.
 *   a [1, M, K], w [1, N, K];  y [M, N] bf16 or fp32, ldy elements from row
 *   to row (ldy >= N), aligned to its element.
 * An operand row with s = 255 makes its row or column of y not a number. */
QSM_API qsm_status mx4_gemm(const qsm_mx4* a, const qsm_mx4* w, int32_t dtype, void* y,
                            int64_t ldy, int32_t* dev_status, cudaStream_t stream);

/* Most rows of x that mx4_gemv takes. */
#define QSM_MX4_GEMV_MAX_ROWS 32

/* y[t, n] = sum_c x[t, c] * w[n, c] for a few rows of 16-bit activations,
 * which enter the product to 2^-16 of the largest magnitude in their block of
 * 32 (a bf16 within 2^-8 of it is not rounded at all); products exact, fp32
 * accumulation.
 *   x [T, K] bf16, row_stride elements from row to row (a multiple of 8);
 *   w [1, N, K];  y [T, N] bf16 (2-byte aligned).
 * A block of x that holds an infinity, a NaN or a magnitude of 2^127 or more
 * makes its row of y not a number and sets QSM_DEV_NONFINITE.
 * Requires 0 <= T <= QSM_MX4_GEMV_MAX_ROWS, K <= 65536. */
QSM_API qsm_status mx4_gemv(const uint16_t* x, int64_t row_stride, int32_t T, const qsm_mx4* w,
                            uint16_t* y, int32_t* dev_status, cudaStream_t stream);

/* One MoE FFN layer as qsm_moe_layer, with MXFP4 weights: gate_up [E, 2I, H],
 * down [E, H, I], shared_gate_up [1, 2I, H], shared_down [1, H, I], and
 * shared_gate [H] fp32 or NULL.  Requires H % 128 == 0, I % 128 == 0,
 * H, I <= 16384, 1 <= k <= min(E, 32), E <= 1024. */
typedef struct {
  int32_t H, I, E, k;
  qsm_mx4 gate_up, down, shared_gate_up, shared_down;
  const float* shared_gate;
} qsm_mx4_layer;

/* What the expert products of moe_mx4_forward multiply the weights with:
 *   QSM_ACTS_BF16  x and h in 16 bits or more, as mx4_gemv (T <= QSM_MX4_MOE_MAX_ROWS:
 *                  every touched weight is read once, few tokens each)
 *   QSM_ACTS_MX4   x and h quantized to MXFP4 by the rule of mx4_quantize (T k
 *                  up to 2^24: grouped 4-bit products) */
typedef enum { QSM_ACTS_BF16 = 0, QSM_ACTS_MX4 = 1 } qsm_acts;
/* Added to QSM_ACTS_BF16: never the one-launch form, whose CTAs wait for one
 * another (see moe_mx4_forward), for callers whose GPU runs other work beside
 * the call. */
#define QSM_ACTS_SEPARATE_LAUNCHES 16
#define QSM_MX4_MOE_MAX_ROWS 64

/* Bytes of workspace moe_mx4_forward needs (for the same acts, its flag included);
 * 0 if the layer, T or acts is not supported. */
QSM_API size_t moe_mx4_workspace_bytes(const qsm_mx4_layer* L, int32_t T, int32_t acts);

/* The whole layer: route (as moe_route, ids and weights the same bits),
 * group, and for every assignment of token t to expert e
 *     gu = W_gate_up[e] x[t],  h = silu(gu[:I]) * gu[I:],  o = W_down[e] h,
 * the same for the shared expert, and
 *     y[t] = sum_j topk_w[t, j] * o(t, j) + g[t] * o_shared(t),
 * g[t] = sigmoid(x[t] . shared_gate), or 1 when shared_gate is NULL.
 * The sums over j run in ascending j, the shared expert first (but see the
 * one-launch form below): y does not depend on timing, and with QSM_ACTS_BF16
 * a token's y not on the other tokens of the call.
 *   x [T, H] bf16;  flags, w_router, logit_bias, topk_idx, topk_w, y, y_f32
 *   as for moe_layer_forward; y may be x itself; with a shared_gate y may not
 *   overlap x otherwise, and y_f32 not at all (QSM_ERR_INVALID_ARGUMENT);
 *   workspace  >= moe_mx4_workspace_bytes(L, T, acts) bytes, zeros before
 *              its first use, and every call leaves it fit for the next of
 *              the same layer shape, T and acts.
 * One or two tokens with QSM_ACTS_BF16 run in one launch whose CTAs exchange
 * words, if E <= 256, H > 768, I <= 4096, the device holds H / 128 clusters of four
 * such CTAs at once (a GB300: H <= 4864), and their shared memory holds three
 * stages of weights beside the router rows of a CTA's experts and the digits of x
 * (or of two slots' h): T, k and the shape alone decide.
 *  - All CTAs have to be resident at once, so a call that shares the GPU with
 *    work that holds SMs for a second sets QSM_DEV_TIMEOUT; its results are then
 *    invalid and the workspace has to be zeroed before the next call.
 *    QSM_ACTS_SEPARATE_LAUNCHES keeps a call out of this form.
 *  - Its order of sums: the call's distinct experts in ascending id, the shared
 *    expert before them, are dealt to four CTAs in turn; each accumulates the
 *    products of weight x h of all its experts in fp32, and the four sums are
 *    added.  y does not depend on timing, but with two tokens the last fp32 bits
 *    of one's y may depend on the experts that the other chose.
 * With QSM_ACTS_MX4 the outputs of the experts are held in fp16 until they are
 * summed, with a power of two of their own for every 128 columns of a row: to
 * 2^-11 of the value, and 2^-39 of the largest magnitude of the 128; y_f32 is the
 * sum of these.  Magnitudes of 2^20 and more do not fit and set
 * QSM_DEV_FP16_RANGE (their y is infinite or not a number). */
QSM_API qsm_status moe_mx4_forward(const qsm_mx4_layer* L, const uint16_t* x, int32_t T,
                                   int32_t acts, const float* w_router, const float* logit_bias,
                                   int32_t flags, int32_t* topk_idx, float* topk_w, uint16_t* y,
                                   float* y_f32, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_status, cudaStream_t stream);

/* The layer without its router: moe_mx4_forward with topk_idx [T, k] and
 * topk_w [T, k] given (moe_route_scores writes them; 4-byte aligned).  Same
 * arithmetic, always in separate launches, on a workspace of
 * moe_mx4_workspace_bytes(L, T, acts), for QSM_ACTS_BF16 with
 * QSM_ACTS_SEPARATE_LAUNCHES added.  An id outside [0, E) sets QSM_DEV_BAD_EXPERT_ID
 * with QSM_ACTS_MX4; its assignment is left out in either form.  An expert that a
 * token names more than once counts with the sum of its weights with QSM_ACTS_MX4;
 * with QSM_ACTS_BF16 the ids of a token have to differ, as a router's do: else that token's y is
 * not a number and QSM_DEV_BAD_EXPERT_ID is set.  y and y_f32 may not overlap
 * topk_idx or topk_w (QSM_ERR_INVALID_ARGUMENT). */
QSM_API qsm_status moe_mx4_experts(const qsm_mx4_layer* L, const uint16_t* x, int32_t T, int32_t acts,
                                   const int32_t* topk_idx, const float* topk_w, uint16_t* y, float* y_f32,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   cudaStream_t stream);

/* ---------------------------------------------- norms around a block */

/* n(v) = w v / sqrt(mean(v^2) + eps) + b (RMS), or the same of v - mean(v)
 * (LAYER), over the H columns of a row.
 *   weight, bias  [H] fp32, 16-byte aligned, or NULL (1 and 0) */
typedef enum { QSM_NORM_NONE = 0, QSM_NORM_RMS = 1, QSM_NORM_LAYER = 2 } qsm_norm_kind;
typedef struct {
  int32_t kind; /* qsm_norm_kind; NONE has no weight and no bias */
  float eps;    /* >= 0 */
  const float* weight;
  const float* bias;
} qsm_norm;

/* What the gate holds: nothing; a value for each column, a row of them for
 * each token or (stride 0) one for all; or one value for each token. */
typedef enum { QSM_GATE_NONE = 0, QSM_GATE_ROWS = 1, QSM_GATE_TOKENS = 2 } qsm_gate;

/* h_dtype of residual_norm, beside the qsm_dtype values: MXFP4. */
#define QSM_MXFP4 3

typedef struct {
  int32_t H;                    /* columns: a multiple of 8, at most 16384 */
  int32_t x_dtype, y_dtype;     /* qsm_dtype of x and x_out, and of y */
  int32_t gate_dtype;           /* qsm_dtype of the gate */
  int32_t h_dtype;              /* qsm_dtype of h, or QSM_MXFP4 (H a multiple of 32) */
  int32_t gate;                 /* qsm_gate */
  int32_t gate_sigmoid;         /* 1: the gate's values pass a sigmoid first */
  float scale;                  /* finite */
  qsm_norm post, pre;
} qsm_residual_norm;

/* The residual stream around a block, in one pass (fp32 between the loads and
 * the stores):
 *   x_out[t] = x[t] + scale * gate[t] * post(y[t])
 *   h[t]     = pre(x_out[t])              of x_out before it is rounded
 * y is the output of the block before (NULL: x_out = x), h the input of the
 * block after.  Infinities and NaN take their way through the formulas, and so
 * does a row whose squares add up to 2^128 or more, which fp32 does not hold: its
 * norm is the bias, or 0.
 *   x, y, x_out, h  [T, H] with ldx, ldy, ldo, ldh elements from row to row
 *       (at least H; rows 16-byte aligned).  x_out or h may be NULL, not both;
 *       h needs a pre.
 *   gate  QSM_GATE_ROWS: [T, H] as above with ldg, or ldg = 0: [H] for all
 *         tokens; QSM_GATE_TOKENS: value t at gate[t ldg], ldg >= 0; needs a y
 *   h as QSM_MXFP4: the codes of h, dense [T, H / 2] bytes (ldh is not used),
 *       and h_scales its scale tiles, mx4_scale_bytes(T, H) bytes, padding
 *       included; the rule is mx4_quantize's, on the fp32 values.  A block with
 *       an infinity or a NaN sets QSM_DEV_NONFINITE in *dev_status (which may
 *       be NULL for other types).
 * x_out and h may be x or y themselves (same address, stride and element
 * size); what is written may overlap nothing else (QSM_ERR_INVALID_ARGUMENT),
 * but may lie beside it in the rows of one matrix.  T at most 2^30. */
QSM_API qsm_status residual_norm(const qsm_residual_norm* n, int32_t T, const void* x, int64_t ldx,
                                 const void* y, int64_t ldy, const void* gate, int64_t ldg,
                                 void* x_out, int64_t ldo, void* h, int64_t ldh, uint8_t* h_scales,
                                 int32_t* dev_status, cudaStream_t stream);

/* --------------------------------------------------- low-rank adapters */

/* n adapters for a projection of K inputs and N outputs, of at most `rank`
 * ranks each:
 *   a      [n, rank, K] bf16, b [n, N, rank] bf16, 16-byte aligned
 *   scale  [n] fp32 or NULL (1)
 *   ranks  [n] int32 or NULL (all `rank`): how many ranks of an adapter count,
 *          taken into 0 .. rank; the others are not used, whatever they hold
 * K a multiple of 8, rank a multiple of 8 and at most 128, N >= 1, both K and N at
 * most 2^28. */
typedef struct {
  int32_t n, rank, K, N;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  const int32_t* ranks;
} qsm_lora;

/* The adapters of a batch beside a shared projection, one launch:
 *   out[t] = y[t] + scale[i] * b[i] (a[i] x[t]),  i = ids[t];
 * a negative id: none, out[t] = y[t].  The ids may come in any order.  Sums in fp32, out rounded once (a bf16
 * out: a[i] x[t] enters the second product to 2^-17).  A token's result does not depend
 * on the other tokens' values; the order of its sums may depend on T and on how many tokens share its
 * adapter.  Where b holds an infinity the result may be NaN instead (scale[i] a[i] x[t] is
 * multiplied with it in parts).
 *   x [T, K] bf16, ldx elements from row to row (a multiple of 8, at least
 *   K), 16-byte aligned;  ids [T] int32;  y [T, N] (NULL: zeros) and out [T, N] of type
 *   dtype (QSM_BF16 or QSM_FP32), ldy and ldo elements from row to row (at least N),
 *   aligned to their elements (16-byte rows and N a multiple of 8 are faster).
 * out may be y itself (same address and stride); other overlaps are refused.
 * An id of n or more counts as none and sets QSM_DEV_BAD_ADAPTER_ID. */
QSM_API qsm_status lora_add(const qsm_lora* L, const uint16_t* x, int64_t ldx, int32_t T,
                            const int32_t* ids, int32_t dtype, const void* y, int64_t ldy, void* out,
                            int64_t ldo, int32_t* dev_status, cudaStream_t stream);

/* ------------------------------------------------------------------ misc */

/* Static description of a status code. */
QSM_API const char* qsm_status_str(qsm_status s);

/* QSM_ABI_VERSION of the loaded library. */
QSM_API int32_t qsm_abi_version(void);

/* Kernels this library has launched since it was loaded, process-wide:
 * every launch of every entry point counts once, including launches
 * recorded into a CUDA graph under stream capture (a replay of the graph
 * launches them again without counting).  Never fails. */
QSM_API uint64_t qsm_launch_count(void);

/* Test hook: 0 = choose the FFN path by T (default), 1 = always the decode
 * kernels, 2 = always the prefill kernels (when T allows).  Process-wide. */
QSM_API qsm_status qsm_debug_force_path(int32_t mode);

/* Test hook for the bounded waits: make the logit exchange of moe_decode_layer
 * (and of moe_mx4_forward's one-launch form) wait for a call tag `skew` ahead
 * of the call's own (0 = off, the default), so that no call can complete it:
 * every wait runs out, the kernel sets QSM_DEV_TIMEOUT in *dev_status,
 * finishes with invalid results (mx4: the workspace then has to be zeroed) and
 * returns, and the context stays usable.  The call ticket stays consistent (every CTA still
 * arrives once).  Process-wide; skew in [0, 1024]. */
QSM_API qsm_status qsm_debug_barrier_skew(int32_t skew);

/* Test hook for the per-row identity of the fused gate_up projection
 * ("oMLX MoE gate/up 融合优化", "融合原理": the rows of the [gate; up]
 * concatenation come out bit-identical to separate gate and up
 * projections).  With buf set (a device buffer of n_floats fp32), every
 * kernel that computes gate_up from Q8_0 or affine-4 weights also writes,
 * before SwiGLU, the fp32 gate value of intermediate i to buf[row * 2I + i] and the up value to
 * buf[row * 2I + I + i], where row is the row of h the kernel writes:
 *   moe_ffn_forward (decode and prefill paths): the sorted assignment row
 *     (< T*k), then T*k + t for token t of the shared expert: at least
 *     (T*k + T) * 2I floats;
 *   moe_decode_layer: slot * T + t, slot 0 the shared expert and slots
 *     1.. the distinct selected experts in ascending id order: at least
 *     (min(E, T*k) + 1) * T * 2I floats.
 * A call whose buffer is too small returns QSM_ERR_INVALID_ARGUMENT.
 * buf = NULL, n_floats = 0 turns the hook off.  Process-wide, not
 * thread-safe; for tests only. */
QSM_API qsm_status qsm_debug_gu_dump(float* buf, size_t n_floats);

#ifdef __cplusplus
}
#endif

#endif /* QSMOE_H */
