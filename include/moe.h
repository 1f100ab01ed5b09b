/*
 * moe.h -- C ABI of the MI355X (gfx950) fused mixture-of-experts layer:
 * top-k routing, token sort into expert order (dispatch), grouped gate/up
 * GEMM with SwiGLU, grouped down GEMM, weighted combine, and the full
 * backward of that layer, for one GPU's share of the work.
 *
 * The operation is the one described on the pages
 *   "Prime Intellect's Prime Mega MoE Trains Giant AI Models 55% Faster"
 *     (section "Where MoE training loses time": dispatch tokens to their
 *     experts, run the expert MLPs, return outputs to their original
 *     positions; the backward repeats the exchange for gradients) and
 *   "Prime Intellect Fused MoE Kernel: 3.11x MoE Training Speed"
 *     (section "What a mixture-of-experts layer actually does": dispatch,
 *     both expert linear layers, SwiGLU and the combine), with the routing
 *     inputs of "Mario/overlap moe kernel integration" (prime-rl PR 3651,
 *     commit on GroupedExperts.forward: either per-expert token counts or
 *     top scores plus selected expert indices).
 *
 * Notation: T tokens, d hidden size, E experts, k experts per token, I expert
 * intermediate size, R = T*k routed rows.  All matrices are row-major and
 * densely packed (leading dimension = last extent).
 *
 * Math (per token t, slot j, expert e = topk_ids[t][j]):
 *   topk_ids[t]  = the k largest logits of row t, largest first, ties to the
 *                  lower expert index (-0.0 equals +0.0);
 *   topk_w[t][j] = exp(l_tj) / sum_{i<k} exp(l_ti)   (softmax over the k
 *                  selected logits = full softmax renormalised over top k);
 *   h = W_gate_up[e] x_t  (rows [0,I) gate g, rows [I,2I) up u),
 *   a = silu(g) * u,  y_tj = W_down[e] a,  out_t = sum_j topk_w[t][j] y_tj.
 *   The backward is the exact gradient of L = sum(dout * out).
 *
 * Ownership: the caller allocates every buffer (device memory unless noted)
 * and keeps it alive until the stream has finished the call.  The library
 * never allocates, frees or keeps device memory between calls, performs no
 * device-to-host copy and no stream synchronisation: every call only
 * enqueues kernels on `stream` (a hipStream_t; NULL = the default stream),
 * so calls may be captured into a HIP graph.  Calls on different streams
 * need separate workspaces and outputs.
 *
 * Errors: every argument check runs on the host before any HIP call; a
 * failing check returns a status and enqueues nothing.  moe_last_error()
 * gives a message for the last failure on the calling thread.  Device-side
 * contract violations in the ids-in form (an id outside [0, E), repeated ids
 * in a row, non-finite values) are not detected; ids are clamped into
 * [0, E) so that no access leaves its buffer, and results are then
 * unspecified.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad extent, k > E, ...     */
  MOE_ERR_UNSUPPORTED = 2,      /* valid but not built (dtype, alignment)   */
  MOE_ERR_WORKSPACE = 3,        /* workspace smaller than moe_workspace_bytes */
  MOE_ERR_HIP = 4               /* a kernel launch failed                   */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* Precision of the GEMM operands.  MOE_PREC_FP8_BLOCK: blockwise FP8
 * ("Prime Mega MoE Trains Giant AI Models 55% Faster", section "Precision and
 * hardware support": one scale shared by a block of values) as OCP e4m3 with
 * fp32 scales over 1x128 activation blocks and 128x128 weight blocks
 * (weight-gradient operands: 128-row blocks along the token dimension), fp32
 * accumulation.  MOE_PREC_MXFP8: the OCP microscaling format MXFP8 (same
 * section: smaller scaling groups than blockwise FP8; "Mario/overlap moe
 * kernel integration" overview: an mxfp8 precision option): e4m3 values in
 * blocks of 32 along every GEMM operand's contraction dimension, each block
 * with a power-of-two scale stored as an E8M0 byte (see
 * moe_quantize_mxfp8), fp32 accumulation.  MOE_PREC_FP8_BWD (the PR's
 * fp8_bwd option): FP8 in the backward only -- the forward of the bf16 layer,
 * then the backward of MOE_PREC_FP8_BLOCK on the saved bf16 H and Aw (the
 * backward quantises the weights itself).  The fp8 precisions require dtype
 * MOE_BF16, d and I multiples of 128 and T*k*max(d, 2I)/128 < 2^31; H and
 * Aw are stored in bf16, and dH is rounded to bf16 before it is encoded. */
typedef enum {
  MOE_PREC_NATIVE = 0,
  MOE_PREC_FP8_BLOCK = 1,
  MOE_PREC_MXFP8 = 2,
  MOE_PREC_FP8_BWD = 3
} moe_precision;

/* MOE_OP_BACKWARD_RECOMPUTE sizes a moe_backward call that gets saved ==
 * NULL and recomputes what moe_forward would have saved. */
typedef enum {
  MOE_OP_ROUTE = 0,
  MOE_OP_FORWARD = 1,
  MOE_OP_BACKWARD = 2,
  MOE_OP_BACKWARD_RECOMPUTE = 3
} moe_op;

typedef struct {
  int64_t T, d, E, k, I;
  int32_t dtype;        /* moe_dtype of x, weights, out, saved, dout, grads */
  int32_t logits_dtype; /* moe_dtype of logits and dlogits                  */
  int32_t precision;    /* moe_precision                                    */
  float swiglu_limit;   /* 0: SwiGLU; > 0 (finite): clamped SwiGLU, below   */
  int32_t flags;        /* moe_flags; unknown bits are rejected            */
} moe_shape;

/* MOE_FLAG_PERSISTENT: the bf16 GEMMs (gate/up and down forward, down and
 * gate/up data gradients, and, in MOE_PREC_NATIVE, both weight gradients;
 * also the forward of MOE_PREC_FP8_BWD) run as persistent kernels, one
 * work-group per CU walking its XCD's tiles, that issue the next tile's
 * first stage (its gathered token rows and weight slice, or for a weight
 * gradient its first 64 rows of both operands) during the current tile's
 * last K step, so that it loads while that step's MFMAs run and while the
 * epilogue stores: the one-GPU form of the overlapped pipeline in "Prime
 * Intellect's Prime Mega MoE Trains Giant AI Models 55% Faster", section
 * "One kernel overlaps the pipeline".  Results are bit-identical to the
 * default engine's (every tile runs at full height, with the same MFMA
 * order).  Other precisions and MOE_F32 ignore the flag.
 *
 * MOE_FLAG_SKIP_MASKED: for moe_combine alone (below); other calls refuse it. */
typedef enum { MOE_FLAG_PERSISTENT = 1, MOE_FLAG_SKIP_MASKED = 2 } moe_flags;

/* swiglu_limit > 0 selects the clamped SwiGLU that "Mario/overlap moe kernel
 * integration" names for DeepSeek V4 (commit on activations.ClampedSilu);
 * the pages give neither its form nor its constant, so the limit L is an
 * argument and the form is read as a = silu(min(g, L)) * clamp(u, -L, L),
 * with no gradient through an active clamp (g > L, |u| > L).  The pages'
 * other clamped variant (sigmoid of 1.702 g, up + 1) is not computed.  H in
 * `saved` holds the unclamped pre-activations. */

/* Limits checked by every call: 1 <= T <= 2^24, 1 <= k <= E <= 1024,
 * T*k <= 2^27, d and I multiples of 8 in [8, 16384]. */

/* Routing tensors (device pointers).  logits [T,E] in logits_dtype, or NULL
 * for the ids-in form, where topk_ids/topk_w are inputs used as given (no
 * renormalisation).  Otherwise topk_ids/topk_w are outputs.
 *   topk_ids [T,k] int32, topk_w [T,k] float32
 *   counts  [E]   int32  rows per expert
 *   offsets [E+1] int32  exclusive prefix sum of counts, offsets[E] = T*k
 *   row_of  [T*k] int32  flat entry t*k+j -> its row in expert order
 *   src_of  [T*k] int32  row -> flat entry; rows are ordered by expert, then
 *                        by flat entry (token order inside each expert) */
typedef struct {
  const void* logits;
  int32_t* topk_ids;
  float* topk_w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* row_of;
  int32_t* src_of;
} moe_routing;

/* Bytes of device workspace a call with this shape needs (op: moe_op);
 * 0 when the shape or op is invalid (moe_last_error() says why).  The
 * caller owns the workspace: the pages' layer owns persistent buffers
 * ("Mario/overlap moe kernel integration", commit list: symmetric buffers
 * that the layer allocates and destroys itself),
 * whereas on one GPU nothing has to outlive a call, so here every call takes
 * its scratch memory from the caller. */
size_t moe_workspace_bytes(const moe_shape* shape, int op);

/* Bytes of the `saved` buffer written by moe_forward and read by
 * moe_backward (0 for an invalid shape): H [T*k, 2I] (gate|up
 * pre-activations) followed by Aw [T*k, I] (SwiGLU output times the row's
 * top-k weight), both in dtype, in expert-sorted row order.  With an fp8
 * forward (MOE_PREC_FP8_BLOCK, MOE_PREC_MXFP8) the buffer also holds the
 * e4m3 weight codes and scales that the backward's data gradients use (both
 * weights are quantised once, in the forward): for MOE_PREC_FP8_BLOCK the
 * forward's own encodings (a 128 x 128 block has one scale whichever axis
 * the contraction runs over), for MOE_PREC_MXFP8 a second, transposed
 * encoding (its 32-value blocks run along one axis).  The
 * forward keeps these so that the backward, which repeats the layer's
 * exchange for gradients ("Prime Mega MoE Trains Giant AI Models 55%
 * Faster", section "Where MoE training loses time"), need not recompute
 * them; moe_backward with saved == NULL recomputes instead. */
size_t moe_saved_bytes(const moe_shape* shape);

/* The same sizes with a status: MOE_OK and *bytes set, or the reason the
 * shape or op is rejected. */
moe_status moe_workspace_size(const moe_shape* shape, int op, size_t* bytes);
moe_status moe_saved_size(const moe_shape* shape, size_t* bytes);

/* Routing only: top-k (when logits != NULL), per-expert counts and offsets,
 * and the stable expert-order permutation.  The router sends each token to
 * a small subset of experts, and dispatch sorts the tokens into expert
 * order ("Prime Mega MoE Trains Giant AI Models 55% Faster", section "Where
 * MoE training loses time"); the routing tensors are the per-token top
 * scores and selected expert indices, or the per-expert token counts
 * ("Mario/overlap moe kernel integration", commit on
 * GroupedExperts.forward(x, *routing)).  Logits in: the k largest per
 * token, weights the softmax over them (see the math above); ids in
 * (logits == NULL): topk_ids and topk_w are read as given, and only counts,
 * offsets, row_of and src_of are written. */
moe_status moe_route(const moe_shape* shape, moe_routing* routing,
                     void* workspace, size_t workspace_bytes, void* stream);

/* moe_route for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * same kernels and results, with no workspace argument.  The counting
 * sort's per-chunk histograms live in a 4 MiB array of device memory that
 * the library holds on each GPU it runs on until the process ends, so
 * 4 * ceil(T*k / 1024) * E must not exceed 4 MiB (T*k*E <= 2^30); larger
 * shapes get MOE_ERR_UNSUPPORTED before anything is enqueued.  Every call on
 * one GPU uses that GPU's one array: calls that overlap in time on the same
 * GPU (different streams, or host threads) race and must be serialised by
 * the caller.  The array needs no clearing between calls (each call writes
 * every histogram it reads).  The first call on a device looks the array up
 * (hipGetSymbolAddress); no call allocates. */
moe_status moe_route_noalloc(const moe_shape* shape, moe_routing* routing, void* stream);

/* Layer forward: routing as moe_route, then out [T,d] (dtype): dispatch
 * into expert order, both expert linear layers with SwiGLU, and the combine
 * that returns each token's k expert outputs to its position, weighted by
 * topk_w ("Prime Intellect Fused MoE Kernel: 3.11x MoE Training Speed",
 * section "What a mixture-of-experts layer actually does"; "Prime Mega MoE
 * Trains Giant AI Models 55% Faster", section "Where MoE training loses
 * time").  x [T,d], w_gate_up [E,2I,d], w_down [E,d,I] in dtype.  saved:
 * NULL, or a buffer of moe_saved_bytes bytes that moe_backward will read.
 * workspace: moe_workspace_bytes(shape, MOE_OP_FORWARD) bytes, 256-byte
 * aligned; x, the weights, out and saved 16-byte aligned. */
moe_status moe_forward(const moe_shape* shape, const void* x, moe_routing* routing,
                       const void* w_gate_up, const void* w_down, void* out,
                       void* saved, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Layer backward from the routing and `saved` of a moe_forward call with
 * the same inputs.  dout [T,d] (dtype).  Outputs: dx [T,d],
 * dw_gate_up [E,2I,d], dw_down [E,d,I] (dtype; experts with no rows get
 * exact zeros), d_topk_w [T,k] float32, and dlogits [T,E] (logits_dtype;
 * zero outside the selected experts) or NULL.  dlogits requires the logits
 * form of routing (routing->logits != NULL).
 * saved == NULL selects recomputation (activation checkpointing, where a
 * layer costs two forwards and one backward: "Prime Intellect added the
 * missing backward pass to DeepSeek's fused MoE kernel ..."; "Prime Mega MoE
 * Trains Giant AI Models 55% Faster", section "Where MoE training loses
 * time"): the call first reruns the gate/up GEMM (and, with an fp8 forward,
 * the weight encodings) from x and the routing into its workspace, with the
 * same kernels as moe_forward, so the results equal those from a saved
 * buffer bit for bit; the workspace must then hold
 * moe_workspace_bytes(shape, MOE_OP_BACKWARD_RECOMPUTE) bytes. */
moe_status moe_backward(const moe_shape* shape, const void* dout, const void* x,
                        const moe_routing* routing, const void* w_gate_up,
                        const void* w_down, const void* saved, void* dx,
                        void* dw_gate_up, void* dw_down, float* d_topk_w,
                        void* dlogits, void* workspace, size_t workspace_bytes,
                        void* stream);

/* The router's projection, which makes the logits, and its gradients (of shape
 * T, d, E, dtype and logits_dtype are used):
 *   logits [T,E] (logits_dtype) = x w_router^T,  x [T,d], w_router [E,d];
 *   dx [T,d] = dx_in + dlogits w_router,  dlogits [T,E] in logits_dtype,
 *     dx_in [T,d] (for instance moe_backward's dx; may be dx itself) or NULL
 *     for zeros;
 *   dw_router [E,d] = dlogits^T x;
 * all others in dtype; float32 sums in a fixed order, one rounding each.  With
 * dtype MOE_BF16 a float32 dlogits enters the products as the sum of two bf16
 * values (up to 2^-17 of it is lost; one beyond bfloat16's range counts as an
 * infinity).  Infinities of x, w_router and dlogits give infinities where the
 * formulas do.  Every pointer 16-byte aligned; dx and
 * dw_router overlap no input (but dx_in, as said) and not each other;
 * workspace: moe_router_workspace_size bytes, for the backward only. */
moe_status moe_router_forward(const moe_shape* shape, const void* x, const void* w_router,
                              void* logits, void* stream);
moe_status moe_router_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_router_backward(const moe_shape* shape, const void* dlogits, const void* x,
                               const void* w_router, const void* dx_in, void* dx,
                               void* dw_router, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Activation checkpoint in 8 bits: the training step with `saved` at about a
 * third of its size.  Of the forward's H and Aw (6 I bytes a row in bf16) only
 * H is kept, as e4m3 codes with one E8M0 scale byte per 32 columns, counted
 * from the first column of either half (moe_quantize_mxfp8's row encoding; a
 * last block may be short); the backward works from the decoded H wherever
 * moe_backward works from H, and rebuilds Aw from it, rounded to dtype.  The
 * forward's out is moe_forward's, bit for bit.  A block with an infinity or a
 * NaN gets the scale byte 255 and decodes to NaN.  Precision
 * MOE_PREC_NATIVE, both dtypes.
 *   saved8:    moe_saved8_size bytes: codes [T*k, 2I], then, at the next
 *              multiple of 256 bytes, scale bytes [T*k, 2 ceil(I/32)];
 *   workspace: moe_workspace8_size bytes (op MOE_OP_FORWARD or
 *              MOE_OP_BACKWARD).
 * Everything else, flags included, is as for moe_forward and moe_backward. */
moe_status moe_saved8_size(const moe_shape* shape, size_t* bytes);
moe_status moe_workspace8_size(const moe_shape* shape, int op, size_t* bytes);
moe_status moe_forward8(const moe_shape* shape, const void* x, moe_routing* routing,
                        const void* w_gate_up, const void* w_down, void* out, void* saved8,
                        void* workspace, size_t workspace_bytes, void* stream);
moe_status moe_backward8(const moe_shape* shape, const void* dout, const void* x,
                         const moe_routing* routing, const void* w_gate_up, const void* w_down,
                         const void* saved8, void* dx, void* dw_gate_up, void* dw_down,
                         float* d_topk_w, void* dlogits, void* workspace,
                         size_t workspace_bytes, void* stream);

/* The checkpoint's row passes alone, on expert-sorted rows r < T*k with weight
 * w_r = topk_w[src_of[r]] (T, k, I, dtype and swiglu_limit of shape are used,
 * and of routing, src_of and topk_w).  moe_swiglu_save8: H [T*k, 2I] -> codes
 * [T*k, 2I], scales [T*k, 2 ceil(I/32)] and, unless Aw is NULL (routing is
 * then not read), Aw [T*k, I] = w_r silu(g) u (in dtype).
 * moe_swiglu_backward8: from G [T*k, I] (dtype; the gradient of silu(g) u
 * before the row's weight) and the decoded H: dH [T*k, 2I], dw [T*k] float32 =
 * sum over columns of G silu(g) u, and Aw unless NULL.  H, G, Aw, dH and codes
 * 16-byte aligned. */
moe_status moe_swiglu_save8(const moe_shape* shape, const void* H, const moe_routing* routing,
                            void* Aw, uint8_t* codes, uint8_t* scales, void* stream);
moe_status moe_swiglu_backward8(const moe_shape* shape, const void* G, const uint8_t* codes,
                                const uint8_t* scales, const moe_routing* routing, void* dH,
                                void* Aw, float* dw, void* stream);

/* The layer for a few tokens (serving): the forward's arithmetic on at most
 * 256 tokens, reading each selected expert's weights once, from weights that
 * may have been encoded beforehand.  No tiles, sort or encoders run: the call
 * is the gate/up products and the down products, with the routing as a small
 * kernel before them (or, for a few tokens, inside the first) and the combine
 * inside the down products (up to 8 tokens with 32 slots in all) or as a small
 * kernel behind them.
 *
 * shape: T <= 256 and precision MOE_PREC_NATIVE (MOE_ERR_UNSUPPORTED
 * otherwise; moe_forward takes more tokens), T*k*I values of dtype below
 * 4 GiB - 512; dtype is that of x and out; flags are ignored.  weights names
 * the expert weights' format:
 *   MOE_WEIGHTS_NATIVE:    in dtype; s_gate_up and s_down are NULL;
 *   MOE_WEIGHTS_FP8_BLOCK: what moe_quantize_fp8 MOE_QUANT_WEIGHT writes:
 *                          codes, and fp32 scales [E, 2I/128, d/128] and
 *                          [E, d/128, I/128];
 *   MOE_WEIGHTS_MXFP8:     what moe_quantize_mxfp8 MOE_QUANT_WEIGHT writes:
 *                          codes, and scale bytes [E, 2I, d/32] and
 *                          [E, d, I/32]; byte 255 (E8M0's NaN) is not
 *                          recognised;
 *   MOE_WEIGHTS_MXFP4:     what moe_quantize_mxfp4 writes: pairs of codes [E, 2I,
 *                          d/2] and [E, d, I/2], and scale bytes as for
 *                          MOE_WEIGHTS_MXFP8; byte 255 makes its block NaN, and a
 *                          code times scale beyond bfloat16's range is an
 *                          infinity.
 * Coded weights need dtype MOE_BF16 and d, I multiples of 128, and stand for
 * code * scale; x and the activations are not quantised, unlike in
 * moe_forward's fp8 precisions.  Between the two products a bf16 call keeps the
 * activations as two bf16 values (up to 2^-17 of one is lost), where moe_forward
 * rounds them to one.
 *
 * routing: logits, topk_ids and topk_w as in moe_forward; the other members
 * are neither read nor written and may be NULL.  A slot can be empty: a given
 * id outside [0, E), or, with logits, a selected logit of -inf (a masked
 * expert; topk_ids then holds -1 and topk_w 0).  An empty slot adds nothing,
 * whatever its weight, and a token whose slots are all empty (the padding of
 * a batch) gets a row of zeros.  An id given twice in a row counts twice.
 * NaN and infinities stay in the tokens they reach, and an infinite weight gives
 * infinities where the formula does.
 *
 * workspace: moe_decode_workspace_size bytes, 256-byte aligned (no initial
 * contents needed); calls that overlap in time, replayed graphs among them,
 * need one each.  The size is that of the format that needs most: for T <= 8 and
 * T*k <= 32 the others take 4*T*k*d bytes (rounded up to 256) less than
 * MOE_WEIGHTS_MXFP4, and are not refused without them. */
typedef enum { MOE_WEIGHTS_NATIVE = 0, MOE_WEIGHTS_FP8_BLOCK = 1, MOE_WEIGHTS_MXFP8 = 2,
               MOE_WEIGHTS_MXFP4 = 3 } moe_weight_format;
moe_status moe_decode_workspace_size(const moe_shape* shape, size_t* bytes);
moe_status moe_decode(const moe_shape* shape, int weights, const void* x, moe_routing* routing,
                      const void* w_gate_up, const void* s_gate_up, const void* w_down,
                      const void* s_down, void* out, void* workspace, size_t workspace_bytes,
                      void* stream);

/* The norms before and after a block with its gate and residual scale, in one
 * pass over the rows.  With N(v; w) = v / sqrt(mean(v^2) + eps) * w over a
 * row's d columns:
 *   z = res_scale * x + gate * N(y; w_post)   (no w_post: N(y) = y; no gate: 1)
 *   h = N(z; w_next)                          (of z before its rounding to dtype)
 * x [T,d] is the residual stream, y [T,d] the block's output; z goes on as the
 * residual stream and h into the next block.  y == NULL: the norm alone, h =
 * N(x; w_next) (then w_post, gate and z are NULL and res_scale is 1).  w_next
 * == NULL: no h (h is then NULL).  gate: [d] with MOE_GATE_CHANNEL, [T] with
 * MOE_GATE_TOKEN.  All tensors in dtype; sums in float32, one rounding of each
 * result.  An infinity or NaN of x or y stays in its row.  A row whose squares
 * pass float32's range has rsqrt 0.
 *
 * moe_norm_backward: the gradient of sum(dz z) + sum(dh h) at z (moe_norm_forward's,
 * or x without a block) and y.  dz or dh may be NULL; dh and w_next are given
 * together (then z too).  Outputs: dx [T,d] and, with a block (dy != NULL; y is
 * needed with w_post or a gate): dy [T,d], dw_post [d] with w_post, dgate (of
 * gate's extents) with a gate; dw_next [d] with w_next.  The sums over tokens
 * are float32, in a fixed order.  T <= 2^24, d as in moe_shape, eps > 0.
 *
 * Every matrix and weight 16-byte aligned (a gate per token and its gradient:
 * by element); outputs overlap no input and not each other, but z may be x or
 * y and dx may be dz.  workspace: moe_norm_workspace_size bytes, 256-byte
 * aligned, for the backward only. */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 } moe_gate_kind;
typedef struct {
  int64_t T, d;
  int32_t dtype;     /* moe_dtype */
  int32_t gate_kind; /* moe_gate_kind */
  float res_scale, eps;
} moe_norm_shape;
moe_status moe_norm_forward(const moe_norm_shape* shape, const void* x, const void* y,
                            const void* w_post, const void* gate, const void* w_next, void* z,
                            void* h, void* stream);
moe_status moe_norm_workspace_size(const moe_norm_shape* shape, size_t* bytes);
moe_status moe_norm_backward(const moe_norm_shape* shape, const void* dz, const void* dh,
                             const void* z, const void* y, const void* w_post, const void* gate,
                             const void* w_next, void* dx, void* dy, void* dw_post, void* dgate,
                             void* dw_next, void* workspace, size_t workspace_bytes, void* stream);

/* Dispatch alone ("token sorting": "Prime Mega MoE Trains Giant AI Models
 * 55% Faster", section "Where MoE training loses time"): xp[r] =
 * x[src_of[r] / k], xp [T*k, d] (dtype), rows in expert order; reads
 * routing->src_of and routing->row_of (as moe_route wrote them: each token's
 * row is copied to its k expert-sorted rows).  x and xp 16-byte aligned. */
moe_status moe_permute(const moe_shape* shape, const void* x,
                       const moe_routing* routing, void* xp, void* stream);

/* Products of expert-sorted rows with their experts' coded matrices (a prompt
 * through experts that moe_decode serves, or experts of another form):
 *   y[r] = W_e a_r,  offsets[e] <= r < offsets[e+1],
 *   a_r = x[src_of[r] / k] (gather != 0; x [T,d]) or x[r] (x [T*k,d]),
 * or with swiglu != 0, where W_e holds N/2 gate rows and then N/2 up rows,
 * y[r] = silu(g) u (clamped with shape->swiglu_limit > 0), not weighted.
 * weights: MOE_WEIGHTS_MXFP4 (MOE_ERR_UNSUPPORTED otherwise): codes [E,N,d/2],
 * scales [E,N,d/32] as moe_quantize_mxfp4 writes them; bf16 products, float32
 * sums, one rounding.  y [T*k, N] or [T*k, N/2]; rows outside every expert's are
 * left as they were, and so is whatever an offset or entry outside [0, T*k]
 * would reach.  Of shape T, d, E, k and swiglu_limit are used (dtype MOE_BF16,
 * d a multiple of 128); N a multiple of 8 (16 with swiglu) up to 32768.  Reads
 * routing->offsets and, with gather, src_of.  NaN and infinities stay in the
 * rows of x and the columns of W that hold them.  x, codes and y 16-byte, scales
 * 4-byte aligned; y overlaps no input. */
moe_status moe_grouped_product(const moe_shape* shape, int weights, const void* x, int gather,
                               const moe_routing* routing, const uint8_t* codes,
                               const uint8_t* scales, int64_t N, int swiglu, void* y, void* stream);

/* Combine alone (outputs returned to their original positions: "Prime Mega
 * MoE Trains Giant AI Models 55% Faster", section "Where MoE training loses
 * time"; the weighted sum of a token's expert outputs: "Prime Intellect
 * Fused MoE Kernel: 3.11x MoE Training Speed", section "What a
 * mixture-of-experts layer actually does"): out[t] = sum_j topk_w[t][j] *
 * rows[row_of[t*k+j]], summed in float32 in slot order; rows [T*k, d], out
 * [T,d] (dtype); reads routing->row_of and topk_w.  rows and out 16-byte
 * aligned.  With MOE_FLAG_SKIP_MASKED in shape->flags a slot whose expert is
 * masked (routing->logits, in logits_dtype, is -inf at topk_ids[t][j]) adds
 * nothing, whatever its row and weight hold, and a token of masked experts
 * alone gets a row of zeros; logits and topk_ids are then read too. */
moe_status moe_combine(const moe_shape* shape, const void* rows,
                       const moe_routing* routing, void* out, void* stream);

/* Block quantisation to OCP e4m3 with fp32 scales, the operand encoding of
 * MOE_PREC_FP8_BLOCK ("Prime Mega MoE Trains Giant AI Models 55% Faster",
 * section "Precision and hardware support": one scale per block of values).
 * For a block with largest magnitude amax the scale is s = amax / 448 (1 for
 * an all-zero block) and each value x becomes the code of the e4m3 number
 * nearest to the float32 quotient x / s (ties to even, saturating at 448);
 * x is then represented as decode(code) * s.  src is bf16, q holds the
 * 8-bit codes, s the float32 scales (device pointers; src and q 16-byte
 * aligned).  Kinds:
 *   MOE_QUANT_ROWS:     src [n0, n1], 1 x 128 blocks along rows
 *                       -> q [n0, n1], s [n0, n1/128]; n1 % 128 == 0;
 *   MOE_QUANT_WEIGHT:   src [n0, n1, n2], 128 x 128 blocks of each [n1, n2]
 *                       matrix -> q [n0, n1, n2], s [n0, n1/128, n2/128];
 *   MOE_QUANT_WEIGHT_T: the same blocks written transposed
 *                       -> q [n0, n2, n1], s [n0, n2/128, n1/128].
 * n2 is ignored for MOE_QUANT_ROWS. */
typedef enum { MOE_QUANT_ROWS = 0, MOE_QUANT_WEIGHT = 1, MOE_QUANT_WEIGHT_T = 2 } moe_quant_kind;
moe_status moe_quantize_fp8(int kind, const void* src, int64_t n0, int64_t n1, int64_t n2,
                            uint8_t* q, float* s, void* stream);

/* Token-block quantisation of a weight-gradient operand (same encoding):
 * blocks are runs of 128 consecutive expert-sorted rows of one expert's
 * segment (counted from the expert's first row, the last run short) by one
 * column.  Row r of the operand is src[src_of[r] / k] when gather != 0 (src
 * [T, C], token rows) and src[r] otherwise (src [T*k, C], expert order).
 * Output transposed and padded: with nblk = ceil(T*k / 128) + E and
 * blk_off[e] = sum over e' < e of ceil(counts[e'] / 128), run i of expert e
 * is block b = blk_off[e] + i, q [C, 128 nblk] holds its codes at
 * q[c][128 b + j] (zero past the segment) and s [C, nblk] its scales at
 * s[c][b]; blocks b >= blk_off[E] are not written.  shape->dtype must be
 * MOE_BF16, C a multiple of 128; routing->offsets (and src_of when
 * gathering) are read; workspace as for moe_route. */
moe_status moe_quantize_tokens_fp8(const moe_shape* shape, const void* src, int64_t C, int gather,
                                   const moe_routing* routing, uint8_t* q, float* s,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* MXFP8 encoding of MOE_PREC_MXFP8 (OCP microscaling: blocks of 32 values,
 * one E8M0 scale byte per block, e4m3 elements).  For a block with largest
 * magnitude amax the scale is 2^X with X the smallest integer such that
 * amax <= 448 * 2^X (the blockwise scale amax / 448 rounded up to a power of
 * two, so no value saturates), X >= -127, and X = 0 for an all-zero block;
 * the scale byte is X + 127 and each value x becomes the code of the e4m3
 * number nearest to x / 2^X (exact in float32; ties to even).  src is bf16,
 * q the 8-bit codes, s the scale bytes (device pointers; src and q 16-byte
 * aligned, s 4-byte aligned).  Kinds (moe_quant_kind):
 *   MOE_QUANT_ROWS:     src [n0, n1], blocks of 32 along each row
 *                       -> q [n0, n1], s [n0, n1/32]; n1 % 128 == 0;
 *   MOE_QUANT_WEIGHT:   src [n0, n1, n2], blocks of 32 along each row of
 *                       every [n1, n2] matrix (the forward GEMMs' encoding)
 *                       -> q [n0, n1, n2], s [n0, n1, n2/32];
 *   MOE_QUANT_WEIGHT_T: blocks of 32 down each column (the data-gradient
 *                       encoding), written transposed
 *                       -> q [n0, n2, n1], s [n0, n2, n1/32];
 *                       n1, n2 multiples of 128 for both weight kinds. */
moe_status moe_quantize_mxfp8(int kind, const void* src, int64_t n0, int64_t n1, int64_t n2,
                              uint8_t* q, uint8_t* s, void* stream);

/* MXFP4 encoding of weights (OCP microscaling: blocks of 32 values, one E8M0
 * scale byte per block, e2m1 elements) for MOE_WEIGHTS_MXFP4.  For a block with
 * largest magnitude amax the scale is 2^X with X the smallest integer such that
 * amax <= 6 * 2^X (so no value saturates), X >= -127, and X = 0 for an all-zero
 * block; the scale byte is X + 127 and each value x becomes the code of the
 * e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to
 * x / 2^X, ties to even.  A block with an infinity or a NaN gets the scale byte
 * 255 (NaN).  src bf16 [n0, n1, n2], blocks of 32 along each row -> q [n0, n1,
 * n2/2] (the even column in the low four bits), s [n0, n1, n2/32]; n2 a multiple
 * of 128, n0 <= 65535, n1 and n2 <= 65535 * 128, 2^41 values in all; src and q
 * 16-byte, s 4-byte aligned. */
moe_status moe_quantize_mxfp4(const void* src, int64_t n0, int64_t n1, int64_t n2, uint8_t* q,
                              uint8_t* s, void* stream);

/* MXFP8 token-block quantisation of a weight-gradient operand: as
 * moe_quantize_tokens_fp8 (same runs of 128 rows, same q layout), but each
 * run holds four blocks of 32 rows with their own E8M0 scales (a short last
 * run: blocks past the segment are all zero, scale byte 127), and
 * s [C, 4 nblk] bytes holds block m of run b of column c at s[c][4 b + m]. */
moe_status moe_quantize_tokens_mxfp8(const moe_shape* shape, const void* src, int64_t C,
                                     int gather, const moe_routing* routing, uint8_t* q,
                                     uint8_t* s, void* workspace, size_t workspace_bytes,
                                     void* stream);

const char* moe_status_string(moe_status status);
const char* moe_last_error(void);

/* Kernel timing for measurement: between moe_profile_begin and
 * moe_profile_end every kernel the library enqueues carries a start and a
 * stop HIP event on its stream, stamped by the runtime with the kernel's
 * own start and end (hipExtLaunchKernel), so timing adds no packets between
 * kernels.  moe_profile_end waits for those events and returns, per kernel
 * name, the number of launches and their summed duration. */
typedef struct {
  char name[48];
  int64_t launches;
  double total_ms;
} moe_kernel_stat;

moe_status moe_profile_begin(void);
moe_status moe_profile_end(moe_kernel_stat* stats, int capacity, int* count);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
