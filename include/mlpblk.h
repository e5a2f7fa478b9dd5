/*
 * mlpblk.h -- C ABI of the GB300 (sm_103a) forward and backward of the
 * pre-normalised residual ReLU² MLP block
 *
 *     n = RMSNorm(x) = x * r * gamma,     r[t] = 1 / sqrt(mean_k x[t,k]^2 + eps)
 *     h = n . W1^T                        (saved)
 *     a = relu(h)^2                       (saved: it is also the W2 operand)
 *     y = x + a . W2^T
 *
 * Sources (page title -- section):
 *   "Nemotron Kernels From Inference To Backpropagation" -- "Setup: The Shared
 *     Transformer Shell" (pre-norm residual shell; backward starts at the residual
 *     split; RMSNorm backward needs x, gamma and the inverse RMS) and "Kernel 3:
 *     Dense ReLU2 Inference And Backpropagation" (project, relu squared, project;
 *     the pre-activation is kept for backward).
 *   "Reverse-mode automatic differentiation" -- section 5 (MatMul: g.B^T and
 *     A^T.g; Relu; LayerNorm rule, here without the mean terms).
 *   "grow_a_language_model_backprop" -- forward/backward kernel pairing, saved
 *     tensors, += accumulation across microbatches, scale_grads(1/n), zero_grads(),
 *     preallocated buffers.
 *
 * Conventions shared by every entry point
 *   - All tensors are dense and row-major.  x, y, dy, dx: [tokens, d_model];
 *     h, a: [tokens, ffn]; W1, dW1: [ffn, d_model]; W2, dW2: [d_model, ffn];
 *     gamma, dgamma: [d_model]; rstd: [tokens].
 *   - Element types.  MLPBLK_BF16: x, gamma, W1, W2, y, h, a, dy, dx are bfloat16
 *     (passed as 16-bit storage); rstd and the gradient buffers dgamma, dW1, dW2
 *     are float32.  MLPBLK_FP32: every tensor is float32.
 *   - Every pointer except `stream` is a DEVICE pointer, 16-byte aligned, owned by
 *     the caller.  The library allocates no device memory and keeps no per-call
 *     state; the scratch it needs lives in the caller's workspace.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *     default stream) and does not synchronise the host.  Argument errors are
 *     reported by the return value before anything is enqueued.  A device-side
 *     failure (a bounded wait that gave up) is reported later by
 *     mlpblk_last_error().
 *   - Limits: d_model and ffn positive multiples of 8 (16-byte rows); tokens >= 0
 *     and tokens * max(d_model, ffn) < 2^31; eps finite and >= 0.  tokens == 0 is a
 *     valid empty microbatch: the call checks the descriptor and returns MLPBLK_OK
 *     without touching any buffer.
 *   - No C++ exception crosses this boundary.
 */
#ifndef MLPBLK_H
#define MLPBLK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define MLPBLK_OK          0  /* success (work enqueued)                                 */
#define MLPBLK_EINVAL      1  /* null or misaligned pointer, bad size, bad eps          */
#define MLPBLK_ENOTSUP     2  /* unknown dtype, or d_model/ffn not a multiple of 8      */
#define MLPBLK_EWORKSPACE  3  /* workspace smaller than mlpblk_workspace_size()         */
#define MLPBLK_ECUDA       4  /* a CUDA runtime call or a kernel launch failed          */
#define MLPBLK_ETIMEOUT    5  /* a device-side bounded wait gave up (mlpblk_last_error) */
#define MLPBLK_ENODEV      6  /* the current device is not sm_103 (GB300)               */

/* Element-type selector for mlpblk_desc.dtype. */
#define MLPBLK_BF16 1
#define MLPBLK_FP32 2

/* Shape of one microbatch through one block. */
typedef struct {
    int64_t tokens;   /* T: rows of x in this microbatch                     */
    int64_t d_model;  /* d: model width                                      */
    int64_t ffn;      /* F: hidden width of the MLP                          */
    float   eps;      /* RMSNorm epsilon, added to mean(x^2) inside the root */
    int32_t dtype;    /* MLPBLK_BF16 or MLPBLK_FP32                          */
} mlpblk_desc;

/*
 * Bytes of device workspace that mlpblk_forward and mlpblk_backward need for
 * `desc` (one size serves both).  Returns 0 for an invalid descriptor.  The
 * workspace holds scratch only (gamma-folded W1, the rstd-scaled dh, dn, the
 * per-block dgamma partials, and the GEMMs' stream-K partial sums and flags,
 * which every call initialises itself); its contents need not be preserved
 * between calls, but two calls in flight at once must not share one workspace.
 */
size_t mlpblk_workspace_size(const mlpblk_desc *desc);

/*
 * Forward of one microbatch ("Setup: The Shared Transformer Shell";
 * "Kernel 3: Dense ReLU2 ...").
 *   in : x[T,d], gamma[d], w1[F,d], w2[d,F]
 *   out: y[T,d]          = x + relu(h)^2 . W2^T                      (written)
 *        h_saved[T,F]    = RMSNorm(x) . W1^T, rounded to the dtype    (written)
 *        a_saved[T,F]    = relu(h)^2, rounded to the dtype            (written)
 *        rstd_saved[T]   = 1/sqrt(mean_k x^2 + eps), float32          (written)
 * y must not alias x.  Returns an MLPBLK_* code.
 */
int mlpblk_forward(const mlpblk_desc *desc,
                   const void *x, const void *gamma, const void *w1, const void *w2,
                   void *y, void *h_saved, void *a_saved, float *rstd_saved,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * W1 * gamma, the forward's first GEMM operand (RMSNorm's gamma folded into W1
 * along d: w1g[f,k] = w1[f,k] * gamma[k], rounded once to the dtype).  It depends
 * on the weights only, so a caller that runs several microbatches with the same
 * weights (gradient accumulation, "grow_a_language_model_backprop", accumulating
 * across microbatches) makes it once per weight update and passes it to
 * mlpblk_forward_prefolded; mlpblk_forward folds on every call.
 *   in : gamma[d], w1[F,d] (desc->dtype)      out: w1g[F,d] (desc->dtype, written)
 * desc->tokens and desc->eps are not used.  w1g must not alias w1.  Pointers
 * are device pointers, 16-byte aligned.  Returns an MLPBLK_* code.
 */
int mlpblk_fold_weights(const mlpblk_desc *desc, const void *gamma, const void *w1, void *w1g,
                        void *stream);

/*
 * mlpblk_forward with the folded weight from mlpblk_fold_weights in place of
 * gamma and w1: the same outputs, bit for bit, without the per-call fold.
 * Workspace as for mlpblk_forward (mlpblk_workspace_size).
 */
int mlpblk_forward_prefolded(const mlpblk_desc *desc, const void *x, const void *w1g, const void *w2,
                             void *y, void *h_saved, void *a_saved, float *rstd_saved,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward of one microbatch (the residual branch copies forward and adds
 * backward; d relu(h)^2/dh = 2 relu(h), 0 at h = 0; RMSNorm backward from the
 * saved rstd).  Consumes the forward's saved h, a and rstd for the same x.
 *   in : dy[T,d], x[T,d], gamma[d], w1[F,d], w2[d,F], h_saved, a_saved, rstd_saved
 *   out: dx[T,d]        = dy + RMSNorm backward of dn                 (written)
 *        dgamma[d]     += sum_t dn[t,k] * x[t,k] * r[t]      float32 (accumulated)
 *        dw1[F,d]      += dh^T . n                           float32 (accumulated)
 *        dw2[d,F]      += dy^T . a                           float32 (accumulated)
 *   where dh = (dy . W2) * 2 relu(h) and dn = dh . W1.  The gradient buffers keep
 *   a running sum across calls until mlpblk_zero_grads.  dx must not alias dy or
 *   x.  Returns an MLPBLK_* code.
 */
int mlpblk_backward(const mlpblk_desc *desc,
                    const void *dy, const void *x, const void *gamma,
                    const void *w1, const void *w2,
                    const void *h_saved, const void *a_saved, const float *rstd_saved,
                    void *dx, float *dgamma, float *dw1, float *dw2,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * The first microbatch of an accumulation window: the same backward with the
 * gradients set rather than added into ("grow_a_language_model_backprop" --
 * accumulation across microbatches: zero_grads() then += is = for the first
 * microbatch):
 *        dgamma[d]  = sum_t dn[t,k] * x[t,k] * r[t]
 *        dw1[F,d]   = dh^T . n,   dw2[d,F] = dy^T . a        (float32, written)
 * The buffers' prior contents do not matter (NaN included), so the window needs
 * no mlpblk_zero_grads; with T = 0 they are set to zero.  The weight-gradient
 * GEMMs store every output tile that one worker sums whole and add the parts of
 * the tiles they split between workers into regions that the call's first
 * launch clears (with dgamma), so the values are those of mlpblk_zero_grads +
 * mlpblk_backward up to the order in which a split tile's parts are added (the
 * fp32 path clears all three buffers and adds).  dx, the other arguments, the
 * workspace and the return codes are as for mlpblk_backward.
 */
int mlpblk_backward_overwrite(const mlpblk_desc *desc,
                              const void *dy, const void *x, const void *gamma,
                              const void *w1, const void *w2,
                              const void *h_saved, const void *a_saved, const float *rstd_saved,
                              void *dx, float *dgamma, float *dw1, float *dw2,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Recompute variant: save x and rstd only, and rebuild h and a at the start of
 * the backward ("Nemotron Kernels From Inference To Backpropagation" -- Part II:
 * training must preserve or later recompute what reverse mode needs, and an
 * engine states what is saved and what is recomputed; "grow_a_language_model_
 * backprop" -- saved tensors dominate activation memory).  It trades the
 * 2*T*F*elt bytes of saved h and a per block for one more W1 GEMM
 * (2*T*d*F FLOP) in the backward; h and a live in the workspace only while a
 * call runs, so one workspace serves every block of a model.
 *
 * mlpblk_workspace_size_recompute: bytes of workspace both recompute calls
 * need (larger than mlpblk_workspace_size by the T x F h and a).  0 for an
 * invalid descriptor.
 *
 * mlpblk_forward_recompute: y and rstd_saved exactly as mlpblk_forward writes
 * them (same kernels and schedule, the W1 epilogue writing a alone into the
 * workspace; bf16 keeps no h at all).
 *
 * mlpblk_backward_recompute: recomputes h and a from x, W1, gamma and
 * rstd_saved with the forward's W1 GEMM (the same bits the forward produced),
 * then runs mlpblk_backward's kernels; dx written, dgamma/dw1/dw2 += as there.
 * Argument rules and return codes as for mlpblk_forward / mlpblk_backward.
 */
size_t mlpblk_workspace_size_recompute(const mlpblk_desc *desc);

int mlpblk_forward_recompute(const mlpblk_desc *desc,
                             const void *x, const void *gamma, const void *w1, const void *w2,
                             void *y, float *rstd_saved,
                             void *workspace, size_t workspace_bytes, void *stream);

int mlpblk_backward_recompute(const mlpblk_desc *desc,
                              const void *dy, const void *x, const void *gamma,
                              const void *w1, const void *w2, const float *rstd_saved,
                              void *dx, float *dgamma, float *dw1, float *dw2,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Optimizer-side steps after the accumulation loop ("grow_a_language_model_
 * backprop" -- the two-stage gradient-norm kernels and the gradient scale used
 * for clipping; "optimizer state": AdamW holds a first and a second moment per
 * weight; "Losing small gradient contributions in BF16": the state an update
 * accumulates into stays float32).  All asynchronous on `stream`; the norm and
 * the clip scale stay on the device, so clipping needs no host round trip.
 *
 * mlpblk_grad_norm: norm_out[0] = sqrt(sum of g^2 over dgamma[d], dw1[F,d],
 *   dw2[d,F]) and clip_scale_out[0] = min(1, max_norm / (norm + 1e-6)), both
 *   float32 device scalars (either may be NULL, not both).  Per-CTA partial sums
 *   (float32 with compensation, then float64) go to `workspace`
 *   (>= mlpblk_workspace_size(desc) bytes) and are added in a fixed order.
 *   max_norm > 0 and finite.  desc->tokens is ignored.
 *
 * mlpblk_clip_grads: dgamma, dw1, dw2 *= clip_scale[0] (a device scalar, e.g.
 *   the one mlpblk_grad_norm wrote).
 *
 * mlpblk_adamw_step: one AdamW update (decoupled weight decay; Loshchilov &
 *   Hutter, "Decoupled Weight Decay Regularization", Algorithm 2) of `count`
 *   tensors, `step` >= 1 counting updates:
 *     g <- g * grad_scale[0] (if grad_scale is not NULL), w <- w * (1 - lr*wd)
 *     (tensors with decay != 0), m <- b1*m + (1-b1)*g, v <- b2*v + (1-b2)*g^2,
 *     w <- w - lr/(1-b1^step) * m / (sqrt(v)/sqrt(1-b2^step) + eps)
 *   on the float32 master weights, then weight = w in `dtype` (MLPBLK_BF16:
 *   rounded to nearest even; weight may be NULL).  master, grad, m, v 16-byte
 *   aligned, weight 8-byte (bf16) / 16-byte (fp32) aligned, n a positive
 *   multiple of 4; grads are read only.  Returns MLPBLK_EINVAL on bad
 *   hyper-parameters (0 <= beta < 1, lr >= 0, eps >= 0, wd >= 0, finite).
 */
typedef struct {
    float       *master;  /* float32 master weights [n] (updated)                 */
    void        *weight;  /* working copy in `dtype` [n] (written) or NULL         */
    const float *grad;    /* float32 gradient [n]                                  */
    float       *m, *v;   /* AdamW first and second moments [n] (updated)         */
    int64_t      n;       /* elements                                             */
    int32_t      decay;   /* nonzero: apply the weight decay to this tensor        */
} mlpblk_param;

typedef struct {
    float lr, beta1, beta2, eps, weight_decay;
} mlpblk_adamw;

int mlpblk_grad_norm(const mlpblk_desc *desc, const float *dgamma, const float *dw1,
                     const float *dw2, float max_norm, float *norm_out, float *clip_scale_out,
                     void *workspace, size_t workspace_bytes, void *stream);

int mlpblk_clip_grads(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2,
                      const float *clip_scale, void *stream);

int mlpblk_adamw_step(const mlpblk_param *params, int count, const mlpblk_adamw *hp,
                      int64_t step, int dtype, const float *grad_scale, void *stream);

/*
 * FP8-operand variant: the same block with the six GEMMs on E4M3 operands
 * (tcgen05 kind::f8f6f4, float32 accumulators; "Nemotron Kernels From
 * Inference To Backpropagation" -- "Where Quantization Fits": quantisation as a
 * policy for particular tensor edges, higher-precision accumulators kept).
 * Tensors in and out are bf16 (desc->dtype = MLPBLK_BF16), d_model and ffn
 * multiples of 16.  Per-tensor scaling: s = amax / 448, codes E4M3(v / s)
 * nearest-even and saturated, the GEMM epilogue multiplies by the operands'
 * scales.  Quantised: n' = x * rstd (scale 1, |n'| <= sqrt(d)), W1 * gamma, W2,
 * a (from its bf16 value), dy, dh (from its bf16 value), W1; everything else as
 * in mlpblk_forward / mlpblk_backward.
 *
 * Saved by the forward for the backward (caller-owned):
 *   h_saved[T,F] bf16, a8_saved[T,F] E4M3 codes (1 byte), n8_saved[T,d] E4M3
 *   codes of n', rstd_saved[T] float32, scales_saved[4] float32 (a's scale
 *   record {amax, 448/amax, amax/448, 0}).
 * mlpblk_workspace_size_fp8: scratch bytes both calls need; 0 for an invalid or
 *   unsupported descriptor.
 */
size_t mlpblk_workspace_size_fp8(const mlpblk_desc *desc);

int mlpblk_forward_fp8(const mlpblk_desc *desc,
                       const void *x, const void *gamma, const void *w1, const void *w2,
                       void *y, void *h_saved, void *a8_saved, void *n8_saved,
                       float *rstd_saved, float *scales_saved,
                       void *workspace, size_t workspace_bytes, void *stream);

int mlpblk_backward_fp8(const mlpblk_desc *desc,
                        const void *dy, const void *x, const void *gamma,
                        const void *w1, const void *w2,
                        const void *h_saved, const void *a8_saved, const void *n8_saved,
                        const float *rstd_saved, const float *scales_saved,
                        void *dx, float *dgamma, float *dw1, float *dw2,
                        void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same FP8 calls with the weights quantised once, e.g. once per optimizer
 * step for every microbatch of a gradient-accumulation window (the weights do not
 * change between the microbatches, so neither do their codes).
 *
 * mlpblk_fp8_weights_size: bytes of a pre-quantised weight buffer `wq`
 *   (caller-owned, 16-byte aligned): E4M3 codes of W1*gamma [F,d], W2 [d,F] and
 *   W1 [F,d], then their three scale records; 0 for an invalid descriptor.
 * mlpblk_fp8_quantize_weights: fills `wq` from gamma, w1, w2 (bf16) with the same
 *   per-tensor scaling as mlpblk_forward_fp8 / mlpblk_backward_fp8 (uses the FP8
 *   workspace for its amax scratch).  Call it again whenever gamma, W1 or W2
 *   change.
 * mlpblk_forward_fp8_prequant / mlpblk_backward_fp8_prequant: as
 *   mlpblk_forward_fp8 / mlpblk_backward_fp8, reading the weights' codes and
 *   scales from `wq`; outputs are bitwise those of the quantising calls (dW1 and
 *   dW2 up to the order of the reduce-adds of a split weight-gradient tile).
 * Returns an MLPBLK_* code.
 */
size_t mlpblk_fp8_weights_size(const mlpblk_desc *desc);

int mlpblk_fp8_quantize_weights(const mlpblk_desc *desc,
                                const void *gamma, const void *w1, const void *w2,
                                void *wq, size_t wq_bytes,
                                void *workspace, size_t workspace_bytes, void *stream);

int mlpblk_forward_fp8_prequant(const mlpblk_desc *desc,
                                const void *x, const void *wq,
                                void *y, void *h_saved, void *a8_saved, void *n8_saved,
                                float *rstd_saved, float *scales_saved,
                                void *workspace, size_t workspace_bytes, void *stream);

int mlpblk_backward_fp8_prequant(const mlpblk_desc *desc,
                                 const void *dy, const void *x, const void *gamma, const void *wq,
                                 const void *h_saved, const void *a8_saved, const void *n8_saved,
                                 const float *rstd_saved, const float *scales_saved,
                                 void *dx, float *dgamma, float *dw1, float *dw2,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* The two FP8 backwards with dgamma, dw1 and dw2 set instead of added into (the
 * first microbatch of an accumulation window), as mlpblk_backward_overwrite is
 * to mlpblk_backward: the weight-gradient GEMMs store the tiles one worker sums
 * whole and add split tiles' parts into regions the call's first launch clears.
 * Arguments, layouts, ownership and error codes are those of the adding forms;
 * the old contents of the three gradient buffers are never read (NaN is fine).
 * With tokens == 0 the call zeroes dgamma, dw1 and dw2 (MLPBLK_EINVAL if one of
 * them is not 16-byte aligned). */
int mlpblk_backward_fp8_overwrite(const mlpblk_desc *desc,
                                  const void *dy, const void *x, const void *gamma,
                                  const void *w1, const void *w2,
                                  const void *h_saved, const void *a8_saved, const void *n8_saved,
                                  const float *rstd_saved, const float *scales_saved,
                                  void *dx, float *dgamma, float *dw1, float *dw2,
                                  void *workspace, size_t workspace_bytes, void *stream);
int mlpblk_backward_fp8_prequant_overwrite(const mlpblk_desc *desc,
                                           const void *dy, const void *x, const void *gamma, const void *wq,
                                           const void *h_saved, const void *a8_saved, const void *n8_saved,
                                           const float *rstd_saved, const float *scales_saved,
                                           void *dx, float *dgamma, float *dw1, float *dw2,
                                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Routed ReLU^2 experts ("Nemotron Kernels From Inference To Backpropagation" --
 * "Kernel 4: Routed ReLU2 MoE Inference And Backpropagation"): the pre-norm
 * shell around a mixture of ReLU^2 experts with a given top-k dispatch,
 *   y[t] = x[t] + sum_j p[t,j] * W2_e relu(W1_e n[t])^2,  e = expert_idx[t,j],
 * n = RMSNorm(x) as in mlpblk_forward.  The dispatch is held fixed ("Hard
 * Top-K Has No Ordinary Derivative"); the backward returns d_hidden (dx),
 * d_routing_weights (dp), d_expert_up (dw1s +=), d_expert_down (dw2s +=) and
 * dgamma (+=).  bf16 tensors (base.dtype = MLPBLK_BF16), float32 routing
 * weights and gradients, int32 expert ids; an id outside [0, experts) selects
 * nothing.  Weights: w1s[E][F][d], w2s[E][d][F].
 *
 * Each expert's (token, slot) assignments run as one segment of a grouped GEMM
 * (segments padded to 256 rows, token order within a segment); every sum has a
 * fixed order except the weight-gradient accumulation (TMA reduce-add).
 *
 * saved: written by the forward, read by the backward (rstd, the dispatch, the
 * gathered inputs, h, a and the experts' outputs); mlpblk_moe_saved_size bytes.
 * workspace: scratch; mlpblk_moe_workspace_size bytes.  Both sizes are 0 for an
 * invalid descriptor (experts 1..256, top_k 1..experts, d_model <= 4096).
 */
typedef struct {
    mlpblk_desc base;   /* tokens, d_model, ffn (per expert), eps, dtype        */
    int32_t experts;    /* E                                                    */
    int32_t top_k;      /* k: experts per token                                 */
} mlpblk_moe_desc;

size_t mlpblk_moe_saved_size(const mlpblk_moe_desc *desc);
size_t mlpblk_moe_workspace_size(const mlpblk_moe_desc *desc);

int mlpblk_moe_forward(const mlpblk_moe_desc *desc,
                       const void *x, const void *gamma, const void *w1s, const void *w2s,
                       const int32_t *expert_idx, const float *routing_weights,
                       void *y, void *saved, size_t saved_bytes,
                       void *workspace, size_t workspace_bytes, void *stream);

int mlpblk_moe_backward(const mlpblk_moe_desc *desc,
                        const void *dy, const void *x, const void *gamma,
                        const void *w1s, const void *w2s, const float *routing_weights,
                        const void *saved, void *dx, float *d_routing_weights,
                        float *dgamma, float *dw1s, float *dw2s,
                        void *workspace, size_t workspace_bytes, void *stream);

/* As mlpblk_moe_backward, with dgamma, dw1s and dw2s set instead of added
 * into (the first microbatch of an accumulation window; see
 * mlpblk_backward_overwrite).  Here each expert's weight-gradient tile is one
 * worker's whole sum, so the GEMMs store it where they would add it (bitwise
 * the same values), and the blocks of experts that no token chose are set to
 * zero by the first launch of the backward. */
int mlpblk_moe_backward_overwrite(const mlpblk_moe_desc *desc,
                                  const void *dy, const void *x, const void *gamma,
                                  const void *w1s, const void *w2s, const float *routing_weights,
                                  const void *saved, void *dx, float *d_routing_weights,
                                  float *dgamma, float *dw1s, float *dw2s,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Tokens sorted by expert and back ("Kernel 4: Routed ReLU2 MoE": select, execute,
 * weight and combine), for programs that bring expert networks of their own; the
 * routed block above does the same inside mlpblk_moe_forward.  The dispatch is given.
 *
 * Entry i = t * top_k + j is slot j of token t.  Expert e's entries, in increasing
 * i, take the rows seg[e] .. seg[e] + count[e] of the sorted order; segments
 * follow one another in expert order and each is padded to a multiple of
 * desc->pad rows.  An id outside [0, experts) selects nothing; a token may name an
 * expert more than once.
 *
 * mlpblk_moe_sort_rows: R, the number of rows that the sorted buffers hold, an upper
 *   bound of seg[experts] for any ids: T*k + min(experts, T*k) * (pad - 1), rounded
 *   up to a multiple of pad.  -1 for an invalid descriptor, 0 for tokens = 0.
 * mlpblk_moe_sort: the plan, one launch, no workspace.
 *     in : expert_idx[T,k]
 *     out: count[E], seg[E+1], pos[T,k] = the entry's row or -1,
 *          row_map[R] = the row's entry i, or -1 for padding and for the rows at
 *          or behind seg[E]                                          (all written)
 * mlpblk_moe_permute: rows[pos[t,j]] = x[t]; padding rows inside the segments are
 *   zero.  Rows at or behind seg[E] are left as they were.
 * mlpblk_moe_permute_backward: dx[t] = sum_j d_rows[pos[t,j]], in slot order
 *   (slots that select nothing add nothing; the padding rows are not read).
 * mlpblk_moe_unpermute: y[t] = residual[t] + sum_j weights[t,j] * rows[pos[t,j]], in
 *   slot order; residual NULL adds nothing, weights NULL weighs each slot by 1; y
 *   may be residual itself.
 * mlpblk_moe_unpermute_backward: d_rows[pos[t,j]] = weights[t,j] * dy[t] (padding
 *   rows zero, rows at or behind seg[E] left as they were) and
 *   d_weights[t,j] = <dy[t], rows[pos[t,j]]> (0 for a slot that selects nothing).
 *   The gradient of residual is dy.  weights NULL weighs by 1; with d_weights NULL
 *   rows is not read and may be NULL.
 *
 * x, y, dx, dy, residual [T, width] and rows, d_rows [R, width] are in
 * desc->dtype, weights and d_weights float32, the rest int32.  Sums are held in
 * float32 and rounded once; their order is fixed.  Any width; rows of a multiple
 * of 16 bytes move in 16-byte accesses.  pos, count and seg are those that
 * mlpblk_moe_sort wrote for the same descriptor.  Limits: width < 2^30, experts
 * 1..256, top_k 1..256, pad 1..1024, R < 2^31.  Pointers are device pointers, 16-byte aligned.
 * Outputs share no byte with an input (MLPBLK_EINVAL) but where stated, nor with each
 * other.  Each returns an
 * MLPBLK_* code; tokens = 0 returns MLPBLK_OK and touches nothing, except that
 * mlpblk_moe_sort still writes count and seg (zeros).
 */
typedef struct {
    int64_t tokens;   /* T >= 0                                       */
    int64_t width;    /* elements of a row, >= 1                       */
    int32_t experts;  /* E                                             */
    int32_t top_k;    /* k                                             */
    int32_t pad;      /* segments are padded to a multiple of this      */
    int32_t dtype;    /* of the rows: MLPBLK_BF16 or MLPBLK_FP32        */
} mlpblk_sort_desc;

int64_t mlpblk_moe_sort_rows(const mlpblk_sort_desc *desc);

int mlpblk_moe_sort(const mlpblk_sort_desc *desc, const int32_t *expert_idx, int32_t *count, int32_t *seg,
                    int32_t *pos, int32_t *row_map, void *stream);

int mlpblk_moe_permute(const mlpblk_sort_desc *desc, const void *x, const int32_t *pos, const int32_t *count,
                       const int32_t *seg, void *rows, void *stream);

int mlpblk_moe_permute_backward(const mlpblk_sort_desc *desc, const void *d_rows, const int32_t *pos, void *dx,
                                void *stream);

int mlpblk_moe_unpermute(const mlpblk_sort_desc *desc, const void *rows, const int32_t *pos, const float *weights,
                         const void *residual, void *y, void *stream);

int mlpblk_moe_unpermute_backward(const mlpblk_sort_desc *desc, const void *dy, const void *rows,
                                  const int32_t *pos, const int32_t *count, const int32_t *seg,
                                  const float *weights, void *d_rows, float *d_weights, void *stream);

/*
 * MXFP4: microscaled 4-bit matrices and their product ("Where Quantization Fits";
 * the format is the OCP Microscaling Formats specification's MXFP4).  32
 * consecutive values of a row share one power-of-two scale (E8M0, a byte: the
 * exponent plus 127) and are kept as E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives).
 *
 * Rounding: scale exponent = floor(log2(max |v| of the block)) - 2, at least -127;
 * codes are v / scale rounded to nearest even and saturated at 6.  A block that
 * holds an infinity or a NaN gets the scale byte 255 and reads back as NaN.  A
 * block of zeros has scale byte 0.
 *
 * A quantised matrix Q[rows, cols] is two buffers, `batch` matrices back to back
 * in each (every expert's weights, say):
 *   codes : rows of ceil(cols / 32) * 16 bytes, two values a byte, the even column in
 *           the low half; columns behind cols are zero codes
 *   scales: tiles of 128 rows x 4 blocks (128 columns), 512 bytes each; the byte of
 *           row r, block b inside a tile is (r % 32) * 16 + (r / 32) * 4 + b (the
 *           order in which tensor memory holds them); the tiles of
 *           128 rows follow one another along the columns, 2 * ceil(cols / 256) of
 *           them (an even count; bytes of rows and blocks that do not exist are 0)
 *
 * mlpblk_fp4_codes_size, mlpblk_fp4_scales_size: their bytes; 0 for an invalid
 *   descriptor.
 * mlpblk_fp4_quantize: Q = x, or with desc->transposed Q = x^T of a source stored
 *   [cols, rows] (blocks of 32 along the source's columns; the operands of a
 *   weight gradient).  desc->act = MLPBLK_FP4_ACT_RELU2 quantises relu(x)^2
 *   (computed in float32).  desc->dtype is x's type.  row_map (NULL: none; a
 *   device array of one int per source row, e.g. the one mlpblk_moe_sort wrote)
 *   maps the source's rows: where row_map[r] < 0 row r is zeros and x is not read
 *   there, otherwise it is x's row row_map[r] / map_div for map_div > 0, and
 *   x's row r for map_div = 0.  With transposed the mapped rows are Q's columns.
 *   A gathering map (map_div > 0) needs desc->source_rows, x's row count: a row that
 *   it maps to source_rows or beyond (a map of a larger batch) is zeros too, so no
 *   access leaves x.  row_map needs batch = 1.  Every byte of codes and scales is
 *   written.
 * mlpblk_fp4_dequantize: y[batch, rows, cols] in desc->dtype (exact in both types).
 *   transposed and act must be 0.
 * Limits: rows, cols >= 0 (with either 0: MLPBLK_OK, nothing is touched),
 * rows * batch and cols < 2^31, ceil(rows / 128) * batch < 2^29, ceil(rows / 128) *
 * batch * ceil(cols / 256) < 2^28 (275 GB of scales), rows * batch * ceil(cols / 256)
 * < 2^31; pointers 16-byte aligned; outputs share no byte with an input or with each
 * other (MLPBLK_EINVAL).
 */
#define MLPBLK_FP4_ACT_NONE   0
#define MLPBLK_FP4_ACT_RELU2  1

typedef struct {
    int64_t rows, cols;   /* of Q                                         */
    int32_t batch;        /* matrices, >= 1                               */
    int32_t dtype;        /* of x or y: MLPBLK_BF16 or MLPBLK_FP32         */
    int32_t transposed;   /* 1: the source is stored [cols, rows]          */
    int32_t act;          /* MLPBLK_FP4_ACT_*                              */
    int64_t source_rows;  /* rows of x under a gathering row_map (>= 1 there,
                             < 2^31); not used otherwise                   */
} mlpblk_fp4_desc;

size_t mlpblk_fp4_codes_size(const mlpblk_fp4_desc *desc);
size_t mlpblk_fp4_scales_size(const mlpblk_fp4_desc *desc);

int mlpblk_fp4_quantize(const mlpblk_fp4_desc *desc, const void *x, const int32_t *row_map, int32_t map_div,
                        void *codes, void *scales, void *stream);

int mlpblk_fp4_dequantize(const mlpblk_fp4_desc *desc, const void *codes, const void *scales, void *y,
                          void *stream);

/*
 * Products of MXFP4 matrices on the tensor cores (tcgen05 kind::mxf4, float32
 * accumulators), no workspace.  C is dense, row-major, in out_dtype;
 * accumulate = 1 (float32 only) adds into C, the gradient rule of this library, 0
 * sets it.  Each output has one fixed order of summation.
 *
 * mlpblk_fp4_matmul: C[m,n] = A[m,k] . B[n,k]^T (k: the quantised columns).  The
 *   three products of a linear layer y = x W^T: y from Q(x), Q(W); dx from
 *   Q(dy), Q(W^T); dW from Q(dy^T), Q(x^T).
 * mlpblk_fp4_matmul_grouped: the experts' products in sorted order.  A [m = R, k]
 *   holds the sorted rows, B is a batch of `experts` matrices [n, k]; for every
 *   row r of expert e's rows, C[r] = A[r] . B[e]^T.  Padding rows of a segment are
 *   either left as they were or get A's padding row times B[e]^T; rows at or
 *   behind seg[E] are left as they were.  pad (that of the sort) is a multiple of 128.
 * mlpblk_fp4_wgrad_grouped: the experts' weight gradients.  A [m, k = R] and B
 *   [n, k = R] are quantised along the sorted order (transposed, with the
 *   row_map, so that padding is zero); C[e][m,n] = the sum over expert e's
 *   segment, zero (or nothing added) for an expert without rows.  pad is a
 *   multiple of 256.
 * count and seg are those of mlpblk_moe_sort.  With m = 0 (wgrad_grouped: k = 0, not
 * accumulating: C is still set to zero) nothing is touched.  Limits: m, n, k and
 * experts * n (wgrad: experts * m) < 2^31, experts 1..256; experts and pad are 0 for
 * mlpblk_fp4_matmul.  Pointers are device pointers, 16-byte aligned; C shares no byte
 * with an operand, count or seg (MLPBLK_EINVAL).  Returns an MLPBLK_* code.
 */
typedef struct {
    int64_t m, n, k;
    int32_t out_dtype;    /* MLPBLK_BF16 or MLPBLK_FP32                   */
    int32_t accumulate;   /* 1: C += (MLPBLK_FP32 only)                    */
    int32_t experts;      /* grouped forms: 1..256; else 0                */
    int32_t pad;          /* grouped forms: the sort's pad; else 0        */
    int64_t max_rows;     /* matmul_grouped: no expert has more rows than this
                             (e.g. T * top_k), rows beyond it are not computed;
                             0: no bound known, and in the other forms      */
} mlpblk_fp4_matmul_desc;

int mlpblk_fp4_matmul(const mlpblk_fp4_matmul_desc *desc, const void *a_codes, const void *a_scales,
                      const void *b_codes, const void *b_scales, void *c, void *stream);

int mlpblk_fp4_matmul_grouped(const mlpblk_fp4_matmul_desc *desc, const void *a_codes, const void *a_scales,
                              const void *b_codes, const void *b_scales, const int32_t *count,
                              const int32_t *seg, void *c, void *stream);

int mlpblk_fp4_wgrad_grouped(const mlpblk_fp4_matmul_desc *desc, const void *a_codes, const void *a_scales,
                             const void *b_codes, const void *b_scales, const int32_t *seg, void *c,
                             void *stream);

/*
 * Test hook: the kernel that the product `desc` takes on a device of `sms` SMs (form 0:
 * mlpblk_fp4_matmul, 1: mlpblk_fp4_matmul_grouped, 2: mlpblk_fp4_wgrad_grouped), so that
 * tests can say which kernel they reach.  One of MLPBLK_FP4_KERNEL_PAIR_TMA and
 * MLPBLK_FP4_KERNEL_PAIR (CTA pairs; C stored by TMA, or by threads), or the number of CTAs
 * that share a tile's K (1, 2, 4, 8) in the kernel of single CTAs; -1 for a descriptor that
 * is invalid or launches nothing.  Host only.
 */
#define MLPBLK_FP4_KERNEL_PAIR_TMA  256
#define MLPBLK_FP4_KERNEL_PAIR      257
int mlpblk_fp4_product_kernel(const mlpblk_fp4_matmul_desc *desc, int form, int sms);

/*
 * The router of routed experts ("Kernel 4: Routed ReLU2 MoE": select): logits -> expert ids
 * and routing weights, as mlpblk_moe_sort, mlpblk_moe_unpermute and mlpblk_moe_forward take
 * them.
 *   s_e   = softmax over the token's open experts, or 1 / (1 + exp(-l_e))   (desc->score)
 *   key_e = s_e + bias_e; bias NULL: s_e.  The bias balances the experts' load; it decides
 *           what is selected and enters nothing else
 *   groups: the experts lie in desc->groups equal runs; a group's mark is the sum of its two
 *           best keys (of the only one, if it has one open expert); the top_groups best marks
 *           stay, ties to the lower group
 *   expert_idx[t,j]      = the j-th best key's expert among those groups, ties to the lower
 *                          expert (so a token names no expert twice); -1 where no open
 *                          expert is left
 *   routing_weights[t,j] = scale * s, or with desc->renorm scale * s / (sum_j s + 1e-20); 0
 *                          beside -1
 * A logit of -infinity or NaN closes its expert to the token; +infinity counts as the largest
 * finite float32 (of bf16 logits, too).  A row whose experts are all closed selects nothing.  The order is that of
 * the scores in float64 (without a bias, of the logits), whatever the arithmetic here:
 * float32 keys that are too close to call are computed again.  A bias of -infinity or NaN
 * closes its expert to selection, whose share of the softmax stays; one of +infinity puts it first.
 *
 * mlpblk_moe_route_backward: d_logits[T,E] (written) from d_routing_weights[T,k], for the
 * ids of the same logits, held fixed ("Hard Top-K Has No Ordinary Derivative").  Ids outside
 * 0 .. E-1 and closed experts have no gradient, and their d_routing_weights no part in the others'.  The bias has none.
 *
 * logits and d_logits [T,E] are in desc->dtype, the rest float32 and int32; scores, sums and
 * quotients are float32, their order fixed.  Limits: tokens < 2^31, experts 1..256, top_k
 * 1..16, groups 1..64 and a divisor of experts, top_groups 1..groups, top_k at most
 * top_groups * experts / groups, scale finite.  Pointers are device pointers, 16-byte
 * aligned; outputs share no byte with an input or with each other (MLPBLK_EINVAL).  tokens = 0 returns
 * MLPBLK_OK and touches nothing.
 */
#define MLPBLK_ROUTE_SOFTMAX  0
#define MLPBLK_ROUTE_SIGMOID  1
#define MLPBLK_ROUTE_MAX_TOP_K 16

typedef struct {
    int64_t tokens;       /* T >= 0                                              */
    int32_t experts;      /* E                                                   */
    int32_t top_k;        /* k                                                   */
    int32_t score;        /* MLPBLK_ROUTE_SOFTMAX or MLPBLK_ROUTE_SIGMOID         */
    int32_t groups;       /* 1: none                                             */
    int32_t top_groups;   /* groups that stay; = groups: all                      */
    int32_t renorm;       /* 1: the weights are divided by their sum              */
    float   scale;        /* of the weights                                      */
    int32_t dtype;        /* of the logits: MLPBLK_BF16 or MLPBLK_FP32             */
} mlpblk_route_desc;

int mlpblk_moe_route(const mlpblk_route_desc *desc, const void *logits, const float *bias, int32_t *expert_idx,
                     float *routing_weights, void *stream);

int mlpblk_moe_route_backward(const mlpblk_route_desc *desc, const void *logits, const int32_t *expert_idx,
                              const float *d_routing_weights, void *d_logits, void *stream);

/*
 * The residual sum and RMSNorm of the pre-norm shell, with an 8-bit output ("Setup: The
 * Shared Transformer Shell"; "Where Quantization Fits"), for programs whose next products
 * are their own:
 *   sum   = x + residual, rounded to the dtype; residual NULL: sum is x itself
 *   rstd  = 1 / sqrt(mean_k sum^2 + eps)
 *   n     = sum * rstd * gamma                                    (optional output, dtype)
 *   scales = max |n| / 448 over the row (desc->block = 0: [T]), or over each run of 128
 *           columns (desc->block = 128: [T, ceil(width / 128)]), rounded to float32; 1
 *           where that is 0
 *   codes = E4M3(n / scale), nearest even                         [T, width], a byte each
 * sum is written where residual is given (and only then) and may be x or residual itself.
 * codes and scales are given together; n, codes and rstd may be NULL, n and codes not both.
 * The codes are those of the real number n / scale, rounded once (where the products
 * sum * gamma are in float32's normal range: smaller ones are rounded to it, one beyond it makes its scale
 * and that scale's codes NaN).  A row that holds an infinity or a NaN, or whose squares' sum leaves float32's range,
 * has a NaN rstd and NaN scales and codes: no row of magnitudes below 2^56, possibly one with a
 * larger magnitude, certainly one with 2^63 or more.  Squares below 2^-149 count as zero, and below 2^-126 they
 * keep as many bits as float32 has there.  A gamma that is NaN or infinite makes the scales over it NaN, and those scales' codes.
 *
 * mlpblk_add_rmsnorm_backward: with dn the gradient of n (as the codes stand for it:
 *   rounding passes it on) and d_sum that of sum (NULL: none),
 *     dx[T,width] = d_sum + rstd * (g - xh * mean_k(g * xh)),  g = dn * gamma, xh = sum * rstd
 *                   (written; the gradient of x and of residual)
 *     dgamma[width] += (overwrite = 1: =) sum_t dn * xh               float32
 *   sum and rstd are the forward's (sum is x where there was no residual).  dx may be dn or
 *   d_sum itself.  Sums are float32 in a fixed order.  workspace: scratch,
 *   mlpblk_add_rmsnorm_workspace_size bytes (0 for an invalid descriptor), not shared by two
 *   calls in flight.  With tokens = 0 dgamma is set to zero when overwriting; nothing else
 *   is touched.
 *
 * x, residual, gamma, sum, n, dn, d_sum, dx are in desc->dtype.  Limits: tokens < 2^31,
 * 1 <= width <= 16384 (MLPBLK_ENOTSUP beyond), eps finite and >= 0.  Rows of a multiple of 16 bytes
 * move in 16-byte accesses.  Pointers are device pointers, 16-byte aligned; outputs share no
 * byte with an input but where stated, nor with each other (MLPBLK_EINVAL).  tokens = 0
 * returns MLPBLK_OK and touches nothing but what is stated.
 */
typedef struct {
    int64_t tokens;   /* T >= 0                                       */
    int64_t width;    /* elements of a row                              */
    float   eps;
    int32_t dtype;    /* MLPBLK_BF16 or MLPBLK_FP32                    */
    int32_t block;    /* columns that share a scale: 0 (a row) or 128   */
} mlpblk_norm_desc;

int mlpblk_add_rmsnorm(const mlpblk_norm_desc *desc, const void *x, const void *residual, const void *gamma,
                       void *sum, void *n, void *codes, float *scales, float *rstd, void *stream);

size_t mlpblk_add_rmsnorm_workspace_size(const mlpblk_norm_desc *desc);

int mlpblk_add_rmsnorm_backward(const mlpblk_norm_desc *desc, const void *dn, const void *d_sum, const void *sum,
                                const float *rstd, const void *gamma, void *dx, float *dgamma, int32_t overwrite,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * Orthogonalised updates for matrices, beside AdamW ("optimizer state": here one moment per
 * weight; the step is Muon's, K. Jordan et al., 2024).
 *
 * mlpblk_orthogonalize: o[batch, rows, cols] (bf16, written) = the result of desc->steps
 *   Newton-Schulz steps on each u[rows, cols] (desc->dtype):
 *     X = u / (|u| + eps),   |u| the Frobenius norm;   then for each step's (a, b, c)
 *     X <- a X + (b G + c G^2) X,  G = X X^T
 *   (the odd polynomial a s + b s^3 + c s^5 on the singular values; a tall u is worked on from
 *   its right, which is the same).  u is not changed; a matrix of zeros gives zeros.
 * mlpblk_muon_step: one update of `batch` weights (float32 master, gradient and momentum):
 *     g <- grad * grad_scale[0] (NULL: 1),  momentum <- beta momentum + g
 *     u = g + beta momentum (nesterov), or momentum;   X as above (not rounded to bf16)
 *     master <- master * (1 - lr * weight_decay) - lr * scale * X
 *   then weight = master in desc->dtype (NULL: none).
 *
 * Precision: products of fp16 values, whose range X's scaling fits, with float32 sums; a X
 * takes X as two fp16 values in all but the last step.  With Muon's coefficients
 * (3.4445, -4.7750, 2.0315), five steps, the error against the formula, in the Frobenius norm and before o's rounding to
 * bf16 (X in muon_step), is
 *   up to 3e-3 where u's entries round independently (noise, low rank, strong directions or a large entry over noise) and
 *   its short side is 64 or more, mostly 1e-3 to 2e-3; up to 6e-3 for short sides from 12 on, up to 2e-2 below;
 *   up to 2e-2 at any size where roundings agree: few entries that are not zero, an orthogonal u (dense ones 1e-3 to 4e-3,
 *   multiples of the identity or of a permutation mostly 1e-3 to 5e-3), a constant or nearly equal rows over noise of 1e-3
 *   of them or less.
 * The matrices b G + c G^2 are fp16 too: every singular
 * value s on the way must keep |b s^2 + c s^4| and, of two neighbouring steps, |a a'| below 60000
 * (with those coefficients s < 13).  A NaN or an
 * infinity in u makes its matrix NaN.  Sums have a fixed order.
 *
 * mlpblk_orthogonalize_workspace_size: bytes of scratch for both; 0 for an invalid
 *   descriptor.  Not shared by two calls in flight.
 * Limits: rows and cols 1 .. 131072, batch 1 .. 65535, rows * cols * batch < 2^40,
 * steps 1 .. MLPBLK_ORTHO_MAX_STEPS, coefficients and hyper-parameters finite, eps >= 0, 0 <= momentum
 * < 1, lr and weight_decay >= 0.  Pointers are device pointers, 16-byte aligned; outputs and
 * the workspace share no byte with an input or with each other (MLPBLK_EINVAL).
 */
#define MLPBLK_ORTHO_MAX_STEPS 16

typedef struct {
    int64_t rows, cols;
    int32_t batch;
    int32_t dtype;        /* of u (orthogonalize) or weight (muon_step)        */
    int32_t steps;
    float   eps;
    float   coefficients[MLPBLK_ORTHO_MAX_STEPS][3];   /* a, b, c of each step */
} mlpblk_ortho_desc;

typedef struct {
    float lr, momentum, weight_decay, scale;
    int32_t nesterov;
} mlpblk_muon;

size_t mlpblk_orthogonalize_workspace_size(const mlpblk_ortho_desc *desc);

int mlpblk_orthogonalize(const mlpblk_ortho_desc *desc, const void *u, void *o, void *workspace,
                         size_t workspace_bytes, void *stream);

int mlpblk_muon_step(const mlpblk_ortho_desc *desc, const mlpblk_muon *hp, float *master, void *weight,
                     const float *grad, float *momentum, const float *grad_scale, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * zero_grads() of the accumulation loop ("grow_a_language_model_backprop" --
 * accumulation across microbatches): dgamma[d], dw1[F,d], dw2[d,F] = 0 (float32).
 * desc->tokens is ignored.  Returns an MLPBLK_* code.
 */
int mlpblk_zero_grads(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2,
                      void *stream);

/*
 * scale_grads(s) of the same loop, e.g. s = 1/n_microbatches:
 * dgamma, dw1, dw2 *= s (float32, one rounding per element).  s must be finite.
 * desc->tokens is ignored.  Returns an MLPBLK_* code.
 */
int mlpblk_scale_grads(const mlpblk_desc *desc, float *dgamma, float *dw1, float *dw2,
                       float s, void *stream);

/*
 * First device-side error recorded since the previous call (MLPBLK_OK if none),
 * then clears it.  Synchronises the current device.  MLPBLK_ETIMEOUT means a
 * kernel's bounded wait on a pipeline barrier gave up and the kernel returned
 * early: its outputs are not valid.
 */
int mlpblk_last_error(void);

/*
 * RMSNorm backward with the residual gradient, for callers that cannot give
 * the library any device scratch memory.  The paper has no counterpart to this
 * entry point: it is the row kernel of mlpblk_backward offered on its own.
 *
 * Who needs it: code that runs inside a host engine which owns all device
 * memory and plans every buffer once at start-up, and gives its extensions no
 * way to allocate (a cudaMalloc there breaks the memory plan and can fail with
 * out-of-memory in the middle of a step); and code on threads that must not
 * stall on the implicit device synchronisation cudaMalloc and cudaFree can
 * cause.  This call allocates nothing: no cudaMalloc, no cudaFree, no
 * allocating library routine.  Its scratch (the per-block dgamma partial sums)
 * is a fixed 4 MiB array inside the library, held by every GPU that loads the
 * library until the process exits.
 *
 *   in : x[T,d], dy[T,d], gamma[d] (desc->dtype), dn[T,d] float32 = the gradient
 *        of the normalised output n = x * r * gamma, rstd[T] float32 = r
 *   out: dx[T,d]     = dy + r * (g - xh * mean_k(g * xh)),  xh = x*r, g = dn*gamma
 *                                                                        (written)
 *        dgamma[d]  += sum_t dn[t,k] * xh[t,k]                float32 (accumulated)
 * Limits: d_model a multiple of 8 and at most 4096 (MLPBLK_ENOTSUP beyond: one
 * partial row must fit the array); any tokens >= 0 (rows are indexed in 64
 * bits; at most min(512, 1048576 / d_model) partial rows are used, and with
 * more tokens each partial row sums more of them).
 * desc->ffn and desc->eps are not used.
 *
 * Set-up: the first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current, so make one call on every
 * device before capturing any stream of that device into a CUDA graph.  Host
 * threads may make a device's first call at the same time (each finds the same
 * address).  Every call also queries the current device, its SM count and the
 * row kernel's occupancy on the host; these enqueue nothing.
 * Every call in a process shares the one array of a device, and each call
 * overwrites the part it reads, so nothing needs clearing; but calls that
 * overlap on the GPU (on other streams, from other threads) race on it and
 * must be serialised by the caller.  Another process has an array of its own.  Pointers are device pointers, 16-byte
 * aligned.  Returns an MLPBLK_* code.
 */
int mlpblk_rmsnorm_backward_noalloc(const mlpblk_desc *desc, const void *x, const float *dn,
                                    const void *dy, const void *gamma, const float *rstd,
                                    void *dx, float *dgamma, void *stream);

/*
 * Kernel timing hook for profiling harnesses (CUDA events, no profiler needed).
 * Kinds reported for each kernel launch the library makes:
 */
#define MLPBLK_KERNEL_FOLD_GAMMA      1  /* statistics pass: rstd, W1g = W1 * gamma;
                                            mlpblk_fold_weights: W1g alone           */
#define MLPBLK_KERNEL_GEMM_FWD_W1     2  /* h, a = RMSNorm(x) . W1^T, relu^2         */
#define MLPBLK_KERNEL_GEMM_FWD_W2     3  /* y = x + a . W2^T                          */
#define MLPBLK_KERNEL_GEMM_DGRAD_H    4  /* dh = (dy . W2) * 2 relu(h)                */
#define MLPBLK_KERNEL_GEMM_WGRAD_W2   5  /* dW2 += dy^T . a                           */
#define MLPBLK_KERNEL_GEMM_DGRAD_N    6  /* dn = dh . W1                              */
#define MLPBLK_KERNEL_GEMM_WGRAD_W1   7  /* dW1 += dh^T . n                           */
#define MLPBLK_KERNEL_NORM_BWD        8  /* RMSNorm backward + residual, dgamma parts */
#define MLPBLK_KERNEL_DGAMMA_REDUCE   9  /* dgamma += sum of parts                    */
#define MLPBLK_KERNEL_ZERO_GRADS     10
#define MLPBLK_KERNEL_SCALE_GRADS    11
#define MLPBLK_KERNEL_RSTD           12  /* statistics pass alone: rstd (prefolded)   */
#define MLPBLK_KERNEL_GRAD_NORM      13  /* per-CTA partial sums of g^2               */
#define MLPBLK_KERNEL_CLIP_GRADS     14  /* g *= clip scale (device scalar)           */
#define MLPBLK_KERNEL_ADAMW          15  /* fused AdamW update                        */
#define MLPBLK_KERNEL_GRAD_NORM_FINAL 16 /* partials -> norm and clip scale           */
#define MLPBLK_KERNEL_QUANT_AMAX     17  /* E4M3: per-CTA maxima of |v|               */
#define MLPBLK_KERNEL_QUANT_SCALE    18  /* E4M3: amax -> scale record                */
#define MLPBLK_KERNEL_QUANT_APPLY    19  /* E4M3: v -> codes                          */
#define MLPBLK_KERNEL_NORM_QUANT     20  /* E4M3: rstd and n' = x * rstd              */
#define MLPBLK_KERNEL_MOE_ROUTE      21  /* experts: counts, segments, ranks, row map */
#define MLPBLK_KERNEL_MOE_GATHER     22  /* experts: rows in segment order            */
#define MLPBLK_KERNEL_MOE_COMBINE    23  /* experts: y = x + weighted outputs         */
#define MLPBLK_KERNEL_MOE_DP         24  /* experts: d_routing_weights and p * dy     */
#define MLPBLK_KERNEL_MOE_SCATTER    25  /* reserved (dn's slot sum is in NORM_BWD)   */
#define MLPBLK_KERNEL_SORT           26  /* mlpblk_moe_sort: the plan                 */
#define MLPBLK_KERNEL_PERMUTE        27  /* rows into sorted order                    */
#define MLPBLK_KERNEL_UNPERMUTE      28  /* rows back per token (and permute's dx)    */
#define MLPBLK_KERNEL_UNPERMUTE_BWD  29  /* d_rows, d_weights                         */
#define MLPBLK_KERNEL_FP4_QUANT      30  /* MXFP4: v -> codes and scales              */
#define MLPBLK_KERNEL_FP4_DEQUANT    31  /* MXFP4: codes and scales -> v              */
#define MLPBLK_KERNEL_FP4_GEMM       32  /* MXFP4 product, dense or grouped           */
#define MLPBLK_KERNEL_ROUTE          33  /* mlpblk_moe_route                          */
#define MLPBLK_KERNEL_ROUTE_BWD      34  /* mlpblk_moe_route_backward                 */
#define MLPBLK_KERNEL_ADD_NORM       35  /* mlpblk_add_rmsnorm                        */
#define MLPBLK_KERNEL_ADD_NORM_BWD   36  /* mlpblk_add_rmsnorm_backward: dx, dgamma parts */
#define MLPBLK_KERNEL_ADD_NORM_DG    37  /* its dgamma from the parts                 */
#define MLPBLK_KERNEL_ORTHO_NORM     38  /* |u|'s partial sums (momentum on the way)   */
#define MLPBLK_KERNEL_ORTHO_SCALE    39  /* X = u / (|u| + eps)                       */
#define MLPBLK_KERNEL_NS_GRAM        40  /* G = X X^T                                 */
#define MLPBLK_KERNEL_NS_SQUARE      41  /* P = b G + c G^2                           */
#define MLPBLK_KERNEL_NS_UPDATE      42  /* X = a X + P X                             */
#define MLPBLK_KERNEL_MUON_APPLY     43  /* master, weight                            */
#define MLPBLK_KERNEL_NS_APPLY       44  /* Y = a Y + P Y (two steps at a time)       */
#define MLPBLK_KERNEL_NS_JOIN        45  /* the polynomial of two steps               */
#define MLPBLK_KERNEL_NS_STEPS       46  /* every step of small matrices              */

/*
 * mlpblk_trace_begin: from now on, launch i of this library records
 * events[2i] on its stream just before the kernel and events[2i+1] just after
 * it, and stores its MLPBLK_KERNEL_* kind in kinds[i], for i < capacity; later
 * launches are not recorded.  events (2*capacity cudaEvent_t handles created by
 * the caller) and kinds (capacity ints, host memory) stay owned by the caller
 * and must outlive the trace.  One trace at a time per process; not
 * thread-safe.  Returns MLPBLK_EINVAL for NULL arrays or capacity < 1.
 * mlpblk_trace_end: stops recording and returns how many launches were
 * recorded (may exceed capacity: the launches beyond it were only counted).
 */
int mlpblk_trace_begin(void **events, int *kinds, int capacity);
int mlpblk_trace_end(void);

/*
 * Failure-detection test hook.  MLPBLK_TEST_FAULT_SKIP_LOADS makes the W1 GEMM
 * of the next bf16 mlpblk_forward issue none of its operand loads: its pipeline
 * waits then run out after their bound (about 2 s), the kernel unwinds (TMEM
 * freed, no trap) and MLPBLK_ETIMEOUT is recorded for mlpblk_last_error(); that
 * forward's outputs are not valid, and the context stays usable.  One-shot; not
 * thread-safe.  Returns MLPBLK_EINVAL for an unknown fault.
 */
#define MLPBLK_RMSNORM_STATS_PASS      0
#define MLPBLK_RMSNORM_IN_W1_PROLOGUE  1
/*
 * Where the bf16 forward computes the RMSNorm statistic rstd[t] ("Setup: The
 * Shared Transformer Shell": the norm feeds the W1 projection):
 *   MLPBLK_RMSNORM_STATS_PASS (default): one HBM pass over x ahead of the W1
 *     GEMM computes rstd and, in the same launch, W1*gamma; the GEMM applies
 *     rstd in its epilogue and runs 256 x 256 pair tiles.
 *   MLPBLK_RMSNORM_IN_W1_PROLOGUE: four extra warps of the W1 GEMM sum x^2 per
 *     row from the x tiles already staged in shared memory for the MMAs (no
 *     extra pass over x; W1*gamma still takes one pass over W1).  Whole-tile
 *     schedule only (every tile needs all of K for its rows' sums).
 * Same results up to float32 summation order.  Process-wide; applies to later
 * mlpblk_forward calls (the recompute variant always uses the statistics
 * pass).  Returns MLPBLK_EINVAL for an unknown mode.
 */
int mlpblk_set_rmsnorm_mode(int mode);

#define MLPBLK_TEST_FAULT_NONE        0
#define MLPBLK_TEST_FAULT_SKIP_LOADS  1
int mlpblk_set_test_fault(int fault);

/* The CUDA runtime's message for the most recent failing CUDA call made inside
 * the library (behind an MLPBLK_ECUDA), or "no CUDA error recorded". */
const char *mlpblk_cuda_error_string(void);

/* Static, NUL-terminated description of an MLPBLK_* code. */
const char *mlpblk_strerror(int code);

/* ABI version (major * 100 + minor).  101: mlpblk_fp4_desc ends with source_rows, and a
 * gathering mlpblk_fp4_quantize needs it.  102: routing, add_rmsnorm, orthogonalize, muon_step. */
int mlpblk_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLPBLK_H */
