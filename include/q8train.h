/*
 * q8train.h -- C ABI of the training-step operators that make the gradients
 * the optimizer steps of q8adamw.h consume, on one GB300 (sm_103a):
 *  - the gated feed-forward product (both projections, the activation and the
 *    product), forward and backward;
 *  - the norms after a block and before the next one, fused with the block's
 *    gate and the residual scale, forward and backward;
 *  - distillation from a teacher's top logits, forward and backward;
 *  - the token embedding: lookup with a scale, and the gradient of its table;
 * and what stands between the backward pass and those steps:
 *  - the norm of all gradients, and their clipping.
 *
 * The conventions of q8adamw.h hold (device pointers owned by the caller, BF16
 * as 16-bit patterns, asynchronous work on `stream`, negative q8_status on
 * argument errors with nothing launched, q8_last_error()), and these:
 *  - A matrix is row-major with unit stride along its rows; `*_stride` is the
 *    distance between consecutive rows in elements, at least the row's length.
 *    Any stride, any size and any base address of the element's own alignment
 *    is accepted; 16-byte aligned bases and strides that are a multiple of 16
 *    bytes are faster.
 *  - Outputs must not overlap inputs or one another unless stated.
 *  - Every output element is one fp32 result rounded once to its type (to
 *    nearest even).  Sums, statistics and accumulators are fp32.  No atomics:
 *    the same call on the same inputs gives the same bits.
 *  - A workspace is device memory of the stated size, 256-byte aligned, whose
 *    contents mean nothing before or after the call.  Calls that may run at
 *    the same time (on different streams) need different workspaces.
 *  - NaN and infinite inputs give what the formulas give where stated, and
 *    unspecified values (never a fault) elsewhere.
 */
#ifndef Q8TRAIN_H
#define Q8TRAIN_H

#include <stdint.h>

#include "q8adamw.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { Q8_BF16 = 0, Q8_F32 = 1 } q8_dtype;

/* ------------------------------------------------- gated feed-forward product
 *
 * With x [tokens, d_model], w_gate and w_up [d_ff, d_model] (rows contiguous,
 * as torch.nn.Linear keeps them), all bf16:
 *   g = x w_gate^T,  u = x w_up^T,  h = act(g) * u            [tokens, d_ff]
 * and for the gradient dh of h:
 *   dg = dh * u * act'(g),  du = dh * act(g)
 *   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x.
 * act: SiLU g*sigmoid(g); GELU in its tanh form
 * g/2*(1 + tanh(sqrt(2/pi)*(g + 0.044715 g^3))); GELU g*Phi(g).
 * g, u and h's product are fp32; dg and du are rounded to bf16 for the
 * products that make dx, dw_gate and dw_up (one rounding more than those
 * outputs' own).
 * 0 <= tokens, 1 <= d_model, 1 <= d_ff, each below 2^30.
 */
typedef enum { Q8_SILU = 0, Q8_GELU_TANH = 1, Q8_GELU = 2 } q8_activation;

typedef struct {
    const uint16_t* x;         /* [tokens, d_model], row stride x_stride     */
    const uint16_t* w_gate;    /* [d_ff, d_model] contiguous                 */
    const uint16_t* w_up;      /* [d_ff, d_model] contiguous                 */
    int64_t tokens, d_model, d_ff;
    int64_t x_stride;
    void* workspace;           /* at least q8_gated_ff_workspace() bytes     */
    int64_t workspace_bytes;
    int32_t act;               /* q8_activation                              */
} q8_gated_ff;

/* Bytes of workspace for a call with these sizes, strides and pointers
 * (workspace fields ignored); backward: 0 for the forward call, 1 for the
 * backward.  May be 0.  Negative: the q8_status of a bad argument. */
int64_t q8_gated_ff_workspace(const q8_gated_ff* ff, int backward);

/* h.  saved: NULL, or float[2 * tokens * d_ff] that receives g, then u, for
 * the backward call. */
int q8_gated_ff_forward(const q8_gated_ff* ff, uint16_t* h, int64_t h_stride, float* saved,
                        q8_stream_t stream);

/* dx, dw_gate, dw_up from dh.  saved: what the forward call wrote, or NULL to
 * compute g and u again (two more matrix products, no memory between the
 * calls).  Any of the three outputs may be NULL and is then not computed.
 * With tokens 0 the weights' gradients are zeros. */
int q8_gated_ff_backward(const q8_gated_ff* ff, const uint16_t* dh, int64_t dh_stride,
                         const float* saved, uint16_t* dx, int64_t dx_stride, uint16_t* dw_gate,
                         uint16_t* dw_up, q8_stream_t stream);

/* --------------------------------- norms around a block's gate and residual
 *
 * With the residual stream r and the block's output y, both [tokens, dim]:
 *   r' = residual_scale * r + gate * N_post(y),   z = N_pre(r')
 * where N is the identity (Q8_NORM_NONE), v / sqrt(mean(v^2) + eps) * w + b
 * (Q8_NORM_RMS) or (v - mean(v)) / sqrt(var(v) + eps) * w + b (Q8_NORM_LAYER,
 * var the mean squared deviation).  z is formed from r' before its rounding.
 * post_* is the norm after this block, pre_* the one before the next.
 * A NULL weight counts as ones, a NULL bias as zeros, a NULL gate as ones;
 * weights and biases of a Q8_NORM_NONE norm must be NULL.  gate has a row of
 * dim for every `gate_tokens` consecutive tokens (a learned channel gate has
 * gate_tokens = tokens, a gate for each token 1): ceil(tokens / gate_tokens)
 * rows, contiguous.  r, r' and their gradients have the type residual_dtype;
 * everything else is bf16.  r' may be written over r.
 * 0 <= tokens < 2^40, 1 <= dim <= Q8_NORM_MAX_DIM, eps >= 0 and finite,
 * residual_scale finite.
 */
typedef enum { Q8_NORM_NONE = 0, Q8_NORM_RMS = 1, Q8_NORM_LAYER = 2 } q8_norm_kind;

enum { Q8_NORM_MAX_DIM = 32768 };

typedef struct {
    const void* residual;          /* r, row stride residual_stride            */
    const uint16_t* y;             /* row stride y_stride                      */
    const uint16_t* post_weight;   /* [dim] or NULL, as the next four          */
    const uint16_t* post_bias;
    const uint16_t* pre_weight;
    const uint16_t* pre_bias;
    const uint16_t* gate;          /* [ceil(tokens / gate_tokens), dim] or NULL */
    int64_t tokens, dim, gate_tokens;
    int64_t residual_stride, y_stride;
    int32_t post_kind, pre_kind;   /* q8_norm_kind                             */
    int32_t residual_dtype;        /* q8_dtype                                 */
    float eps, residual_scale;
} q8_block_norm;

/* r' and z; either may be NULL (not written). */
int q8_block_norm_forward(const q8_block_norm* bn, void* residual_out, int64_t residual_out_stride,
                          uint16_t* z, int64_t z_stride, q8_stream_t stream);

/*
 * Gradients for dr' (type residual_dtype) and dz; either may be NULL (zeros).
 * The norms are computed again from r and y (as given to the forward call).
 * d_residual, d_y: row matrices with the given strides; the others contiguous
 * bf16 arrays shaped like what they are the gradient of, summed over all
 * tokens (d_gate: over its group's).  Any may be NULL (not computed), and must
 * be where there is nothing to take a gradient of (a Q8_NORM_NONE norm, a NULL
 * gate); the gradient of a NULL weight or bias is computed as for ones and
 * zeros.  d_residual may be written over d_residual_out, d_y over dz.
 */
typedef struct {
    const void* d_residual_out;
    const uint16_t* dz;
    void* d_residual;
    uint16_t* d_y;
    uint16_t* d_post_weight;
    uint16_t* d_post_bias;
    uint16_t* d_pre_weight;
    uint16_t* d_pre_bias;
    uint16_t* d_gate;
    int64_t d_residual_out_stride, dz_stride, d_residual_stride, d_y_stride;
    void* workspace;               /* at least q8_block_norm_workspace() bytes */
    int64_t workspace_bytes;
} q8_block_norm_grads;

/* Bytes of workspace of the backward call (it may be 0); negative: the
 * q8_status of a bad argument. */
int64_t q8_block_norm_workspace(const q8_block_norm* bn, const q8_block_norm_grads* g);

int q8_block_norm_backward(const q8_block_norm* bn, const q8_block_norm_grads* g, q8_stream_t stream);

/* ------------------------------------ distillation from a teacher's top logits
 *
 * For each row with student logits s [vocab], teacher entries (id_k, t_k),
 * k < K, and a label:
 *   p = softmax(t / tau) over the row's valid entries (0 <= id_k < vocab)
 *   q = softmax(s / tau)
 *   loss = kd_weight * tau^2 * sum_k p_k (log p_k - log q[id_k])
 *          + ce_weight * (logsumexp(s) - s[label])
 *   d loss / d s_j = kd_weight * tau * (q_j - sum of p_k with id_k = j)
 *                    + ce_weight * (softmax(s)_j - [j = label])
 * An entry whose id lies outside [0, vocab) is padding.  A row without valid
 * entries (or K = 0) has no first term, one whose label lies outside
 * [0, vocab) no second: neither adds to its loss or gradient, and a row with
 * neither has loss 0 and a zero gradient.  An id that appears twice counts
 * twice.  An entry whose p_k is 0 in fp32 (a teacher logit of -inf, or one some
 * 104 tau below the largest) adds nothing; a student
 * logit of -inf has q_j = 0 (a row all of whose logits are -inf, or with NaN
 * or +inf among them, gives NaN).
 * labels NULL: no row has a label.  A term of weight 0 is not computed.
 * 0 <= rows, 1 <= vocab < 2^31, 0 <= k <= Q8_DISTILL_MAX_K; temperature
 * finite and > 0; weights finite and >= 0.
 */
enum { Q8_DISTILL_MAX_K = 1024 };

typedef struct {
    const void* logits;            /* [rows, vocab], type logits_dtype         */
    const int64_t* teacher_ids;    /* [rows, k] contiguous; may be NULL if k = 0 */
    const float* teacher_logits;   /* [rows, k] contiguous                     */
    const int64_t* labels;         /* [rows] or NULL                           */
    const float* row_weight;       /* [rows] or NULL (ones): see below         */
    int64_t rows, vocab, k;
    int64_t logits_stride;
    int32_t logits_dtype;          /* q8_dtype                                 */
    float temperature, kd_weight, ce_weight;
} q8_distill_topk;

/*
 * loss: float[rows], the unweighted losses.  stats: NULL, or float[rows * 2]
 * that receives each row's logsumexp(s) and logsumexp(s / tau) (0 for a term
 * of weight 0) for the backward call.  dlogits: NULL, or the gradient of
 * sum_t row_weight[t] * loss[t], of the logits' type, written in the same call
 * (the logits are then read from memory once); it may be the logits
 * themselves.
 */
int q8_distill_topk_forward(const q8_distill_topk* d, float* loss, float* stats, void* dlogits,
                            int64_t dlogits_stride, q8_stream_t stream);

/* dlogits alone, from the forward call's stats; row_weight is the gradient of
 * the losses.  dlogits may be the logits themselves.  A logsumexp is one rounded
 * float, so that q_j and softmax(s)_j are off by about |logsumexp| * 2^-24 of
 * themselves (logits over tau in the hundreds: some 2^-16); the forward call's
 * own dlogits works relative to the row's maximum and is not. */
int q8_distill_topk_backward(const q8_distill_topk* d, const float* stats, void* dlogits,
                             int64_t dlogits_stride, q8_stream_t stream);

/* ----------------------------------------------------------- token embedding
 *
 * With a table W [vocab, dim] (bf16, contiguous, as torch.nn.Embedding keeps
 * it) and a token id for each of `tokens` rows:
 *   out[t] = scale * W[ids[t]]                                  [tokens, dim]
 * and for the gradient dout of out:
 *   dW[v] = scale * (sum of dout[t] over the t with ids[t] = v)  [vocab, dim].
 * An id outside [0, vocab) is no token: its row of out is zeros, and its row of
 * dout is not read.  out and dout have the type dtype.  The sum of a table row
 * is fp32, over the tokens' order in an association that depends on the ids and
 * the sizes alone.
 * 0 <= tokens < 2^30, 1 <= vocab < 2^31, 1 <= dim < 2^30, scale finite.
 */
typedef struct {
    const int64_t* ids;        /* [tokens]                                   */
    int64_t tokens, vocab, dim;
    int32_t dtype;             /* q8_dtype                                   */
    float scale;
} q8_embedding;

int q8_embedding_forward(const q8_embedding* e, const uint16_t* table, void* out, int64_t out_stride,
                         q8_stream_t stream);

/* Bytes of workspace of the backward call (it may be 0); negative: the
 * q8_status of a bad argument. */
int64_t q8_embedding_workspace(const q8_embedding* e);

/* accumulate 0: all of dtable is written, zeros in rows that no token has.
 * accumulate 1: the sums are added to what dtable holds (a table that is also
 * the output layer's weight, or a further micro-batch; one rounding of each
 * result), and rows that no token has are neither read nor written. */
int q8_embedding_backward(const q8_embedding* e, const void* dout, int64_t dout_stride, uint16_t* dtable,
                          int accumulate, void* workspace, int64_t workspace_bytes, q8_stream_t stream);

/* --------------------------------------- norm of all gradients, and clipping
 *
 * Over a list of `count` gradients g_i (host array), as one flat vector:
 *   norm = sqrt(sum over i, j of g_ij^2)
 *   c = min(1, max_norm / (norm + 1e-6)),  out_ij = c * g_ij.
 * Squares are summed in fp32 over at most 64 elements, scaled by a power of
 * two where they would leave fp32's range, these sums in pairs of fp32 (or
 * double) and those of the CTAs as whole numbers: no norm below 2^128 overflows,
 * none is lost, and beyond the 64 terms' roundings the norm carries two roundings
 * of fp32 and c five, of up to 2^27 tensors and 2^34 elements in all.  With an
 * infinite gradient the norm is infinite and c is 0 (infinite elements then give
 * NaN); with NaN both are NaN and all results are.
 * grad and out are contiguous, on their elements' own alignment; out may be
 * grad itself where both have one type, and out_dtype may differ from
 * grad_dtype elsewhere.  An out that overlaps another entry's out or grad, or its
 * own grad in another way, is refused (the same tensor twice, in place): entries
 * are clipped in no order.  Clipping in place with c = 1 writes nothing.
 * numel 0 entries are skipped.  0 <= count, 0 <= numel < 2^40; max_norm >= 0
 * (it may be infinite: c is then 1 or NaN).
 */
typedef struct {
    const void* grad;
    void* out;                 /* q8_grad_norm: not used                     */
    int64_t numel;
    int32_t grad_dtype;        /* q8_dtype                                   */
    int32_t out_dtype;         /* q8_dtype; q8_grad_norm: not used           */
} q8_grad;

/* Bytes of workspace of either call on a list of `count` entries; negative:
 * the q8_status of a bad argument. */
int64_t q8_grad_norm_workspace(int count);

/* norm: device float[1]. */
int q8_grad_norm(const q8_grad* list, int count, float* norm, void* workspace, int64_t workspace_bytes,
                 q8_stream_t stream);

/* norm: device float[1], the norm before clipping.  Nothing synchronises with
 * the host: c is formed on the device. */
int q8_clip_grads(const q8_grad* list, int count, double max_norm, float* norm, void* workspace,
                  int64_t workspace_bytes, q8_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* Q8TRAIN_H */
