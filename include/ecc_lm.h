/*
 * ecc_lm.h -- C ABI of the language-model operators that stand next to the
 * coders of ecc.h: they make the e4m3 and BF16 tensors the coders take
 * (activations of a layer norm or a matrix product, gradients), multiply the
 * bytes a decoder returns, and give a model's own code lengths (token log
 * probabilities; -log2 p bits is the ideal length of a token, the entropy the
 * ideal rate, as ecc_entropy_bits is for bytes), and update a model's
 * parameters, with moments in bytes that the coders take.
 *
 * Conventions: those of ecc.h (status returns, caller-owned device memory and
 * workspaces, work only enqueued on `stream`, nothing kept between calls),
 * and
 *  - matrices are row-major with a leading dimension `ld` in elements, at
 *    least the number of columns; the elements of a row are contiguous.
 *    Pointers and leading dimensions need the alignment of one element only;
 *    16-byte aligned rows take the fast paths;
 *  - element types are ECC_F32, ECC_BF16, ECC_F16 and ECC_E4M3 (OCP E4M3FN
 *    bytes: bias 7, largest value 448, no infinities);
 *  - sums, statistics and products are held in float32; a value is rounded
 *    once, to nearest even, when it is stored.  A stored e4m3 byte holds
 *    value * y_scale, saturated to +-448, NaN kept;
 *  - the tensor cores' additions truncate: a sum of K products of a matrix
 *    product, float32 outputs' too, is off by up to (K + 8) 2^-23 of the sum of
 *    their magnitudes (K = 3464: 4e-6 of the outputs' size on average);
 *  - outputs never depend on the order in which blocks run: the same call on
 *    the same inputs gives the same bits;
 *  - an output may not overlap an input unless the entry says so;
 *  - the elements between a row's end and the next row's start may be read
 *    (their values change nothing); they are never written;
 *  - a count of zero rows is valid: nothing is read, sums over rows are zero.
 */
#ifndef ECC_LM_H
#define ECC_LM_H

#include "ecc.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { ECC_F32 = 0, ECC_BF16 = 1, ECC_F16 = 2, ECC_E4M3 = 3 };

/* Activations: identity, max(a, 0), a Phi(a) (the exact erf form),
 * a (1 + tanh(sqrt(2/pi) (a + 0.044715 a^3))) / 2, a / (1 + e^-a).  Phi is
 * computed to an absolute 1.5e-7 (which is a relative 2e-3 of it at a = -5 and
 * 1e-2 at -8), the exponentials to a relative 2^-22 (1 + |argument|). */
enum { ECC_ACT_NONE = 0, ECC_ACT_RELU = 1, ECC_ACT_GELU = 2, ECC_ACT_GELU_TANH = 3, ECC_ACT_SILU = 4 };

/*
 * ecc_layer_norm -- y = (x - mean) * rstd * weight + bias for each row, with
 * mean and rstd = 1 / sqrt(var + eps) over the row's columns (var is the mean
 * square deviation from the mean, summed in a second pass over the row).
 *   x       [rows, cols] of x_type (F32, BF16 or F16), leading dimension ldx.
 *   weight, bias  [cols] of p_type (x_type or F32); NULL = ones / zeros.
 *   y       [rows, cols] of y_type (x_type or E4M3), leading dimension ldy;
 *           may be x itself (same type and leading dimension).
 *   y_scale factor of an e4m3 output; must be 1 for the other types.
 *   mean, rstd  float32[rows], or NULL if not wanted.
 * Errors: ECC_ERR_ARG (no columns, a NULL or misaligned pointer, ld below
 * cols, a type not listed, eps negative or not finite), ECC_ERR_CUDA.
 */
ecc_status ecc_layer_norm(const void *x, uint64_t ldx, uint32_t x_type, const void *weight, const void *bias,
                          uint32_t p_type, uint64_t rows, uint64_t cols, float eps, void *y, uint64_t ldy,
                          uint32_t y_type, float y_scale, float *mean, float *rstd, void *stream);

/*
 * ecc_layer_norm_grad -- the backward pass.  With xh = (x - mean) * rstd and
 * g = dy * weight: dx = rstd * (g - avg(g) - xh * avg(g * xh)) (averages over
 * the row), dweight = sum over rows of dy * xh, dbias = sum over rows of dy.
 *   dy, x, dx   [rows, cols] of `type` (F32, BF16 or F16); dx may be dy or x
 *               (same leading dimension), or NULL if not wanted.
 *   weight      [cols] of p_type, NULL = ones; mean, rstd as written by
 *               ecc_layer_norm.
 *   dweight, dbias  float32[cols], written; NULL if not wanted.
 *   ws          16-byte aligned scratch of
 *               ecc_layer_norm_grad_workspace_bytes(rows, cols) bytes.
 * Errors: as ecc_layer_norm, and ECC_ERR_ARG for a small workspace.
 */
size_t ecc_layer_norm_grad_workspace_bytes(uint64_t rows, uint64_t cols);
ecc_status ecc_layer_norm_grad(const void *dy, uint64_t lddy, const void *x, uint64_t ldx, uint32_t type,
                               const void *weight, uint32_t p_type, const float *mean, const float *rstd,
                               uint64_t rows, uint64_t cols, void *dx, uint64_t lddx, float *dweight, float *dbias,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * ecc_linear -- out = act(a) + residual, a = scale * x w^T + bias: a layer's
 * matrix product with its epilogue.
 *   x     [M, K], w [N, K] of in_type: BF16, F16, or E4M3 (the bytes a
 *         decoder returns; `scale` is then the product of their scales).
 *   bias  [N] of bias_type (F32, BF16, F16) or NULL.
 *   residual  [M, N] of res_type (F32, BF16, F16) or NULL.
 *   out   [M, N] of out_type (F32, BF16, F16, or E4M3 = out * out_scale;
 *         out_scale must be 1 for the other types); may be residual itself
 *         (same type and leading dimension).
 *   pre   [M, N] of pre_type (F32, BF16, F16): a, for the backward pass; or
 *         NULL.
 *   M, N, K  any, K = 0 giving a = bias.  M and N below 2^31, K below 2^31.
 *   ws    16-byte aligned scratch of ecc_linear_workspace_bytes(job) bytes
 *         (0 when the rows of x and w start on 16-byte boundaries, for single
 *         tokens of 16-bit types and for small products of up to four rows).
 *   status  device uint32[1]: ECC_OK, or ECC_ERR_TIMEOUT if a bounded wait of
 *         the kernel ran out (the output is then incomplete).
 * Errors: ECC_ERR_ARG, ECC_ERR_CUDA.
 */
typedef struct ecc_linear_job {
    const void *x, *w, *bias, *residual;
    void *out, *pre;
    uint64_t M, N, K;
    uint64_t ldx, ldw, ldres, ldout, ldpre;
    float scale, out_scale;
    uint32_t in_type, bias_type, res_type, out_type, pre_type, act;
} ecc_linear_job;

size_t ecc_linear_workspace_bytes(const ecc_linear_job *job);
ecc_status ecc_linear(const ecc_linear_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream);

/*
 * ecc_linear_grad -- the backward pass of ecc_linear's product: with
 * t = dy * act'(pre) (t = dy for ECC_ACT_NONE),
 *   dx = scale * t w, dw = scale * t^T x, dbias = sum over rows of t.
 * (The residual's gradient is dy itself.)
 *   dy    [M, N], x [M, K], w [N, K], dx [M, K] of in_type (BF16 or F16);
 *         pre [M, N] of pre_type (F32, BF16, F16), ignored for ECC_ACT_NONE.
 *   dw    [N, K] of dw_type (in_type or F32).
 *   dbias float32[N].
 *   dx, dw, dbias: NULL if not wanted (w is only read for dx, x for dw).
 *   t is rounded to in_type before the products (the tensor cores' operand);
 *   dbias sums it before that rounding.
 * ws, status and errors as for ecc_linear.
 */
typedef struct ecc_linear_grad_job {
    const void *dy, *x, *w, *pre;
    void *dx, *dw;
    float *dbias;
    uint64_t M, N, K;
    uint64_t lddy, ldx, ldw, ldpre, lddx, lddw;
    float scale;
    uint32_t in_type, pre_type, dw_type, act, reserved;
} ecc_linear_grad_job;

size_t ecc_linear_grad_workspace_bytes(const ecc_linear_grad_job *job);
ecc_status ecc_linear_grad(const ecc_linear_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status,
                           void *stream);

/*
 * ecc_gated_linear -- out = act(g) * u with g = scale * x w_gate^T + bias_gate
 * and u = up_scale * x w_up^T + bias_up: a gated feed-forward block's
 * projections, its activation and their product.
 *   x     [M, K], w_gate, w_up [N, K] of in_type: BF16, F16 or E4M3.
 *   bias_gate, bias_up  [N] of bias_type (F32, BF16, F16), each NULL if there
 *         is none.
 *   out   [M, N] of out_type (F32, BF16, F16, or E4M3 = out * out_scale;
 *         out_scale must be 1 for the other types).
 *   pre_gate, pre_up  [M, N] of pre_type (F32, BF16, F16): g and u, for the
 *         backward pass; or both NULL.
 * M, N, K, ws, status and errors as for ecc_linear (`reserved` is 0).
 */
typedef struct ecc_gated_linear_job {
    const void *x, *w_gate, *w_up, *bias_gate, *bias_up;
    void *out, *pre_gate, *pre_up;
    uint64_t M, N, K;
    uint64_t ldx, ldgate, ldup, ldout, ldpre_gate, ldpre_up;
    float scale, up_scale, out_scale;
    uint32_t in_type, bias_type, out_type, pre_type, act, reserved;
} ecc_gated_linear_job;

size_t ecc_gated_linear_workspace_bytes(const ecc_gated_linear_job *job);
ecc_status ecc_gated_linear(const ecc_gated_linear_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream);

/*
 * ecc_gated_linear_grad -- the backward pass: with tg = dy u act'(g) and tu =
 * dy act(g), g and u as kept in pre_gate and pre_up,
 *   dx = scale * tg w_gate + up_scale * tu w_up,
 *   dw_gate = scale * tg^T x, dw_up = up_scale * tu^T x,
 *   dbias_gate, dbias_up = sums over rows of tg, tu.
 *   dy    [M, N], x [M, K], w_gate, w_up [N, K], dx [M, K] of in_type (BF16 or
 *         F16); pre_gate, pre_up [M, N] of pre_type (F32, BF16, F16).
 *   dw_gate, dw_up  [N, K] of dw_type (in_type or F32), both or neither.
 *   dbias_gate, dbias_up  float32[N], both or neither.
 *   dx, dw_*, dbias_*: NULL if not wanted.
 *   tg and tu are rounded to in_type before the products; the dbias sums are
 *   taken before that.  BF16: each times its scale's share of the larger scale.
 *   F16: for dx the same, times a power of two that brings the largest finite
 *   value to 2^14; for the weights' gradients each as it is, times a power of
 *   two of its own that does (so that products dy u outside float16's range
 *   and scales far apart cost no bits; the workspace holds both forms).
 * ws, status and errors as for ecc_linear.
 */
typedef struct ecc_gated_linear_grad_job {
    const void *dy, *x, *w_gate, *w_up, *pre_gate, *pre_up;
    void *dx, *dw_gate, *dw_up;
    float *dbias_gate, *dbias_up;
    uint64_t M, N, K;
    uint64_t lddy, ldx, ldgate, ldup, ldpre_gate, ldpre_up, lddx, lddw_gate, lddw_up;
    float scale, up_scale;
    uint32_t in_type, pre_type, dw_type, act;
} ecc_gated_linear_grad_job;

size_t ecc_gated_linear_grad_workspace_bytes(const ecc_gated_linear_grad_job *job);
ecc_status ecc_gated_linear_grad(const ecc_gated_linear_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status,
                                 void *stream);

/*
 * ecc_token_logprob -- for each row z = scale * logits: the log partition
 * lse = log sum e^z, the given token's log probability z[token] - lse, the
 * entropy H = -sum p log p (p log p = 0 where p = 0) and the `top` most
 * probable tokens with their log probabilities, in nats.
 *   logits  [rows, vocab] of `type` (F32, BF16, F16), leading dimension ld.
 *   tokens  int64[rows], or NULL.  A negative token means none: its log
 *           probability is 0.  A token >= vocab gets NaN.
 *   scale   > 0, below 2^127 (the reciprocal of a temperature).
 *   logprob, entropy, lse  float32[rows]; logprob is not written without
 *           tokens; each may be NULL.
 *   top     0..32 and at most vocab; top_logprob float32[rows, top],
 *           top_index int32[rows, top]: larger logits first, equal ones by
 *           the lower index (-0 equals +0), NaN before everything.
 * A logit of -infinity is a token without probability.  A row of nothing
 * else has lse and every log probability -infinity and entropy 0.  A row
 * with a NaN has NaN results; a row with +infinity has lse = +infinity and
 * entropy NaN.  Where scale * logits leaves float32's range lse does too
 * (+-infinity); the log probabilities and the entropy are those of the values
 * all the same.
 * Errors: ECC_ERR_ARG (no columns, vocab >= 2^31, ...), ECC_ERR_CUDA.
 */
#define ECC_MAX_TOP 32
ecc_status ecc_token_logprob(const void *logits, uint64_t ld, uint32_t type, const int64_t *tokens, uint64_t rows,
                             uint64_t vocab, float scale, uint32_t top, float *logprob, float *entropy, float *lse,
                             float *top_logprob, int32_t *top_index, void *stream);

/*
 * ecc_token_logprob_grad -- the gradient of sum over rows of
 * dlogprob * logprob + dentropy * entropy with respect to the logits:
 *   dlogits = scale * (dlogprob (1[v = token] - p) - dentropy p (log p + H)),
 * p = e^(z - lse), the second term 0 where p = 0.
 *   lse, entropy  as written by ecc_token_logprob for the same logits and
 *           scale (not joined from several calls: where |lse| is above 256,
 *           too large for its float32 rounding not to show, the row's maximum
 *           and log sum are found again, at two more reads of the row);
 *           entropy may be NULL if dentropy is.
 *   dlogprob, dentropy  float32[rows]; NULL = zeros.  Rows whose token is
 *           negative or >= vocab take no part in dlogprob; a row of -infinity
 *           only has gradient 0, one with a NaN or +infinity has gradient NaN.
 *   dlogits [rows, vocab] of `type`, leading dimension ldd; may be logits
 *           itself (ldd = ld).
 * Errors: ECC_ERR_ARG, ECC_ERR_CUDA.
 */
ecc_status ecc_token_logprob_grad(const void *logits, uint64_t ld, uint32_t type, const int64_t *tokens,
                                  uint64_t rows, uint64_t vocab, float scale, const float *lse,
                                  const float *entropy, const float *dlogprob, const float *dentropy, void *dlogits,
                                  uint64_t ldd, void *stream);

/*
 * ecc_linear_logprob -- what ecc_token_logprob gives of z = scale * x w^T (a
 * head's logits), which are never stored: the log partition lse, the entropy
 * and the given token's log probability of each row, from float32 logits.
 *   x     [rows, K], w [vocab, K] of in_type: BF16, F16 or E4M3.
 *   tokens  int64[rows], or NULL.  A negative token means none: its log
 *         probability is 0.  A token >= vocab gets NaN.
 *   logprob, entropy, lse  float32[rows]; logprob is not written without
 *         tokens; each may be NULL.
 *   A row with a logit that is not finite has NaN results.  Exponentials are
 *   computed to a relative 2^-22 (1 + |argument|); a logit's products are summed
 *   by the tensor cores in accumulators of 512 (E4M3 1024) or, for few tokens, up
 *   to a quarter of K, whose additions truncate, and those in float32.
 *   ws    16-byte aligned scratch of ecc_linear_logprob_workspace_bytes(job)
 *         bytes (16 bytes a row for each share of the vocabulary, which is 128
 *         tokens or fewer for small products, and copies of x and w whose rows
 *         are not on 16-byte boundaries).
 * vocab from 1 to 2^31 - 1, rows and K below 2^31; K = 0 gives logits of 0.
 * scale of any sign, its magnitude below 2^127 (here and in the gradient).
 * status and errors as for ecc_linear (`reserved` is 0).
 */
typedef struct ecc_linear_logprob_job {
    const void *x, *w;
    const int64_t *tokens;
    float *logprob, *entropy, *lse;
    uint64_t rows, vocab, K, ldx, ldw;
    float scale;
    uint32_t in_type, reserved;
} ecc_linear_logprob_job;

size_t ecc_linear_logprob_workspace_bytes(const ecc_linear_logprob_job *job);
ecc_status ecc_linear_logprob(const ecc_linear_logprob_job *job, void *ws, size_t ws_bytes, uint32_t *status, void *stream);

/*
 * ecc_linear_logprob_grad -- the gradient of sum over rows of dlogprob * logprob
 * + dentropy * entropy: with
 *   t = dlogprob (1[v = token] - p) - dentropy p (log p + H), p = e^(z - lse),
 *   dx = scale * t w, dw = scale * t^T x.
 * The logits are computed again, a piece of the vocabulary at a time.
 *   x [rows, K], w [vocab, K], dx [rows, K] of in_type (BF16 or F16).
 *   lse, entropy  as written by ecc_linear_logprob for the same x and w (lse's
 *         rounding is p's relative error: 2^-24 |lse|); entropy may be NULL
 *         if dentropy is.
 *   dlogprob, dentropy  float32[rows]; NULL = zeros.  Rows whose token is
 *         negative or >= vocab take no part in dlogprob.
 *   dw    [vocab, K] of dw_type (in_type or F32).
 *   dx, dw: NULL if not wanted.
 *   t is rounded to in_type before the products; with F16 the largest finite
 *   dlogprob (of rows with a token) and dentropy give a power of two that
 *   keeps small probabilities in its range.
 *   ws    16-byte aligned scratch of ecc_linear_logprob_grad_workspace_bytes(job)
 *         bytes (t of a piece, at most 256 MiB or 512 bytes a row, dx's sum
 *         over the pieces, copies as above).
 * status and errors as for ecc_linear (`reserved` is 0).
 */
typedef struct ecc_linear_logprob_grad_job {
    const void *x, *w;
    const int64_t *tokens;
    const float *lse, *entropy, *dlogprob, *dentropy;
    void *dx, *dw;
    uint64_t rows, vocab, K, ldx, ldw, lddx, lddw;
    float scale;
    uint32_t in_type, dw_type, reserved;
} ecc_linear_logprob_grad_job;

size_t ecc_linear_logprob_grad_workspace_bytes(const ecc_linear_logprob_grad_job *job);
ecc_status ecc_linear_logprob_grad(const ecc_linear_logprob_grad_job *job, void *ws, size_t ws_bytes, uint32_t *status,
                                   void *stream);

/*
 * ecc_adamw -- one step of AdamW over many tensors at once.  With g =
 * grad_scale * grad, t = step:
 *   m = beta1 m + (1 - beta1) g, v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * in float32, with m and v as they are before they are stored (the quotient's
 * root and reciprocal to a relative 2^-22).
 *   param   [n] of param_type, grad [n] of grad_type (F32, BF16 or F16).
 *   master  float32[n] or NULL: with it, p is read from and written to it,
 *           and param receives its rounding.
 *   m, v    by state_type: ECC_F32, float32[n] of the moments, or ECC_E4M3,
 *           bytes[n] with a scale for each ECC_ADAMW_GROUP values (the last
 *           group may be shorter): m = m_scale * byte, sqrt(v) = v_scale *
 *           byte, scale = largest magnitude of the group / 448.  A value is
 *           stored as one of its two e4m3 neighbours, the upper one with the
 *           probability that its distance from the lower one is of theirs (so
 *           that the mean of many steps is kept, where rounding to nearest
 *           would never take a step smaller than half their distance), but a
 *           positive v is at least the smallest positive code.  The random bits of
 *           value i are mix((i mod 2^32) ^ mix(mix(mix(seed) + step) + i /
 *           2^32)), the upper 16 for m, the lower for v, with mix(x): x ^= x >> 16,
 *           x *= 0x7FEB352D, x ^= x >> 15, x *= 0x846CA68B, x ^= x >> 16 in 32
 *           bits (a mixing published by C. Wellons, "Prospecting for Hash
 *           Functions", 2018): the same call gives the same bytes, and equal
 *           places of a call's tensors have the same random bits (each value's
 *           mean is kept all the same; calls with seeds of their own keep
 *           tensors' roundings apart).  A root is off by 4% a step on
 *           average, and the errors of 1 / (1 - beta2) steps add up: at beta2 =
 *           0.95 to a sixth, at 0.999 to more than the root, which wants float32
 *           states.  A group with a NaN or an infinity gets scales of NaN, and
 *           one of magnitudes below 2^-119 (1.5e-36) zeros.
 *   eps     0, or any positive number; below 2^-126 it counts as that.
 *   step    1 for the first.  step_at, lr_at, grad_scale_at: device int64 and
 *           float32 read by the kernel in place of step, lr and grad_scale (for
 *           a captured step that is replayed), or NULL.
 * All arrays contiguous, aligned to an element; none that is written may
 * overlap another one of the job (gradients and what step_at, lr_at and
 * grad_scale_at point to included).  Tensors with n = 0 are passed over.
 * Errors: ECC_ERR_ARG (a NULL or misaligned pointer, overlapping arrays, a
 * type not listed, n >= 2^40, beta outside [0, 1), eps below 0, a value that is
 * not finite in float32, step = 0), ECC_ERR_CUDA.
 */
#define ECC_ADAMW_GROUP 256
typedef struct ecc_adamw_tensor {
    void *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale, *master;
    uint64_t n;
    uint32_t param_type, grad_type, state_type, reserved;
} ecc_adamw_tensor;
typedef struct ecc_adamw_job {
    const ecc_adamw_tensor *tensors;
    uint64_t count;
    double lr, beta1, beta2, eps, weight_decay, grad_scale;
    uint64_t step;
    const int64_t *step_at;
    const float *lr_at, *grad_scale_at;
    uint32_t seed, reserved;
} ecc_adamw_job;
ecc_status ecc_adamw(const ecc_adamw_job *job, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ECC_LM_H */
