/*
 * poetx_model.h - the operators of libpoetx.so that stand around a POET-X
 * layer in a language model: the RMS norm of the residual stream before it
 * (training, or with int8 rows out for serving), the int8 product that
 * serves a merged quantised layer, and the vocabulary cross entropy behind
 * the last layer, with its gradient and without keeping the logits.
 *
 * The conventions of poetx.h hold here too: device pointers owned by the
 * caller, everything asynchronous and ordered on `stream`, arguments
 * validated before any launch (nothing is launched and no output touched on
 * an error), status codes and dtypes of poetx.h, scratch memory from the
 * caller, no state kept between calls, steps visible in the timing log.
 *
 *  - Matrices are row-major. A row stride `ld` is in elements; a row of `cols`
 *    elements needs ld >= cols, and every row has to start on a 16-byte
 *    boundary (ld a multiple of 8 for bfloat16, of 4 for float, of 16 for
 *    int8). Matrices without a stride argument are contiguous. Every pointer
 *    is 16-byte aligned, but those to one value a token (target, loss, lse,
 *    dloss, rstd, q_scale, x_scale), which are aligned as their type.
 *  - Outputs must not overlap inputs or each other unless stated otherwise.
 *  - T = 0 tokens succeed (and write what does not depend on tokens: zero
 *    gradients of parameters).
 *  - Sums, statistics and scales are float32 (int32 for integer products,
 *    exact); bfloat16 outputs are rounded once, to nearest even.
 *  - Results do not depend on the run: no output is summed by atomics.
 *  - Sizes within the limits below whose product makes more tiles than one
 *    launch holds (about 2^38 outputs), or w rows further apart than 2^22
 *    elements, give POETX_EUNSUPPORTED.
 */
#ifndef POETX_MODEL_H
#define POETX_MODEL_H

#include "poetx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --- RMS norm of the residual stream -------------------------------------
 *
 *   s = x + res,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * gain
 *
 * over rows of n features (n a multiple of 8, 8 <= n <= 2^24, T <= 2^30),
 * dtype POETX_F32 or POETX_BF16 for x, res, h, y and the gradients.
 *   x [T][n] (stride ldx); res [T][n] (stride ldr) or NULL (s = x).
 *   gain [n] float. eps >= 0 and finite.
 *   h [T][n]: s in the activation type, or NULL. May be x or res itself
 *       (same address, contiguous). The norm uses s before that rounding.
 *   y [T][n].
 *   rstd [T] float, for the backward, or NULL.
 * Rows with infinities or NaN give what the formula gives in float32. */
POETX_API int poetx_rmsnorm_forward(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, const void* res,
                                    int64_t ldr, const float* gain, float eps, void* h, void* y, float* rstd,
                                    hipStream_t stream);

/* The same norm with y as int8 rows and one scale per token, the input of
 * poetx_linear_i8: a = max_j |y_j|, scale = a / 127, q_j = rint(y_j * (127 /
 * a)) (ties to even), |q_j| <= 127. A row with a < 2^-100 counts as zero
 * (codes 0, scale 1). A row holding NaN or infinity has the scale NaN or
 * infinity, so that a product of it is not finite either.
 *   q [T][n] int8, q_scale [T] float; n also a multiple of 16. */
POETX_API int poetx_rmsnorm_forward_q8(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, const void* res,
                                       int64_t ldr, const float* gain, float eps, void* h, int8_t* q,
                                       float* q_scale, hipStream_t stream);

/* int8 rows of x [T][n] (stride ldx) by the rule above, for products whose
 * input does not come from a norm. */
POETX_API int poetx_quantize_rows(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, int8_t* q,
                                  float* q_scale, hipStream_t stream);

/* Gradients of the norm, with u = h * rstd:
 *   dx = rstd * (dy * gain - u * mean(dy * gain * u)) + dh,
 *   dgain = sum_t dy * u
 * dx is the gradient of x and of res alike.
 *   dy [T][n] (stride lddy); h [T][n] and rstd [T] as the forward wrote them
 *       (h = x if the forward had no res); gain [n] float.
 *   dh [T][n] (stride lddh): the gradient that reaches h past the norm, along
 *       the residual stream, or NULL for none.
 *   dx [T][n]; may be dy or dh itself (same address, contiguous).
 *   dgain [n] float, overwritten; or NULL.
 *   ws: poetx_rmsnorm_ws_bytes(T, n) bytes (unused without dgain). */
POETX_API int poetx_rmsnorm_backward(int64_t T, int64_t n, int dtype, const void* dy, int64_t lddy, const void* h,
                                     const float* rstd, const float* gain, const void* dh, int64_t lddh, void* dx,
                                     float* dgain, void* ws, size_t ws_bytes, hipStream_t stream);

/* Workspace bytes of poetx_rmsnorm_backward; 0 for invalid sizes or T = 0. */
POETX_API size_t poetx_rmsnorm_ws_bytes(int64_t T, int64_t n);

/* --- int8 product with scales per token and output -----------------------
 *
 *   z[t][c] = x_scale[t] * w_scale[c] * sum_k xq[t][k] * wt[c][k]
 *
 * the integer sum exact. Serves an int8 base weight after its merge: the
 * weight W0 [m][n] with its scales [n] as poetx_weight_export writes them,
 * laid out once by poetx_linear_i8_prepare as wt [n][m].
 * m and n multiples of 16, 16 <= n <= 2^24, 16 <= m <= 131056 (the largest
 * width whose sums of any int8 codes stay below 2^31), T <= 2^24.
 *   xq [T][m] int8, x_scale [T], wt [n][m] int8, w_scale [n].
 *   z [T][n] (stride ldz), out_dtype POETX_BF16 or POETX_F32. */
POETX_API int poetx_linear_i8(int64_t T, int64_t m, int64_t n, int out_dtype, const int8_t* xq,
                              const float* x_scale, const int8_t* wt, const float* w_scale, void* z, int64_t ldz,
                              hipStream_t stream);

/* wt [n][m] = transpose of w0 [m][n] (int8 codes, sizes as above). */
POETX_API int poetx_linear_i8_prepare(int64_t m, int64_t n, const int8_t* w0, int8_t* wt, hipStream_t stream);

/* --- softmax cross entropy over a vocabulary ------------------------------
 *
 *   l[t][v] = sum_k h[t][k] * w[v][k],  lse[t] = log sum_v exp(l[t][v])
 *   loss[t] = lse[t] - l[t][target[t]]
 *
 * from the rows h [T][d] of the last hidden state and the vocabulary matrix
 * w [V][d]. The logits are formed tile by tile and not kept: the forward
 * keeps a maximum and a sum per row, the backward forms them again, piece by
 * piece of the vocabulary, and multiplies each piece's gradient out at once.
 * The loss is formed as (max_v l[t][v] - l[t][target[t]]) + log sum_v exp(l[t][v]
 * - max): two terms of at least 0, so that it is never negative and the rounding
 * of a large lse is not in it.
 * A token whose target is outside [0, V) (such as -100) is not counted: its
 * loss, lse and dh are 0, it adds nothing to dw, and its row of h is never
 * used, whatever it holds.
 * dtype (h, w, dh, dw): POETX_BF16, or POETX_F32 (float32 products).
 * d a multiple of 8, 8 <= d <= 2^17; 1 <= V <= 2^24; T <= 2^24. */
typedef struct poetx_vocab {
  int64_t d;      /* features of a hidden row */
  int64_t V;      /* vocabulary size, rows of w */
  int32_t dtype;  /* POETX_BF16 or POETX_F32 */
  int32_t piece;  /* vocabulary rows whose gradients the backward holds at a time
                   * (rounded up to a multiple of 256); 0 = chosen for the token
                   * count so that a piece holds 256 MB or the vocabulary, and
                   * at least 1024 rows (2048 T bytes in bfloat16, 4096 T in float:
                   * more than 256 MB past 131072 or 65536 tokens) */
} poetx_vocab;

enum { POETX_OP_VOCAB_FORWARD = 0, POETX_OP_VOCAB_BACKWARD = 1 };

/* Workspace bytes of the two entry points below; 0 for an invalid descriptor,
 * token count or op. Fewer tokens can take more (their sums are split over more
 * workgroups), yet a workspace of the size for T tokens serves every smaller
 * count: with less than the size for their own, the entry points take a plan that
 * fits, slower and with sums in another order, and refuse only what none fits
 * (POETX_EWORKSPACE). */
POETX_API size_t poetx_vocab_ws_bytes(const poetx_vocab* D, int64_t T, int op);

/*   h [T][d] (stride ldh), w [V][d] (stride ldw), target [T] int64.
 *   loss [T], lse [T] float. */
POETX_API int poetx_vocab_loss_forward(const poetx_vocab* D, int64_t T, const void* h, int64_t ldh, const void* w,
                                       int64_t ldw, const int64_t* target, float* loss, float* lse, void* ws,
                                       size_t ws_bytes, hipStream_t stream);

/* Gradients of sum_t g[t] * loss[t], with g[t] = scale * dloss[t], or with
 * dloss NULL g[t] = scale / (number of counted tokens), the mean's gradient:
 *   dl[t][v] = g[t] * (exp(l[t][v] - lse[t]) - [v = target[t]]),
 *   dh = dl w,  dw = dl^T h
 *   lse [T] as the forward wrote it; dh [T][d], dw [V][d] overwritten.
 * With dtype POETX_BF16, dl is rounded to bfloat16 before the two products (at
 * most 2^-8 relative each, independent from term to term of their sums), in
 * units of the largest finite |g[t]|, which is applied to the sums in float32; a
 * g[t] that is not finite reaches its own row of dh, and dw. */
POETX_API int poetx_vocab_loss_backward(const poetx_vocab* D, int64_t T, const void* h, int64_t ldh, const void* w,
                                        int64_t ldw, const int64_t* target, const float* lse, const float* dloss,
                                        float scale, void* dh, void* dw, void* ws, size_t ws_bytes,
                                        hipStream_t stream);

/* --- log probabilities of given tokens, entropy, most likely tokens --------
 *
 *   l[t][v] = (sum_k h[t][k] * w[v][k]) / temperature
 *   lse[t] = log sum_v exp(l[t][v]),  p[t][v] = exp(l[t][v] - lse[t])
 *   logprob[t] = l[t][target[t]] - lse[t]
 *   entropy[t] = -sum_v p[t][v] * log p[t][v]
 *
 * for scoring, policy training and answers with alternatives; sizes, types,
 * strides and rows as for the loss above (poetx_vocab; `piece` concerns the
 * backward). The temperature is positive and finite, and so is log2(e) / temperature
 * in float32 (from 4.24e-39 on). The logits are formed tile by tile; with
 * alternatives, those of some tokens at a time are held in the workspace in 16 bits
 * (1 GB, and at least 256 tokens: 512 V bytes, more than 1 GB past V = 2^21).
 *  - target [T] int64, or NULL: every token is counted, and there is no logprob
 *    (logprob has to be NULL). A token whose target is outside [0, V) (such as
 *    -100) is not counted: its logprob, entropy and stat are 0, its alternatives
 *    -1 and 0, and its row of h is never used, whatever it holds.
 *  - top: 0 <= top <= 64, top <= V. top_ids and top_logprobs [T][top]: the most
 *    likely tokens, most likely first, and their log probabilities; both NULL for
 *    top = 0. Both go by the logits in double (products of h and w summed in
 *    double), equal ones by the lower index: so the order does not depend on
 *    float32's rounding, or on how many tokens a call holds. What is ordered so is
 *    what float32 logits put among the top + 8 largest, at least; of logits that are
 *    equal to the last of these in float32, and with the others are more than 512, the
 *    512 of the lowest index.
 *  - stat [T][2], 8-byte aligned, for the backward: the row's largest logit before
 *    the temperature, max, and log sum_v exp(l[t][v] - max / temperature), so that lse
 *    = stat[0] / temperature + stat[1]. Rows that are sure of a token keep the
 *    precision of logprob and entropy near 0 in it.
 *  - A row with logits that are NaN or +infinity has no finite logprob, entropy, stat[1]
 *    or top_logprobs; NaN counts as -infinity in the order. */
POETX_API int poetx_token_logprobs(const poetx_vocab* D, int64_t T, float temperature, const void* h, int64_t ldh,
                                   const void* w, int64_t ldw, const int64_t* target, int32_t top, float* logprob,
                                   float* entropy, float* stat, int64_t* top_ids, float* top_logprobs, void* ws,
                                   size_t ws_bytes, hipStream_t stream);

/* Gradients of sum_t (dlogprob[t] * logprob[t] + dentropy[t] * entropy[t]):
 *   dl[t][v] = dlogprob[t] * ([v = target[t]] - p[t][v])
 *              - dentropy[t] * p[t][v] * (log p[t][v] + entropy[t])
 *   dh = dl w / temperature,  dw = dl^T h / temperature
 *   stat, entropy as the forward wrote them (entropy is read only with
 *       dentropy); dh [T][d], dw [V][d] overwritten.
 *   dlogprob, dentropy [T]: one of them may be NULL (none); dlogprob needs targets.
 * Rounding of dl with POETX_BF16, gradients that are not finite and the workspace as
 * for the loss above; its unit is the largest finite |dlogprob[t]| or
 * |dentropy[t]|. What the rounding takes off the targets' terms, which are most of dl, is
 * put back in float32 (in dw for words that are at most 16 tokens' target). */
POETX_API int poetx_token_logprobs_backward(const poetx_vocab* D, int64_t T, float temperature, const void* h,
                                            int64_t ldh, const void* w, int64_t ldw, const int64_t* target,
                                            const float* stat, const float* entropy, const float* dlogprob,
                                            const float* dentropy, void* dh, void* dw, void* ws, size_t ws_bytes,
                                            hipStream_t stream);

/* Workspace bytes of the two entry points above (op POETX_OP_VOCAB_FORWARD or
 * POETX_OP_VOCAB_BACKWARD, the latter with top = 0); 0 for invalid arguments or T = 0. A
 * workspace of the size for T tokens serves every smaller count, as the loss's
 * does. */
POETX_API size_t poetx_token_ws_bytes(const poetx_vocab* D, int64_t T, int op, int32_t top);

/* --- norm of all gradients, and clipping -----------------------------------
 *
 *   norm = sqrt(sum_i sum_j g[i][j]^2)
 *   out[i][j] = g[i][j] * min(1, max_norm / (norm + 1e-6))
 *
 * over `count` tensors (0 <= count <= 2^20) of n[i] values each (0 <= n[i] <= 2^40,
 * POETX_F32 or POETX_BF16 by dtype[i], contiguous and aligned as their type; an
 * empty one's pointer is not used), such as the packed gradients of all layers, the
 * gains' and the vocabulary matrix's. The pointers, sizes and types are host
 * arrays, read before the call returns. Squares and sums are in double, the sum
 * rounded once, to the norm; the factor is formed in double and applied in float32, one
 * below float32's normal numbers in two steps.
 *   norm [1] float on the device.
 *   out[i] may be g[i] itself, which a factor of 1 leaves untouched; apart from
 *       that no output may overlap an input or another output (POETX_EINVAL): a
 *       tensor listed twice is refused, for it would be scaled twice.
 *   max_norm >= 0 and finite. A norm that is infinite gives the factor 0 (and NaN
 *       where a gradient is infinite), one that is NaN makes all outputs NaN: what the
 *       formula gives.
 *   ws: poetx_grad_ws_bytes(count) bytes.
 *   Tensors of 2^45 bytes together (in units of 16 KB each) give POETX_EUNSUPPORTED. */
POETX_API int poetx_grad_norm(int64_t count, const void* const* g, const int64_t* n, const int32_t* dtype, float* norm,
                              void* ws, size_t ws_bytes, hipStream_t stream);
POETX_API int poetx_grad_clip(int64_t count, const void* const* g, void* const* out, const int64_t* n,
                              const int32_t* dtype, float max_norm, float* norm, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* Workspace bytes of the two entry points above; 0 for count = 0 or an invalid one. */
POETX_API size_t poetx_grad_ws_bytes(int64_t count);

#ifdef __cplusplus
}
#endif

#endif /* POETX_MODEL_H */
