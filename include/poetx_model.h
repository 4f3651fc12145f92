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

#ifdef __cplusplus
}
#endif

#endif /* POETX_MODEL_H */
