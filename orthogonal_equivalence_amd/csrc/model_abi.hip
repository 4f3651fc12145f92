// C ABI of poetx_model.h: argument validation, workspace layout and the
// launches of the operators around the layer.
#include "../../include/poetx_model.h"
#include "abi_common.hpp"
#include "kernels.hpp"
#include "model_kernels.hpp"

#include <algorithm>
#include <cmath>

using namespace poetx;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxWidth = int64_t(1) << 24;

bool act_ok(int dtype) { return dtype == POETX_F32 || dtype == POETX_BF16; }
int elem(int dtype) { return dtype == POETX_F32 ? 4 : (dtype == POETX_BF16 ? 2 : 1); }

bool rows_ok(int64_t T, int64_t n, int mult) { return T >= 0 && T <= kMaxRows && n >= mult && n <= kMaxWidth && n % mult == 0; }

// values one a token, read one at a time: aligned as their type
bool tokens_ok(std::initializer_list<const void*> ps, uintptr_t size) {
  for (const void* p : ps)
    if (!p || reinterpret_cast<uintptr_t>(p) % size) return false;
  return true;
}

// a row stride: at least the row, every row 16-byte aligned
bool stride_ok(int64_t ld, int64_t cols, int es) { return ld >= cols && ld <= (int64_t(1) << 40) && ld * es % 16 == 0; }

// `out` may be the input `in` itself only where both are contiguous
bool alias_ok(const void* out, const void* in, int64_t ld, int64_t cols) { return out != in || ld == cols; }

int ws_ok(const void* ws, size_t have, size_t need) {
  if (need == 0) return POETX_OK;
  if (have < need) return POETX_EWORKSPACE;
  return ws && aligned16(ws) ? POETX_OK : POETX_EINVAL;
}

// --- norm ----------------------------------------------------------------------

int norm_common(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, const void* res, int64_t ldr,
                const float* gain, float eps, void* h, NormFwdDesc& d) {
  if (!act_ok(dtype) || !(eps >= 0.f) || !std::isfinite(eps)) return POETX_EINVAL;
  if (!stride_ok(ldx, n, elem(dtype)) || (res && !stride_ok(ldr, n, elem(dtype)))) return POETX_EINVAL;
  if (T > 0) {
    if (!ptrs_ok({x, gain})) return POETX_EINVAL;
    if ((res && !aligned16(res)) || (h && !aligned16(h))) return POETX_EINVAL;
    if (h && (!alias_ok(h, x, ldx, n) || (res && !alias_ok(h, res, ldr, n)))) return POETX_EINVAL;
  }
  d.x = x;
  d.ldx = ldx;
  d.res = res;
  d.ldr = ldr;
  d.gain = gain;
  d.eps = eps;
  d.h = h;
  d.T = T;
  d.n = n;
  d.bf16 = dtype == POETX_BF16;
  return POETX_OK;
}

// --- vocabulary loss -------------------------------------------------------------

constexpr int64_t kVocabTokens = int64_t(1) << 24;
constexpr int64_t kPieceBytes = int64_t(1) << 28;
constexpr int64_t kPieceMax = int64_t(1) << 20;
constexpr int64_t kVocabStride = int64_t(1) << 22;  // a tile's offsets stay below 2^31 bytes

bool vocab_ok(const poetx_vocab* D, int64_t T) {
  return D && D->d >= 8 && D->d <= (int64_t(1) << 17) && D->d % 8 == 0 && D->V >= 1 && D->V <= kMaxWidth &&
         act_ok(D->dtype) && D->piece >= 0 && T >= 0 && T <= kVocabTokens;
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// pieces of at most `most` rows, a multiple of 256, evened out
int64_t even_piece(int64_t all, int64_t most) {
  const int64_t pieces = (all + most - 1) / most;
  return round256((all + pieces - 1) / pieces);
}

// Vocabulary rows of a piece: as asked, or as many as kPieceBytes hold (at
// least 1024: adding a piece to dh's float sums moves 8 T d bytes, more time than
// the products of 256 rows, a third of that of 1024), evened out over the pieces.
int64_t piece_of(const poetx_vocab* D, int64_t T) {
  const int64_t all = round256(D->V);
  if (D->piece > 0) return std::min({round256(D->piece), all, kPieceMax});
  const int64_t most = std::min(kPieceMax, std::max<int64_t>(1024, kPieceBytes / (std::max<int64_t>(T, 1) * elem(D->dtype)) / 256 * 256));
  return even_piece(all, most);
}

// Sizes, tiles and splits of a call, without its memory. `lean`: the plan that
// takes the least memory with pieces of this size.
VocabDesc vocab_sizes(const poetx_vocab* D, int64_t T, int op, int64_t piece, bool lean) {
  VocabDesc v;
  v.T = T;
  v.d = D->d;
  v.V = D->V;
  v.bf16 = D->dtype == POETX_BF16;
  v.piece = piece;
  const int es = elem(D->dtype);
  v.ldhc = (D->d * es + 127) / 128 * 128 / es;
  v.backward = op == POETX_OP_VOCAB_BACKWARD;
  vocab_plan(v, lean);
  return v;
}

void carve_vocab(VocabDesc& v, Carve& c) {
  const int64_t T = v.T, es = v.bf16 ? 2 : 4;
  if (T > 2 * kVocabChunk) v.rows.chunk = c.take<int2>((T + kVocabChunk - 1) / kVocabChunk);
  v.rows.pos = c.take<int32_t>(T);
  v.rows.idx = c.take<int32_t>(T);
  v.rows.tgt = c.take<int32_t>(T);
  v.rows.count = c.take<int32_t>(1);
  v.hc = c.take<char>(T * v.ldhc * es);
  if (v.backward) {
    v.rows.g = c.take<float>(T);
    v.rows.lse = c.take<float>(T);
    v.rows.unit = c.take<float>(1);
    v.p = c.take<char>(T * v.piece * es);
    if (v.piece < v.V || v.dh_plan.splits > 1) v.acc = c.take<float>(v.dh_plan.splits * T * v.d);
    if (v.dw_plan.splits > 1) v.acc_w = c.take<float>(v.dw_plan.splits * std::min(v.piece, v.V) * v.d);
  } else {
    v.tl = c.take<float>(T);
    v.stat = c.take<float2>(static_cast<int64_t>(v.stat_tiles) * T);
  }
}

size_t vocab_bytes(VocabDesc v) {
  Carve c(nullptr);
  carve_vocab(v, c);
  return c.off;
}

// The plan for a workspace of `bytes`: the fastest one, whose size the query
// returns, or where that is larger the lean one, in smaller pieces if need be. A
// workspace of the fastest plan for more tokens always holds it: that plan's
// piece with these tokens takes no more in any part, as all parts grow with T.
VocabDesc vocab_within(const poetx_vocab* D, int64_t T, int op, size_t bytes) {
  VocabDesc v = vocab_sizes(D, T, op, piece_of(D, T), false);
  if (!v.fits || vocab_bytes(v) <= bytes) return v;
  v = vocab_sizes(D, T, op, v.piece, true);
  const size_t need = vocab_bytes(v);
  if (need <= bytes || !v.backward || D->piece > 0) return v;
  // what the plan holds beside the piece, dh's sums over pieces included
  const size_t row = static_cast<size_t>(T) * elem(D->dtype);
  const size_t sums = v.piece < v.V ? 0 : static_cast<size_t>(round256(T * v.d * 4));
  const size_t rest = need - static_cast<size_t>(v.piece) * row + sums;
  const int64_t most = bytes > rest ? static_cast<int64_t>((bytes - rest) / row / 256 * 256) : 0;
  return most > 0 ? vocab_sizes(D, T, op, even_piece(round256(v.V), most), true) : v;
}

// A checked call's description, its workspace laid out.
int vocab_call(const poetx_vocab* D, int64_t T, int op, const void* h, int64_t ldh, const void* w, int64_t ldw,
               const int64_t* target, void* ws, size_t ws_bytes, VocabDesc& v) {
  const int es = elem(D->dtype);
  if (!stride_ok(ldh, D->d, es) || !stride_ok(ldw, D->d, es)) return POETX_EINVAL;
  if (!ptrs_ok({h, w}) || !tokens_ok({target}, 8)) return POETX_EINVAL;
  v = vocab_within(D, T, op, ws_bytes);
  if (ldw > kVocabStride || !v.fits) return POETX_EUNSUPPORTED;
  if (const int e = ws_ok(ws, ws_bytes, vocab_bytes(v))) return e;
  Carve c(ws);
  carve_vocab(v, c);
  v.h = h;
  v.ldh = ldh;
  v.w = w;
  v.ldw = ldw;
  v.target = target;
  return POETX_OK;
}

}  // namespace

extern "C" {

int poetx_rmsnorm_forward(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, const void* res, int64_t ldr,
                          const float* gain, float eps, void* h, void* y, float* rstd, hipStream_t stream) {
  if (!rows_ok(T, n, 8)) return POETX_EINVAL;
  NormFwdDesc d;
  if (const int e = norm_common(T, n, dtype, x, ldx, res, ldr, gain, eps, h, d)) return e;
  if (T > 0 && (!ptrs_ok({y}) || (rstd && !tokens_ok({rstd}, 4)))) return POETX_EINVAL;
  clear_pending_error();
  if (T == 0) return POETX_OK;
  d.y = y;
  d.rstd = rstd;
  ProfScope p("rmsnorm_fwd", stream);
  norm_forward(d, stream);
  return launch_status();
}

int poetx_rmsnorm_forward_q8(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, const void* res,
                             int64_t ldr, const float* gain, float eps, void* h, int8_t* q, float* q_scale,
                             hipStream_t stream) {
  if (!rows_ok(T, n, 16)) return POETX_EINVAL;
  NormFwdDesc d;
  if (const int e = norm_common(T, n, dtype, x, ldx, res, ldr, gain, eps, h, d)) return e;
  if (T > 0 && (!ptrs_ok({q}) || !tokens_ok({q_scale}, 4))) return POETX_EINVAL;
  clear_pending_error();
  if (T == 0) return POETX_OK;
  d.q = q;
  d.scale = q_scale;
  ProfScope p("rmsnorm_fwd_q8", stream);
  norm_forward(d, stream);
  return launch_status();
}

int poetx_quantize_rows(int64_t T, int64_t n, int dtype, const void* x, int64_t ldx, int8_t* q, float* q_scale,
                        hipStream_t stream) {
  if (!rows_ok(T, n, 16) || !act_ok(dtype) || !stride_ok(ldx, n, elem(dtype))) return POETX_EINVAL;
  if (T > 0 && (!ptrs_ok({x, q}) || !tokens_ok({q_scale}, 4))) return POETX_EINVAL;
  clear_pending_error();
  if (T == 0) return POETX_OK;
  NormFwdDesc d;
  d.x = x;
  d.ldx = ldx;
  d.q = q;
  d.scale = q_scale;
  d.T = T;
  d.n = n;
  d.bf16 = dtype == POETX_BF16;
  ProfScope p("quantize_rows", stream);
  norm_forward(d, stream);
  return launch_status();
}

size_t poetx_rmsnorm_ws_bytes(int64_t T, int64_t n) {
  if (!rows_ok(T, n, 8) || T == 0) return 0;
  return static_cast<size_t>(norm_bwd_groups(T, n)) * n * sizeof(float);
}

int poetx_rmsnorm_backward(int64_t T, int64_t n, int dtype, const void* dy, int64_t lddy, const void* h,
                           const float* rstd, const float* gain, const void* dh, int64_t lddh, void* dx,
                           float* dgain, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!rows_ok(T, n, 8) || !act_ok(dtype)) return POETX_EINVAL;
  if (!stride_ok(lddy, n, elem(dtype)) || (dh && !stride_ok(lddh, n, elem(dtype)))) return POETX_EINVAL;
  if (dgain && !aligned16(dgain)) return POETX_EINVAL;
  if (T > 0) {
    if (!ptrs_ok({dy, h, gain, dx}) || !tokens_ok({rstd}, 4) || (dh && !aligned16(dh))) return POETX_EINVAL;
    if (!alias_ok(dx, dy, lddy, n) || (dh && !alias_ok(dx, dh, lddh, n))) return POETX_EINVAL;
    if (dgain)
      if (const int e = ws_ok(ws, ws_bytes, poetx_rmsnorm_ws_bytes(T, n))) return e;
  }
  clear_pending_error();
  if (T == 0) {
    if (dgain) fill_zero_f32(dgain, n, stream);
    return launch_status();
  }
  NormBwdDesc d;
  d.dy = dy;
  d.lddy = lddy;
  d.h = h;
  d.rstd = rstd;
  d.gain = gain;
  d.dh = dh;
  d.lddh = lddh;
  d.dx = dx;
  d.part = dgain ? static_cast<float*>(ws) : nullptr;
  d.dgain = dgain;
  d.T = T;
  d.n = n;
  d.bf16 = dtype == POETX_BF16;
  ProfScope p("rmsnorm_bwd", stream);
  norm_backward(d, stream);
  return launch_status();
}

// --- int8 product ----------------------------------------------------------------

namespace {
// The widest sum of products of any int8 codes that stays below 2^31.
constexpr int64_t kMaxI8Width = 131056;
bool i8_sizes_ok(int64_t m, int64_t n) {
  return m >= 16 && m % 16 == 0 && m <= kMaxI8Width && n >= 16 && n % 16 == 0 && n <= kMaxWidth;
}
}  // namespace

int poetx_linear_i8(int64_t T, int64_t m, int64_t n, int out_dtype, const int8_t* xq, const float* x_scale,
                    const int8_t* wt, const float* w_scale, void* z, int64_t ldz, hipStream_t stream) {
  if (!i8_sizes_ok(m, n) || T < 0 || T > kVocabTokens || !act_ok(out_dtype)) return POETX_EINVAL;
  if (!stride_ok(ldz, n, elem(out_dtype))) return POETX_EINVAL;
  if (T > 0 && (!ptrs_ok({xq, wt, w_scale, z}) || !tokens_ok({x_scale}, 4))) return POETX_EINVAL;
  clear_pending_error();
  if (T == 0) return POETX_OK;
  LinearI8Desc d;
  d.xq = xq;
  d.xs = x_scale;
  d.wt = wt;
  d.ws = w_scale;
  d.z = z;
  d.ldz = ldz;
  d.T = T;
  d.m = m;
  d.n = n;
  d.out_bf16 = out_dtype == POETX_BF16;
  ProfScope p("linear_i8", stream);
  if (!linear_i8(d, stream)) return POETX_EUNSUPPORTED;
  return launch_status();
}

int poetx_linear_i8_prepare(int64_t m, int64_t n, const int8_t* w0, int8_t* wt, hipStream_t stream) {
  if (!i8_sizes_ok(m, n) || !ptrs_ok({w0, wt})) return POETX_EINVAL;
  clear_pending_error();
  ProfScope p("linear_i8_prepare", stream);
  if (!transpose(w0, wt, m, n, 1, stream)) return POETX_EUNSUPPORTED;
  return launch_status();
}

// --- vocabulary loss -----------------------------------------------------------

size_t poetx_vocab_ws_bytes(const poetx_vocab* D, int64_t T, int op) {
  if (!vocab_ok(D, T) || (op != POETX_OP_VOCAB_FORWARD && op != POETX_OP_VOCAB_BACKWARD)) return 0;
  return vocab_bytes(vocab_sizes(D, T, op, piece_of(D, T), false));
}

int poetx_vocab_loss_forward(const poetx_vocab* D, int64_t T, const void* h, int64_t ldh, const void* w, int64_t ldw,
                             const int64_t* target, float* loss, float* lse, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
  if (!vocab_ok(D, T)) return POETX_EINVAL;
  if (T == 0) {
    clear_pending_error();
    return POETX_OK;
  }
  if (!tokens_ok({loss, lse}, 4)) return POETX_EINVAL;
  VocabDesc v;
  if (const int e = vocab_call(D, T, POETX_OP_VOCAB_FORWARD, h, ldh, w, ldw, target, ws, ws_bytes, v)) return e;
  clear_pending_error();
  v.loss = loss;
  v.lse = lse;
  ProfScope p("vocab_loss_fwd", stream);
  vocab_forward(v, stream);
  return launch_status();
}

int poetx_vocab_loss_backward(const poetx_vocab* D, int64_t T, const void* h, int64_t ldh, const void* w,
                              int64_t ldw, const int64_t* target, const float* lse, const float* dloss, float scale,
                              void* dh, void* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!vocab_ok(D, T) || !ptrs_ok({dw})) return POETX_EINVAL;
  if (T == 0) {
    clear_pending_error();
    fill_zero_f32(static_cast<float*>(dw), D->V * D->d * elem(D->dtype) / 4, stream);
    return launch_status();
  }
  if (!ptrs_ok({dh}) || !tokens_ok({lse}, 4) || (dloss && !tokens_ok({dloss}, 4))) return POETX_EINVAL;
  VocabDesc v;
  if (const int e = vocab_call(D, T, POETX_OP_VOCAB_BACKWARD, h, ldh, w, ldw, target, ws, ws_bytes, v)) return e;
  clear_pending_error();
  v.lse_in = lse;
  v.dloss = dloss;
  v.scale = scale;
  v.dh = dh;
  v.dw = dw;
  ProfScope p("vocab_loss_bwd", stream);
  vocab_backward(v, stream);
  return launch_status();
}

}  // extern "C"
