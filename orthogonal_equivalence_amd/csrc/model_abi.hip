// C ABI of poetx_model.h: argument validation, workspace layout and the
// launches of the operators around the layer.
#include "../../include/poetx_model.h"
#include "abi_common.hpp"
#include "kernels.hpp"
#include "model_kernels.hpp"

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

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

// What is asked of the vocabulary: the loss or the log probabilities, forward or
// backward, with how many alternatives.
struct VocabOp {
  bool backward = false, token = false;
  int top = 0;
};

// Tokens whose logits (16 bits each, whole tiles) are held at a time for the
// alternatives: as many as 1 GB holds, at least 256. (T = 8192, d = 4096, V = 131072:
// 6.94 ms of products in one launch, 7.27 in eight of 256 MB each.)
constexpr int64_t kChunkBytes = int64_t(1) << 30;
int64_t chunk_of(const poetx_vocab* D, int64_t T) {
  return std::min(T, std::max<int64_t>(256, kChunkBytes / (round256(D->V) * 2) / 256 * 256));
}

// Sizes, tiles and splits of a call, without its memory. `lean`: the plan that
// takes the least memory with pieces of this size.
VocabDesc vocab_sizes(const poetx_vocab* D, int64_t T, const VocabOp& op, int64_t piece, bool lean) {
  VocabDesc v;
  v.T = T;
  v.d = D->d;
  v.V = D->V;
  v.bf16 = D->dtype == POETX_BF16;
  v.piece = piece;
  const int es = elem(D->dtype);
  v.ldhc = (D->d * es + 127) / 128 * 128 / es;
  v.backward = op.backward;
  v.token = op.token;
  v.top = op.top;
  if (op.top > 0) {
    v.chunk = chunk_of(D, T);
    v.ldl = round256(D->V);
  }
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
    if (!v.token) v.rows.lse = c.take<float>(T);
    v.rows.unit = c.take<float>(1);
    if (v.token) {
      v.rows.stat = c.take<float2>(T);
      v.rows.gent = c.take<float>(T);
      v.rows.ent = c.take<float>(T);
      if (v.bf16) v.rows.resid = c.take<float>(T);
    }
    v.p = c.take<char>(T * v.piece * es);
    if (v.piece < v.V || v.dh_plan.splits > 1) v.acc = c.take<float>(v.dh_plan.splits * T * v.d);
    if (v.dw_plan.splits > 1) v.acc_w = c.take<float>(v.dw_plan.splits * std::min(v.piece, v.V) * v.d);
  } else {
    v.tl = c.take<float>(T);
    if (!v.top) v.stat = c.take<float2>(static_cast<int64_t>(v.stat_tiles) * T);
    if (!v.top && v.token) v.statu = c.take<float>(static_cast<int64_t>(v.stat_tiles) * T);
    if (v.top) {
      v.rec = c.take<char>(v.chunk * v.stat_tiles * kTokenRec);
      v.codes = c.take<uint16_t>(v.chunk * v.ldl);
    }
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
VocabDesc vocab_within(const poetx_vocab* D, int64_t T, const VocabOp& op, size_t bytes) {
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
int vocab_call(const poetx_vocab* D, int64_t T, const VocabOp& op, const void* h, int64_t ldh, const void* w, int64_t ldw,
               const int64_t* target, void* ws, size_t ws_bytes, VocabDesc& v) {
  const int es = elem(D->dtype);
  if (!stride_ok(ldh, D->d, es) || !stride_ok(ldw, D->d, es)) return POETX_EINVAL;
  if (!ptrs_ok({h, w}) || (!(op.token && !target) && !tokens_ok({target}, 8))) return POETX_EINVAL;
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
  return vocab_bytes(vocab_sizes(D, T, {op == POETX_OP_VOCAB_BACKWARD}, piece_of(D, T), false));
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
  if (const int e = vocab_call(D, T, {}, h, ldh, w, ldw, target, ws, ws_bytes, v)) return e;
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
  if (const int e = vocab_call(D, T, {true}, h, ldh, w, ldw, target, ws, ws_bytes, v)) return e;
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

// --- log probabilities -----------------------------------------------------------

namespace {
// factor of the logits, or 0 for a temperature that is refused: that of their powers of
// two is finite, too (0, the maximum's distance, times infinity would be NaN)
float inverse(float temperature) {
  const float f = 1.f / temperature;
  return temperature > 0.f && std::isfinite(temperature) && std::isfinite(f * kLog2e) ? f : 0.f;
}
bool top_ok(const poetx_vocab* D, int32_t top) { return top >= 0 && top <= kTopMost && top <= D->V; }
}  // namespace

size_t poetx_token_ws_bytes(const poetx_vocab* D, int64_t T, int op, int32_t top) {
  if (!vocab_ok(D, T) || (op != POETX_OP_VOCAB_FORWARD && op != POETX_OP_VOCAB_BACKWARD)) return 0;
  const bool backward = op == POETX_OP_VOCAB_BACKWARD;
  if (T == 0 || !top_ok(D, top) || (backward && top)) return 0;
  return vocab_bytes(vocab_sizes(D, T, {backward, true, top}, piece_of(D, T), false));
}

int poetx_token_logprobs(const poetx_vocab* D, int64_t T, float temperature, const void* h, int64_t ldh, const void* w,
                         int64_t ldw, const int64_t* target, int32_t top, float* logprob, float* entropy, float* stat,
                         int64_t* top_ids, float* top_logprobs, void* ws, size_t ws_bytes, hipStream_t stream) {
  const float f = inverse(temperature);
  if (!vocab_ok(D, T) || f == 0.f || !top_ok(D, top)) return POETX_EINVAL;
  if (T == 0) {
    clear_pending_error();
    return POETX_OK;
  }
  if (!tokens_ok({entropy}, 4) || !tokens_ok({stat}, 8) || (target ? !tokens_ok({logprob}, 4) : logprob != nullptr)) return POETX_EINVAL;
  if (top ? !tokens_ok({top_ids}, 8) || !tokens_ok({top_logprobs}, 4) : top_ids || top_logprobs) return POETX_EINVAL;
  VocabDesc v;
  if (const int e = vocab_call(D, T, {false, true, top}, h, ldh, w, ldw, target, ws, ws_bytes, v)) return e;
  clear_pending_error();
  v.inv_temp = f;
  v.logprob = logprob;
  v.entropy = entropy;
  v.row_stat = reinterpret_cast<float2*>(stat);
  v.top_ids = top_ids;
  v.top_logprobs = top_logprobs;
  ProfScope p("token_logprobs", stream);
  token_forward(v, stream);
  return launch_status();
}

int poetx_token_logprobs_backward(const poetx_vocab* D, int64_t T, float temperature, const void* h, int64_t ldh,
                                  const void* w, int64_t ldw, const int64_t* target, const float* stat,
                                  const float* entropy, const float* dlogprob, const float* dentropy, void* dh, void* dw,
                                  void* ws, size_t ws_bytes, hipStream_t stream) {
  const float f = inverse(temperature);
  if (!vocab_ok(D, T) || f == 0.f || !ptrs_ok({dw})) return POETX_EINVAL;
  if (T == 0) {
    clear_pending_error();
    fill_zero_f32(static_cast<float*>(dw), D->V * D->d * elem(D->dtype) / 4, stream);
    return launch_status();
  }
  if (!ptrs_ok({dh}) || !tokens_ok({stat}, 8) || (!dlogprob && !dentropy)) return POETX_EINVAL;
  if (dlogprob && (!target || !tokens_ok({dlogprob}, 4))) return POETX_EINVAL;
  if (dentropy && !tokens_ok({dentropy, entropy}, 4)) return POETX_EINVAL;
  VocabDesc v;
  if (const int e = vocab_call(D, T, {true, true}, h, ldh, w, ldw, target, ws, ws_bytes, v)) return e;
  clear_pending_error();
  v.inv_temp = f;
  v.stat_in = reinterpret_cast<const float2*>(stat);
  v.dloss = dlogprob;
  v.scale = -1.f;  // a loss is a negative log probability
  v.dent = dentropy;
  v.ent_in = entropy;
  if (!dentropy) v.rows.gent = v.rows.ent = nullptr;
  v.dh = dh;
  v.dw = dw;
  ProfScope p("token_logprobs_bwd", stream);
  vocab_backward(v, stream);
  return launch_status();
}

// --- gradient norm -------------------------------------------------------------

namespace {

constexpr int64_t kMaxTensors = int64_t(1) << 20;
constexpr int64_t kMaxValues = int64_t(1) << 40;
constexpr int64_t kMaxUnits = int64_t(1) << 31;

struct Span {
  uintptr_t from, to;
  bool operator<(const Span& o) const { return from < o.from; }
};

// every tensor's size, type and address
int grads_ok(int64_t count, const void* const* g, const int64_t* n, const int32_t* dtype) {
  if (count < 0 || count > kMaxTensors || (count > 0 && (!g || !n || !dtype))) return POETX_EINVAL;
  int64_t units = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (n[i] < 0 || n[i] > kMaxValues || !act_ok(dtype[i])) return POETX_EINVAL;
    if (n[i] > 0 && !tokens_ok({g[i]}, elem(dtype[i]))) return POETX_EINVAL;
    units += grad_units(n[i], dtype[i] == POETX_BF16);
  }
  return units < kMaxUnits ? POETX_OK : POETX_EUNSUPPORTED;
}

// Outputs apart from each other, and from every input but, at the same address,
// their own.
int outs_ok(int64_t count, const void* const* g, void* const* out, const int64_t* n, const int32_t* dtype) {
  const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[count]);
  if (!spans) return POETX_EUNSUPPORTED;
  int64_t m = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (n[i] == 0) continue;
    if (!tokens_ok({out[i]}, elem(dtype[i]))) return POETX_EINVAL;
    const uintptr_t p = reinterpret_cast<uintptr_t>(out[i]);
    spans[m++] = {p, p + static_cast<uintptr_t>(n[i]) * elem(dtype[i])};
  }
  std::sort(spans.get(), spans.get() + m);
  for (int64_t i = 1; i < m; ++i)
    if (spans[i].from < spans[i - 1].to) return POETX_EINVAL;
  for (int64_t i = 0; i < count; ++i) {
    if (n[i] == 0 || g[i] == out[i]) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(g[i]);
    // the last output that starts before the input's end
    const Span* s = std::lower_bound(spans.get(), spans.get() + m, Span{p + static_cast<uintptr_t>(n[i]) * elem(dtype[i]), 0});
    if (s != spans.get() && (s - 1)->to > p) return POETX_EINVAL;
  }
  return POETX_OK;
}

int grad_call(int64_t count, const void* const* g, void* const* out, const int64_t* n, const int32_t* dtype,
              float max_norm, float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (const int e = ws_ok(ws, ws_bytes, poetx_grad_ws_bytes(count))) return e;
  clear_pending_error();
  GradDesc d;
  d.count = count;
  d.g = g;
  d.out = out;
  d.n = n;
  d.dtype = dtype;
  d.bf16_code = POETX_BF16;
  d.max_norm = max_norm;
  d.norm = norm;
  Carve c(ws);
  d.part = c.take<double>(grad_parts(count));
  d.table = c.take<GradEntry>(count);
  ProfScope p(out ? "grad_clip" : "grad_norm", stream);
  grad_norm(d, stream);
  return launch_status();
}

}  // namespace

size_t poetx_grad_ws_bytes(int64_t count) {
  if (count <= 0 || count > kMaxTensors) return 0;
  Carve c(nullptr);
  c.take<double>(grad_parts(count));
  c.take<GradEntry>(count);
  return c.off;
}

int poetx_grad_norm(int64_t count, const void* const* g, const int64_t* n, const int32_t* dtype, float* norm, void* ws,
                    size_t ws_bytes, hipStream_t stream) {
  if (const int e = grads_ok(count, g, n, dtype)) return e;
  if (!tokens_ok({norm}, 4)) return POETX_EINVAL;
  return grad_call(count, g, nullptr, n, dtype, 0.f, norm, ws, ws_bytes, stream);
}

int poetx_grad_clip(int64_t count, const void* const* g, void* const* out, const int64_t* n, const int32_t* dtype,
                    float max_norm, float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (const int e = grads_ok(count, g, n, dtype)) return e;
  if (!tokens_ok({norm}, 4) || !(max_norm >= 0.f) || !std::isfinite(max_norm) || (count > 0 && !out)) return POETX_EINVAL;
  if (count == 0) return grad_call(0, g, nullptr, n, dtype, 0.f, norm, ws, ws_bytes, stream);
  if (const int e = outs_ok(count, g, out, n, dtype)) return e;
  return grad_call(count, g, out, n, dtype, max_norm, norm, ws, ws_bytes, stream);
}

}  // extern "C"
