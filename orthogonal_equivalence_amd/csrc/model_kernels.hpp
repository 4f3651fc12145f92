// Launchers of the operators around the layer (rmsnorm.hip, linear_i8.hip,
// vocab_loss.hip). All launch on `stream`; their callers have validated the
// sizes (poetx_model.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace poetx {

constexpr float kLog2e = 1.4426950408889634f;

// The norm of x + res (res optional) with y or int8 codes q out; gain null:
// only the row quantisation of x.
struct NormFwdDesc {
  const void* x = nullptr;
  int64_t ldx = 0;
  const void* res = nullptr;
  int64_t ldr = 0;
  const float* gain = nullptr;
  float eps = 0.f;
  void* h = nullptr;
  void* y = nullptr;
  float* rstd = nullptr;
  int8_t* q = nullptr;
  float* scale = nullptr;
  int64_t T = 0, n = 0;
  bool bf16 = true;
};
void norm_forward(const NormFwdDesc& d, hipStream_t stream);

struct NormBwdDesc {
  const void* dy = nullptr;
  int64_t lddy = 0;
  const void* h = nullptr;
  const float* rstd = nullptr;
  const float* gain = nullptr;
  const void* dh = nullptr;
  int64_t lddh = 0;
  void* dx = nullptr;
  float* part = nullptr;   // norm_bwd_groups(T, n) * n floats of scratch, with dgain
  float* dgain = nullptr;
  int64_t T = 0, n = 0;
  bool bf16 = true;
};
// Row groups of the backward: each sums its rows' share of dgain.
int norm_bwd_groups(int64_t T, int64_t n);
void norm_backward(const NormBwdDesc& d, hipStream_t stream);

// z = (xq wt^T) scaled per row and column (poetx_linear_i8).
struct LinearI8Desc {
  const int8_t* xq = nullptr;
  const float* xs = nullptr;
  const int8_t* wt = nullptr;
  const float* ws = nullptr;
  void* z = nullptr;
  int64_t ldz = 0;
  int64_t T = 0, m = 0, n = 0;
  bool out_bf16 = true;
};
// false, with nothing launched, where T and n make more tiles than one launch holds.
bool linear_i8(const LinearI8Desc& d, hipStream_t stream);

// Vocabulary cross entropy (poetx_vocab_loss_*). The counted tokens (target
// in [0, V)) are gathered to the front: compact row c is token idx[c], and
// pos[t] is token t's compact row or -1.
constexpr int kVocabChunk = 4096;
// Elements from row to row of what a product reads in its place: the offsets of a
// tile's rows (256 of bfloat16, 128 of float) stay below 2^31 bytes.
constexpr int64_t kVocabStride = int64_t(1) << 22;
struct VocabRows {
  int2* chunk;     // [T / kVocabChunk, rounded up] counted tokens and largest gradient (more than two chunks)
  int32_t* pos;    // [T]
  int32_t* idx;    // [T]
  int32_t* tgt;    // [T] target of compact row c
  float* g;        // [T] upstream gradient of compact row c, in units of the largest (backward)
  float* unit;     // [1] that unit (backward)
  float* lse;      // [T] lse of compact row c (backward of the loss)
  float2* stat;    // [T] its maximum and log of the sum (backward of log probabilities)
  float* gent;     // [T] upstream gradient of its entropy, in the same units, or null (backward of log probabilities)
  float* ent;      // [T] its entropy (with gent)
  float* resid;    // [T] what bfloat16 took off its target's term (backward of log probabilities with targets)
  int32_t* count;  // [1] counted tokens
};
// Tile of dh's or dw's product, and the sets of workgroups that its K is split over.
struct KPlan {
  int tile = 0, splits = 1;
};
struct VocabDesc {
  const void* h = nullptr;
  int64_t ldh = 0;
  const void* w = nullptr;
  int64_t ldw = 0;
  const int64_t* target = nullptr;  // null (log probabilities only): every token is counted
  int64_t T = 0, d = 0, V = 0;
  bool bf16 = true, backward = false;
  bool fits = true;         // every product's tiles in one launch
  VocabRows rows{};
  void* hc = nullptr;       // [T][ldhc] compact rows of h
  int64_t ldhc = 0;         // whole 128-byte lines, so that a tile's rows take no more lines than they fill
  // forward
  int stat_tile = 0, stat_tiles = 0;  // tile of the product, and column tiles
  float2* stat = nullptr;   // [stat_tiles][T] maximum and sum of a tile's columns
  float* tl = nullptr;      // [T] target's logit of a compact row
  float* loss = nullptr;
  float* lse = nullptr;
  // backward
  const float* lse_in = nullptr;
  const float* dloss = nullptr;
  float scale = 1.f;
  void* p = nullptr;        // [T][piece] gradient of a piece's logits
  int64_t piece = 0;        // a multiple of 256
  KPlan dh_plan, dw_plan;
  float* acc = nullptr;     // [splits][T][d] sums of dh (more than one split or piece)
  float* acc_w = nullptr;   // [splits][piece][d] sums of a piece of dw (more than one split)
  void* dh = nullptr;
  void* dw = nullptr;
  // log probabilities with entropy and alternatives (poetx_token_logprobs*)
  bool token = false;
  float inv_temp = 1.f;     // factor of the logits
  int top = 0;              // alternatives a token
  int64_t chunk = 0;        // compact rows whose logits are held at a time (with alternatives, else all at once, not held)
  float* statu = nullptr;   // [stat_tiles][T] sum of a tile's exponentials times their exponents
  void* rec = nullptr;        // with alternatives, in place of stat and statu: [chunk][stat_tiles] of kTokenRec bytes
  uint16_t* codes = nullptr;  // [chunk][ldl] logits of the rows, below their groups' maxima
  int64_t ldl = 0;            // V, whole tiles
  float* logprob = nullptr;
  float* entropy = nullptr;
  float2* row_stat = nullptr;  // maximum and log of the sum
  int64_t* top_ids = nullptr;
  float* top_logprobs = nullptr;
  const float2* stat_in = nullptr;  // backward: row_stat
  const float* dent = nullptr;    // backward: gradients of the entropies (null: none)
  const float* ent_in = nullptr;  // and the entropies
};
// Sets the tiles, splits and `fits` from the sizes; `lean`: the widest column tiles
// (the fewest pairs) and no splits.
void vocab_plan(VocabDesc& d, bool lean);
void vocab_forward(const VocabDesc& d, hipStream_t stream);
void vocab_backward(const VocabDesc& d, hipStream_t stream);
// The counted tokens' rows to the front (vocab_loss.hip), for both operators.
void vocab_gather(const VocabDesc& d, bool backward, hipStream_t stream);

// Log probabilities of given tokens, entropy and the kTopMost most likely tokens at
// most. Candidates: as many more are ordered as kTopSpare allows (token_logprobs.hip).
constexpr int kTopMost = 64, kTopSpare = 8, kTokenRec = 32;
void token_forward(const VocabDesc& d, hipStream_t stream);
// The gradient of a piece's logits, for vocab_backward; sets a.tiles_n.
struct TileArgs;
void token_dlogits(const VocabDesc& d, TileArgs& a, hipStream_t stream);

// Norm of many tensors, and their scaling (poetx_grad_*).
constexpr int kGradUnit = 16384;  // bytes of a unit of work
inline int64_t grad_units(int64_t n, bool bf16) { return (n * (bf16 ? 2 : 4) + kGradUnit - 1) / kGradUnit; }
struct GradEntry {
  const void* g;
  void* out;
  int64_t n;
  uint32_t first;  // its first unit
  bool bf16;
};
struct GradDesc {
  int64_t count = 0;            // tensors (any of them may be empty)
  const void* const* g = nullptr;
  void* const* out = nullptr;   // null: the norm alone
  const int64_t* n = nullptr;
  const int32_t* dtype = nullptr;
  int32_t bf16_code = 0;
  bool bf16(int64_t i) const { return dtype[i] == bf16_code; }
  float max_norm = 0.f;
  float* norm = nullptr;
  double* part = nullptr;       // [grad_parts(count)]
  GradEntry* table = nullptr;   // [count]
};
int64_t grad_parts(int64_t count);
void grad_norm(const GradDesc& d, hipStream_t stream);

}  // namespace poetx
