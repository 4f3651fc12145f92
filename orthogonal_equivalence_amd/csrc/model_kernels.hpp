// Launchers of the operators around the layer (rmsnorm.hip, linear_i8.hip,
// vocab_loss.hip). All launch on `stream`; their callers have validated the
// sizes (poetx_model.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace poetx {

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
struct VocabRows {
  int2* chunk;     // [T / kVocabChunk, rounded up] counted tokens and largest gradient (more than two chunks)
  int32_t* pos;    // [T]
  int32_t* idx;    // [T]
  int32_t* tgt;    // [T] target of compact row c
  float* g;        // [T] upstream gradient of compact row c, in units of the largest (backward)
  float* unit;     // [1] that unit (backward)
  float* lse;      // [T] lse of compact row c (backward)
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
  const int64_t* target = nullptr;
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
};
// Sets the tiles, splits and `fits` from the sizes; `lean`: the widest column tiles
// (the fewest pairs) and no splits.
void vocab_plan(VocabDesc& d, bool lean);
void vocab_forward(const VocabDesc& d, hipStream_t stream);
void vocab_backward(const VocabDesc& d, hipStream_t stream);

}  // namespace poetx
