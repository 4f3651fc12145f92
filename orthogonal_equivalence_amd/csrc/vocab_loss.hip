// Softmax cross entropy over a vocabulary from hidden rows h [T][d] and the
// vocabulary matrix w [V][d], without the [T][V] logits:
//
//   forward   per 256 x 256 tile of h w^T: each row's maximum and sum of
//             exponentials over the tile's columns, and the target's logit;
//             then lse and loss from the tiles' pairs
//   backward  per piece of the vocabulary: the tiles again, as
//             dl = g (exp(l - lse) - [v = target]) in bfloat16, then
//             dh += dl w and dw = dl^T h on the piece
//
// Both first gather the counted tokens (target in [0, V)) to the front, so
// that the products spend nothing on the others and never see their rows;
// how many there are stays on the device, and tiles past it end at once.
#include "gemm.hpp"
#include "model_kernels.hpp"
#include "tile_gemm.hpp"

namespace poetx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct RowsArgs {
  const int64_t* target;
  int64_t V;
  int T;
  VocabRows r;
  const float* lse_in;  // backward (else null)
  const float* dloss;
  float scale;
};

// Compact row numbers of the counted tokens in token order, and their
// targets; in the backward also their gradients and lse. One workgroup: a
// thread counts and then numbers a run of consecutive tokens.
__global__ void __launch_bounds__(1024) k_vocab_rows(const RowsArgs a) {
  __shared__ int wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.T + 1023) / 1024;
  const int t0 = min(a.T, tid * per), t1 = min(a.T, t0 + per);
  int mine = 0;
  for (int t = t0; t < t1; ++t) {
    const int64_t y = a.target[t];
    mine += y >= 0 && y < a.V;
  }
  int before = mine;  // inclusive scan over the wave
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(before, o);
    if (lane >= o) before += v;
  }
  if (lane == 63) wsum[wave] = before;
  __syncthreads();
  int total = 0, base = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    if (w < wave) base += wsum[w];
    total += wsum[w];
  }
  int c = base + before - mine;
  const float mean = a.scale / static_cast<float>(total);
  for (int t = t0; t < t1; ++t) {
    const int64_t y = a.target[t];
    const bool counted = y >= 0 && y < a.V;
    a.r.pos[t] = counted ? c : -1;
    if (counted) {
      a.r.idx[c] = t;
      a.r.tgt[c] = static_cast<int>(y);
      if (a.lse_in) {
        a.r.g[c] = a.dloss ? a.scale * a.dloss[t] : mean;
        a.r.lse[c] = a.lse_in[t];
      }
      ++c;
    }
  }
  if (tid == 0) *a.r.count = total;
}

// Row t of h to its compact row of hc (a token that is not counted: zeros to
// its row of dh, if there is one). With `pad`, compact rows from the count to
// T are zeroed too, by the workgroup of that number. 16-byte chunks.
__global__ void __launch_bounds__(256) k_vocab_gather(const uint4* h, int64_t ldh, const int32_t* pos,
                                                      const int32_t* count, uint4* hc, uint4* dh, int chunks, bool pad) {
  const int64_t t = blockIdx.x;
  const int p = pos[t];
  const uint4 z = make_uint4(0, 0, 0, 0);
  if (p >= 0) {
    for (int c = threadIdx.x; c < chunks; c += 256) hc[static_cast<int64_t>(p) * chunks + c] = h[t * ldh + c];
  } else if (dh) {
    for (int c = threadIdx.x; c < chunks; c += 256) dh[t * chunks + c] = z;
  }
  if (pad && t >= *count)
    for (int c = threadIdx.x; c < chunks; c += 256) hc[t * chunks + c] = z;
}

// --- bfloat16 tiles -----------------------------------------------------------

struct TileArgs {
  TileOperand A, B;
  VocabRows r;
  int T, d;
  int v0, vn;      // the vocabulary rows [v0, v0 + vn) of this launch
  int tiles_n;     // column tiles of the launch
  // statistics
  float2* stat;
  float* tl;
  // gradient of the logits
  bf16_t* p;
  int64_t ldp;
  // dh, dw
  float* acc32;
  int first, last;
  bf16_t* out;
};

// Tile index of the workgroup among the tiles of the counted rows; false past
// them.
template <int BM>
__device__ __forceinline__ bool vocab_place(int count, int tiles_n, int& tm, int& tn) {
  const int tiles_m = (count + BM - 1) / BM;
  const int bid = static_cast<int>(blockIdx.x);
  if (bid >= tiles_m * tiles_n) return false;
  tile_place(xcd_remap(bid, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  return true;
}

// exp(x) of a logit against a reference, both times log2(e)
__device__ __forceinline__ float exp_rel(float l, float ref2) {
  return __builtin_amdgcn_exp2f(fmaf(l, kLog2e, -ref2));
}

// Joins (m, s) with (m2, s2): sums of 2^(x - m) over disjoint sets. An empty
// set is (-inf, 0).
__device__ __forceinline__ void join_stat(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;
  s = s * __builtin_amdgcn_exp2f(m - ref) + s2 * __builtin_amdgcn_exp2f(m2 - ref);
  // a NaN logit leaves its mark in the sum; fmaxf drops it
  m = top;
}

// Maximum and sum of every row over the tile's columns, in powers of two, and
// the targets' logits.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT, 1) k_vocab_stat(const TileArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];
  const int count = *a.r.count;
  int tm, tn;
  if (!vocab_place<Cfg::BM>(count, a.tiles_n, tm, tn)) return;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A;
  A.rows = count;
  f32x16_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.B, m0, n0, a.d, 0, (a.d + Cfg::BK - 1) / Cfg::BK, smem, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
  float2* red = reinterpret_cast<float2*>(smem);  // [WN][BM]
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
    const int row = tile_row<Cfg>(wm, lane, i);
    const int tcol = m0 + row < count ? a.r.tgt[m0 + row] - n0 : -1;
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int col = tile_col<Cfg>(wn, lane, j, r);
        if (col == tcol) a.tl[m0 + row] = acc[i][j][r];
        m = fmaxf(m, n0 + col < a.vn ? acc[i][j][r] : -INFINITY);
      }
    m *= kLog2e;
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int col = tile_col<Cfg>(wn, lane, j, r);
        s += n0 + col < a.vn ? exp_rel(acc[i][j][r], ref) : 0.f;
      }
    join_stat(m, s, __shfl_xor(m, 32), __shfl_xor(s, 32));
    if (lane < 32) red[wn * Cfg::BM + row] = make_float2(m, s);
  }
  __syncthreads();
  const int row = threadIdx.x;
  if (row < Cfg::BM && m0 + row < count) {
    float2 v = red[row];
#pragma unroll
    for (int w = 1; w < Cfg::WN; ++w) join_stat(v.x, v.y, red[w * Cfg::BM + row].x, red[w * Cfg::BM + row].y);
    a.stat[static_cast<int64_t>(tn) * a.T + m0 + row] = v;
  }
}

// lse and loss of every token from the tiles' pairs: 64 tokens a workgroup,
// 16 waves over every 16th tile.
__global__ void __launch_bounds__(1024) k_vocab_join(const float2* stat, int tiles, const float* tl, const int32_t* pos,
                                                     int T, float* loss, float* lse) {
  __shared__ float2 red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 64 + lane;
  const int c = t < T ? pos[t] : -1;
  float m = -INFINITY, s = 0.f;
  if (c >= 0)
    for (int k = wave; k < tiles; k += 16) {
      const float2 v = stat[static_cast<int64_t>(k) * T + c];
      join_stat(m, s, v.x, v.y);
    }
  red[wave][lane] = make_float2(m, s);
  __syncthreads();
  if (wave || t >= T) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) join_stat(m, s, red[w][lane].x, red[w][lane].y);
  const float l = c >= 0 ? (m + __builtin_amdgcn_logf(s)) * kLn2 : 0.f;
  lse[t] = l;
  loss[t] = c >= 0 ? l - tl[c] : 0.f;
}

// Gradient of the logits of a piece, rounded to bfloat16: p [count][ldp],
// zero in the columns past the vocabulary.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT, 1) k_vocab_dlogits(const TileArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];
  const int count = *a.r.count;
  int tm, tn;
  if (!vocab_place<Cfg::BM>(count, a.tiles_n, tm, tn)) return;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A;
  A.rows = count;
  f32x16_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.B, m0, n0, a.d, 0, (a.d + Cfg::BK - 1) / Cfg::BK, smem, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
    const int row = m0 + tile_row<Cfg>(wm, lane, i);
    const bool in = row < count;
    const int tcol = in ? a.r.tgt[row] - a.v0 - n0 : -1;
    const float ref = in ? a.r.lse[row] * kLog2e : 0.f, g = in ? a.r.g[row] : 0.f;
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int col = tile_col<Cfg>(wn, lane, j, r);
        const float e = exp_rel(acc[i][j][r], ref) - (col == tcol ? 1.f : 0.f);
        acc[i][j][r] = n0 + col < a.vn ? g * e : 0.f;
      }
  }
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    if (m0 + row < count) tile_store8(a.p + static_cast<int64_t>(m0 + row) * a.ldp + n0 + col, v);
  });
}

// dh: the piece's product with its rows of w, added to the earlier pieces'
// sums in float32; the last piece writes the tokens' rows.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT, 1) k_vocab_dh(const TileArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];
  const int count = *a.r.count;
  int tm, tn;
  if (!vocab_place<Cfg::BM>(count, a.tiles_n, tm, tn)) return;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A;
  A.rows = count;
  f32x16_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.B, m0, n0, a.vn, 0, (a.vn + Cfg::BK - 1) / Cfg::BK, smem, acc);
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    const int c = m0 + row, k = n0 + col;
    if (c >= count || k >= a.d) return;
    float o[8];
    float* sum = a.acc32 + static_cast<int64_t>(c) * a.d + k;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i];
    if (!a.first) {
      const float4 s0 = *reinterpret_cast<const float4*>(sum), s1 = *reinterpret_cast<const float4*>(sum + 4);
      o[0] += s0.x; o[1] += s0.y; o[2] += s0.z; o[3] += s0.w;
      o[4] += s1.x; o[5] += s1.y; o[6] += s1.z; o[7] += s1.w;
    }
    if (a.last) tile_store8(a.out + static_cast<int64_t>(a.r.idx[c]) * a.d + k, o);
    else tile_store8(sum, o);
  });
}

// dw rows of a piece: the product over the counted tokens.
template <class Cfg>
__global__ void __launch_bounds__(Cfg::NT, 1) k_vocab_dw(const TileArgs a, int tiles_m) {
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];
  const int count = *a.r.count;
  int tm, tn;
  tile_place(xcd_remap(blockIdx.x, gridDim.x), tiles_m, a.tiles_n, tm, tn);
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A, B = a.B;
  A.rows = count;
  B.rows = count;
  f32x16_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, B, m0, n0, count, 0, (count + Cfg::BK - 1) / Cfg::BK, smem, acc);
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    const int m = m0 + row, k = n0 + col;
    if (m < a.vn && k < a.d) tile_store8(a.out + static_cast<int64_t>(a.v0 + m) * a.d + k, v);
  });
}

// --- float32 -------------------------------------------------------------------

// Running maximum and sum of every compact row over a piece of logits
// p [T][ldp], columns [0, vn), and the targets' logits. A wave per row.
__global__ void __launch_bounds__(256) k_vocab_stat_f32(const float* p, int64_t ldp, int v0, int vn, VocabRows r,
                                                        float2* run, float* tl, int first) {
  const int c = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (c >= *r.count) return;
  const float* row = p + static_cast<int64_t>(c) * ldp;
  float m = -INFINITY;
  for (int v = lane; v < vn; v += 64) m = fmaxf(m, row[v]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  m *= kLog2e;
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
  for (int v = lane; v < vn; v += 64) s += exp_rel(row[v], ref);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane) return;
  const int tv = r.tgt[c] - v0;
  if (tv >= 0 && tv < vn) tl[c] = row[tv];
  if (!first) join_stat(m, s, run[c].x, run[c].y);
  run[c] = make_float2(m, s);
}

__global__ void __launch_bounds__(256) k_vocab_join_f32(const float2* run, const float* tl, const int32_t* pos, int T,
                                                        float* loss, float* lse) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= T) return;
  const int c = pos[t];
  const float l = c >= 0 ? (run[c].x + __builtin_amdgcn_logf(run[c].y)) * kLn2 : 0.f;
  lse[t] = l;
  loss[t] = c >= 0 ? l - tl[c] : 0.f;
}

// Logits of a piece to their gradient, in place; rows past the count zero.
__global__ void __launch_bounds__(256) k_vocab_dlogits_f32(float* p, int64_t ldp, int v0, int vn, VocabRows r, int T) {
  const int c = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (c >= T) return;
  float* row = p + static_cast<int64_t>(c) * ldp;
  if (c >= *r.count) {
    for (int v = lane; v < vn; v += 64) row[v] = 0.f;
    return;
  }
  const float ref = r.lse[c] * kLog2e, g = r.g[c];
  const int tv = r.tgt[c] - v0;
  for (int v = lane; v < vn; v += 64) row[v] = g * (exp_rel(row[v], ref) - (v == tv ? 1.f : 0.f));
}

// dh rows of the counted tokens from the sums
__global__ void __launch_bounds__(256) k_vocab_scatter_f32(const float4* acc, VocabRows r, float4* dh, int chunks) {
  const int64_t c = blockIdx.x;
  if (c >= *r.count) return;
  const int64_t t = r.idx[c];
  for (int k = threadIdx.x; k < chunks; k += 256) dh[t * chunks + k] = acc[c * chunks + k];
}

template <bool KTAIL>
using CfgLogits = TileCfg<2, 256, 256, 2, 4, 2, true, true, KTAIL>;
using CfgDh = TileCfg<2, 256, 256, 2, 4, 2, true, false, false>;
using CfgDw = TileCfg<2, 256, 256, 2, 4, 2, false, false, false>;

int tiles(int64_t n, int b) { return static_cast<int>((n + b - 1) / b); }

void rows_of(const VocabDesc& D, bool backward, hipStream_t st) {
  const RowsArgs a{D.target, D.V, static_cast<int>(D.T), D.rows, backward ? D.lse_in : nullptr, D.dloss, D.scale};
  hipLaunchKernelGGL(k_vocab_rows, dim3(1), dim3(1024), 0, st, a);
  const int es = D.bf16 ? 2 : 4;
  hipLaunchKernelGGL(k_vocab_gather, dim3(static_cast<unsigned>(D.T)), dim3(256), 0, st,
                     static_cast<const uint4*>(D.h), D.ldh * es / 16, D.rows.pos, D.rows.count,
                     static_cast<uint4*>(D.hc), static_cast<uint4*>(backward ? D.dh : nullptr),
                     static_cast<int>(D.d * es / 16), !D.bf16);
}

TileArgs tile_args(const VocabDesc& D) {
  TileArgs a{};
  a.r = D.rows;
  a.T = static_cast<int>(D.T);
  a.d = static_cast<int>(D.d);
  return a;
}

// logits of vocabulary rows [v0, v0 + vn), all compact rows (float32 path)
bool logits_f32(const VocabDesc& D, int64_t v0, int64_t vn, hipStream_t st) {
  GemmDesc g;
  g.A = D.hc;
  g.lda = D.d;
  g.B = static_cast<const float*>(D.w) + v0 * D.ldw;
  g.ldb = D.ldw;
  g.C = D.p;
  g.ldc = D.piece;
  g.M = static_cast<int>(D.T);
  g.N = static_cast<int>(vn);
  g.K = static_cast<int>(D.d);
  return gemm_f32(g, A_KCONTIG, B_KCONTIG, st);
}

}  // namespace

bool vocab_forward(const VocabDesc& D, hipStream_t st) {
  rows_of(D, false, st);
  const int T = static_cast<int>(D.T);
  if (D.bf16) {
    TileArgs a = tile_args(D);
    a.A = {D.hc, D.d, D.T, D.d};
    a.B = {D.w, D.ldw, D.V, D.d};
    a.vn = static_cast<int>(D.V);
    a.tiles_n = tiles(D.V, 256);
    a.stat = D.stat;
    a.tl = D.tl;
    const dim3 grid(static_cast<unsigned>(tiles(D.T, 256)) * a.tiles_n);
    if (D.d % 64) hipLaunchKernelGGL((k_vocab_stat<CfgLogits<true>>), grid, dim3(512), 0, st, a);
    else hipLaunchKernelGGL((k_vocab_stat<CfgLogits<false>>), grid, dim3(512), 0, st, a);
    hipLaunchKernelGGL(k_vocab_join, dim3(tiles(D.T, 64)), dim3(1024), 0, st, D.stat, a.tiles_n, D.tl, D.rows.pos, T,
                       D.loss, D.lse);
    return true;
  }
  for (int64_t v0 = 0; v0 < D.V; v0 += D.piece) {
    const int64_t vn = D.V - v0 < D.piece ? D.V - v0 : D.piece;
    if (!logits_f32(D, v0, vn, st)) return false;
    hipLaunchKernelGGL(k_vocab_stat_f32, dim3(tiles(D.T, 4)), dim3(256), 0, st, static_cast<const float*>(D.p),
                       D.piece, static_cast<int>(v0), static_cast<int>(vn), D.rows, D.run, D.tl, v0 == 0);
  }
  hipLaunchKernelGGL(k_vocab_join_f32, dim3(tiles(D.T, 256)), dim3(256), 0, st, D.run, D.tl, D.rows.pos, T, D.loss,
                     D.lse);
  return true;
}

bool vocab_backward(const VocabDesc& D, hipStream_t st) {
  rows_of(D, true, st);
  for (int64_t v0 = 0; v0 < D.V; v0 += D.piece) {
    const int64_t vn = D.V - v0 < D.piece ? D.V - v0 : D.piece;
    const bool first = v0 == 0, last = v0 + vn >= D.V;
    if (D.bf16) {
      const bf16_t* w = static_cast<const bf16_t*>(D.w) + v0 * D.ldw;
      TileArgs a = tile_args(D);
      a.v0 = static_cast<int>(v0);
      a.vn = static_cast<int>(vn);
      a.first = first;
      a.last = last;
      a.p = static_cast<bf16_t*>(D.p);
      a.ldp = D.piece;
      a.acc32 = D.acc;
      const int tmT = tiles(D.T, 256);
      // dl
      a.A = {D.hc, D.d, D.T, D.d};
      a.B = {w, D.ldw, vn, D.d};
      a.tiles_n = tiles(vn, 256);
      const dim3 grid(static_cast<unsigned>(tmT) * a.tiles_n);
      if (D.d % 64) hipLaunchKernelGGL((k_vocab_dlogits<CfgLogits<true>>), grid, dim3(512), 0, st, a);
      else hipLaunchKernelGGL((k_vocab_dlogits<CfgLogits<false>>), grid, dim3(512), 0, st, a);
      // dh: the columns of p up to the next multiple of 64 are zero, and so
      // are rows past the operand's end
      a.A = {D.p, D.piece, D.T, D.piece};
      a.B = {w, D.ldw, vn, D.d};
      a.tiles_n = tiles(D.d, 256);
      a.out = static_cast<bf16_t*>(D.dh);
      hipLaunchKernelGGL((k_vocab_dh<CfgDh>), dim3(static_cast<unsigned>(tmT) * a.tiles_n), dim3(512), 0, st, a);
      // dw
      a.A = {D.p, D.piece, D.T, D.piece};
      a.B = {D.hc, D.d, D.T, D.d};
      a.out = static_cast<bf16_t*>(D.dw);
      const int tmV = tiles(vn, 256);
      hipLaunchKernelGGL((k_vocab_dw<CfgDw>), dim3(static_cast<unsigned>(tmV) * a.tiles_n), dim3(512), 0, st, a, tmV);
      continue;
    }
    if (!logits_f32(D, v0, vn, st)) return false;
    hipLaunchKernelGGL(k_vocab_dlogits_f32, dim3(tiles(D.T, 4)), dim3(256), 0, st, static_cast<float*>(D.p), D.piece,
                       static_cast<int>(v0), static_cast<int>(vn), D.rows, static_cast<int>(D.T));
    GemmDesc g;
    g.A = D.p;
    g.lda = D.piece;
    g.B = static_cast<const float*>(D.w) + v0 * D.ldw;
    g.ldb = D.ldw;
    g.C = D.acc;
    g.ldc = D.d;
    g.M = static_cast<int>(D.T);
    g.N = static_cast<int>(D.d);
    g.K = static_cast<int>(vn);
    if (!first) {
      g.D = D.acc;
      g.ldd = D.d;
      g.beta = 1.f;
    }
    if (!gemm_f32(g, A_KCONTIG, B_NCONTIG, st)) return false;
    GemmDesc u;
    u.A = D.p;
    u.lda = D.piece;
    u.B = D.hc;
    u.ldb = D.d;
    u.C = static_cast<float*>(D.dw) + v0 * D.d;
    u.ldc = D.d;
    u.M = static_cast<int>(vn);
    u.N = static_cast<int>(D.d);
    u.K = static_cast<int>(D.T);
    if (!gemm_f32(u, A_MCONTIG, B_NCONTIG, st)) return false;
  }
  if (!D.bf16)
    hipLaunchKernelGGL(k_vocab_scatter_f32, dim3(static_cast<unsigned>(D.T)), dim3(256), 0, st,
                       reinterpret_cast<const float4*>(D.acc), D.rows, static_cast<float4*>(D.dh),
                       static_cast<int>(D.d / 4));
  return true;
}

}  // namespace poetx
