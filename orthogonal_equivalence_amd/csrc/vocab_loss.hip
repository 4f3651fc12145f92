// Softmax cross entropy over a vocabulary from hidden rows h [T][d] and the
// vocabulary matrix w [V][d], without the [T][V] logits:
//
//   forward   per tile of h w^T: each row's maximum and sum of exponentials
//             over the tile's columns, and the target's logit; then lse and loss
//             from the tiles' pairs
//   backward  per piece of the vocabulary: the tiles again, as
//             dl = g (exp(l - lse) - [v = target]) in the storage type, then
//             dh += dl w and dw = dl^T h on the piece
//
// Both first gather the counted tokens (target in [0, V)) to the front, so
// that the products spend nothing on the others and never see their rows;
// how many there are stays on the device, and tiles past it end at once.
//
// 8 T d V operations, a quarter of them for logits a second time: kept in
// float32 they would be the memory that the operator is there to save, in
// bfloat16 they would be off by 2^-9 of their size, which at logits of 10 to 20
// is a few percent of the exponentials. Large calls are bound by the matrix cores at the chip's power
// limit (a clock of 1.9 to 2.0 GHz): T = 8192, d = 4096, V = 131072 in 26.5 ms,
// 1.33 PFLOP/s, where the library's plain products of these shapes reach 1.47 to
// 1.57. Few tokens are bound by the bytes of w and dw (d = 4096, V = 131072, T =
// 64: forward 0.21 ms for 1.07 GB, backward 0.80 ms for 3.2), small calls by the
// latency of six launches.
#include "model_kernels.hpp"
#include "tile_gemm.hpp"

#include <algorithm>

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
  const uint4* h;  // rows in 16-byte chunks
  int64_t ldh;
  uint4* hc;
  int64_t ldhc;
  uint4* dh;       // backward
  int chunks;
};

// |v|, or 0 where it is not finite: such a gradient stays with its own token
__device__ __forceinline__ float finite_size(float v) {
  v = fabsf(v);
  return v < INFINITY ? v : 0.f;
}

// Counted tokens of every kVocabChunk tokens and their largest gradient, for
// the gather of many tokens.
__global__ void __launch_bounds__(1024) k_vocab_count(const RowsArgs a) {
  __shared__ int red[16];
  __shared__ float redg[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n = 0;
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kVocabChunk / 1024; ++i) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kVocabChunk + i * 1024 + tid;
    if (t >= a.T) break;
    const int64_t y = a.target[t];
    if (y < 0 || y >= a.V) continue;
    ++n;
    if (a.dloss) most = fmaxf(most, finite_size(a.scale * a.dloss[t]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    n += __shfl_xor(n, o);
    most = fmaxf(most, __shfl_xor(most, o));
  }
  if (lane == 0) {
    red[wave] = n;
    redg[wave] = most;
  }
  __syncthreads();
  if (tid) return;
  for (int w = 1; w < 16; ++w) {
    n += red[w];
    most = fmaxf(most, redg[w]);
  }
  a.r.chunk[blockIdx.x] = make_int2(n, __float_as_int(most));
}

// Gathers the counted tokens' rows of h to the front of hc in token order, with
// their targets and, in the backward, their gradients and lse; a token that is
// not counted gets zeros in its row of dh. A workgroup does `per` tokens, 64 at
// a time, and finds its first compact row by counting the targets before its
// own, all workgroups at the same time; with CHUNKS, from the counts of
// k_vocab_count, those of its own chunk only. The rows' bytes, read and written
// once, take half of its time (T = 4096, d = 4096: 67 MB in 25 to 30 us, 13 at a
// copy's rate): 6 us pass before the first row, and the compiler keeps the eight
// loads that a lane has in flight in scratch memory, 144 bytes a lane.
template <int NW, bool CHUNKS>
__global__ void __launch_bounds__(64 * NW) k_vocab_gather(const RowsArgs a, int per) {
  __shared__ int red[2][NW];
  __shared__ float redg[NW];
  __shared__ int pos[64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.x * per, t1 = min(a.T, t0 + per);
  int before = 0, total = 0;
  float most = 0.f;
  if constexpr (CHUNKS)
    for (int k = tid; k < (a.T + kVocabChunk - 1) / kVocabChunk; k += 64 * NW) {
      const int2 c = a.r.chunk[k];
      total += c.x;
      before += (k + 1) * kVocabChunk <= t0 ? c.x : 0;
      most = fmaxf(most, __int_as_float(c.y));
    }
#pragma unroll 4
  for (int t = (CHUNKS ? t0 / kVocabChunk * kVocabChunk : 0) + tid; t < (CHUNKS ? t0 : a.T); t += 64 * NW) {
    const int64_t y = a.target[t];
    const int c = y >= 0 && y < a.V;
    before += t < t0 ? c : 0;
    if constexpr (CHUNKS) continue;
    total += c;
    if (a.dloss && c) most = fmaxf(most, finite_size(a.scale * a.dloss[t]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    before += __shfl_xor(before, o);
    total += __shfl_xor(total, o);
    most = fmaxf(most, __shfl_xor(most, o));
  }
  if (lane == 0) {
    red[0][wave] = before;
    red[1][wave] = total;
    redg[wave] = most;
  }
  __syncthreads();
  int base = 0;
  total = 0;
  most = 0.f;  // gradients in units of their largest: 1 for all of a mean loss's
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    base += red[0][w];
    total += red[1][w];
    most = fmaxf(most, redg[w]);
  }
  if (blockIdx.x == 0 && tid == 0) {
    *a.r.count = total;
    // with no token counted the sums are empty, and 0 whatever the scale
    if (a.lse_in) *a.r.unit = a.dloss ? most : total ? a.scale / static_cast<float>(total) : 0.f;
  }
  for (int b = t0; b < t1; b += 64) {
    // every wave numbers the 64 tokens alike; the first writes
    const int t = b + lane;
    const int64_t y = t < t1 ? a.target[t] : -1;
    const bool counted = y >= 0 && y < a.V;
    const unsigned long long m = __ballot(counted);
    const int p = counted ? base + __popcll(m & ((1ull << lane) - 1)) : -1;
    base += __popcll(m);
    if (wave == 0 && t < t1) {
      pos[lane] = p;
      a.r.pos[t] = p;
      if (counted) {
        a.r.idx[p] = t;
        a.r.tgt[p] = static_cast<int>(y);
        if (a.lse_in) {
          const float g = a.dloss ? a.scale * a.dloss[t] : 1.f;
          a.r.g[p] = a.dloss && most != 0.f ? g / most : g;
          a.r.lse[p] = a.lse_in[t];
        }
      }
    }
    __syncthreads();
    const int n = min(64, t1 - b);
    for (int i = wave; i < n; i += NW) {
      const int to = pos[i];
      if (to >= 0) {
        const uint4* src = a.h + (b + i) * a.ldh;
        uint4* dst = a.hc + to * a.ldhc;
        for (int c = lane; c < a.chunks; c += 512) {  // 8 KB a wave at a time
          uint4 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (c + u * 64 < a.chunks) v[u] = src[c + u * 64];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (c + u * 64 < a.chunks) dst[c + u * 64] = v[u];
        }
      } else if (a.dh) {
        uint4* dst = a.dh + static_cast<int64_t>(b + i) * a.chunks;
        for (int c = lane; c < a.chunks; c += 64) dst[c] = make_uint4(0, 0, 0, 0);
      }
    }
    __syncthreads();
  }
}

// --- tiles ----------------------------------------------------------------------

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
  void* p;
  int64_t ldp;
  // dh, dw
  float* acc32;
  int first, last;
  int splits;      // of K over workgroups
  void* out;
  int tile;        // of the wide ones: dw's, and dh's where it is split
};

// storage of a tile's element size
template <int ES>
struct Elem {
  typedef bf16_t type;
};
template <>
struct Elem<4> {
  typedef float type;
};

// The tiles of 256 columns, one workgroup a CU, come in one kernel, which picks
// among them.
template <bool AKC, bool BKC, bool KTAIL>
struct WideTiles {
  typedef TileCfg<2, 128, 256, 2, 4, 3, AKC, BKC, KTAIL> T128;
  typedef TileCfg<2, 256, 256, 2, 4, 2, AKC, BKC, KTAIL> T256;
  // (192 rows do not divide into the whole-row loads of an operand with K as its rows)
  typedef TileCfg<2, AKC ? 192 : 256, 256, 2, 4, 2, AKC, BKC, KTAIL> T192;
  static constexpr int NT = 512, BN = 256;
  static constexpr int LDS = T128::LDS > T256::LDS ? T128::LDS : T256::LDS;
};
template <class C>
struct IsWide {
  static constexpr bool value = false;
};
template <bool AKC, bool BKC, bool KTAIL>
struct IsWide<WideTiles<AKC, BKC, KTAIL>> {
  static constexpr bool value = true;
};

// the same tiles for dw's operands, which both have K as their rows
template <class C>
struct Turned;
template <int ES, int BM, int BN, int WM, int WN, int NS, int KG>
struct Turned<TileCfg<ES, BM, BN, WM, WN, NS, true, false, false, KG>> {
  typedef TileCfg<ES, BM, BN, WM, WN, NS, false, false, false, KG> type;
};
template <>
struct Turned<WideTiles<true, false, false>> {
  typedef WideTiles<false, false, false> type;
};

// Which of them for the counted rows, whose number the host does not know: the
// cheapest whose tiles fit the launch (T = 1111 of which 555 count, d = 2056, V
// = 50021, this product: 143 us with three rounds of 192 rows and 166 with three of
// 256 where w is in the last-level cache, 178 and 185 where it is not).
__device__ __forceinline__ int pick_wide(int rows, int tiles_n, int most) {
  int best = kTile256;
  float least = INFINITY;
#pragma unroll
  for (int k = kTile128x256; k <= kTile256; ++k) {
    const int bm = kTileCosts[k].bm;
    const int64_t n = static_cast<int64_t>((rows + bm - 1) / bm) * tiles_n;
    const float us = static_cast<float>((n + 255) / 256) * static_cast<float>(kTileCosts[k].us);
    if (n <= most && us < least) {
      best = k;
      least = us;
    }
  }
  return best;
}

// Tile index of a workgroup, number bid, among the tiles of the counted rows;
// false past them.
template <int BM>
__device__ __forceinline__ bool vocab_place(int bid, int count, int tiles_n, int& tm, int& tn) {
  const int tiles_m = (count + BM - 1) / BM;
  if (bid >= tiles_m * tiles_n) return false;
  tile_place(xcd_remap(bid, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  return true;
}

// exp(l - ref). The difference is taken first, exact where the two are near: as one
// fused step against ref in powers of two (no faster, the products bound these
// kernels) its rounding, 1e-5 at logits of 200, would be in every term.
__device__ __forceinline__ float exp_rel(float l, float ref) {
  return __builtin_amdgcn_exp2f((l - ref) * kLog2e);
}

// Joins (m, s) with (m2, s2): sums of exp(x - m) over disjoint sets whose largest
// is m. An empty set is (-inf, 0), any other s at least 1.
__device__ __forceinline__ void join_stat(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;
  s = s * exp_rel(m, ref) + s2 * exp_rel(m2, ref);
  // a NaN logit leaves its mark in the sum; fmaxf drops it
  m = top;
}

// Columns of the tile from `left` on (past the vocabulary) set to v; nothing
// to do in any but the last tile of a row.
template <class Cfg>
__device__ __forceinline__ void mask_columns(f32x4_t (&acc)[Cfg::TM][Cfg::TN], int wn, int lane, int left, float v) {
  if (left >= Cfg::BN) return;
#pragma unroll
  for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool past = tile_col<Cfg>(wn, lane, j, r) >= left;
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i) acc[i][j][r] = past ? v : acc[i][j][r];
    }
}

// Maximum and sum of every row over the tile's columns, and the targets' logits.
// The exponentials come from the sums as they lie in the registers (T = 8192, d
// = 4096, V = 131072: 6.4 ms, 1.38 PFLOP/s, matrix cores busy in 72% of the
// cycles).
template <class Cfg>
__device__ __forceinline__ void stat_tile(const TileArgs& a, int bid, int count, char* smem) {
  int tm, tn;
  if (!vocab_place<Cfg::BM>(bid, count, a.tiles_n, tm, tn)) return;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A;
  A.rows = count;
  f32x4_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.B, m0, n0, 0, (a.d + Cfg::BK - 1) / Cfg::BK, smem, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
  float2* red = reinterpret_cast<float2*>(smem);  // [WN][BM]
  // the first K group's waves hold the sums
  if (wave < Cfg::NW) {
    mask_columns<Cfg>(acc, wn, lane, a.vn - n0, -INFINITY);
#pragma unroll
    for (int i = 0; i < Cfg::TM; ++i) {
      const int row = tile_row<Cfg>(wm, lane, i);
      const int tcol = m0 + row < count ? a.r.tgt[m0 + row] - n0 : -1;
      if (__any(static_cast<unsigned>(tcol - wn * Cfg::WTN) < Cfg::WTN)) {
#pragma unroll
        for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (tile_col<Cfg>(wn, lane, j, r) == tcol) a.tl[m0 + row] = acc[i][j][r];
      }
      float m = acc[i][0][0], s = 0.f;
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) s += exp_rel(acc[i][j][r], ref);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (lane < 16) red[wn * Cfg::BM + row] = make_float2(m, s);
    }
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

template <class C>
__global__ void __launch_bounds__(C::NT, 1) k_vocab_stat(const TileArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int bid = blockIdx.x, count = *a.r.count;
  if constexpr (IsWide<C>::value) {
    switch (pick_wide(count, a.tiles_n, gridDim.x)) {
      case kTile128x256: stat_tile<typename C::T128>(a, bid, count, smem); return;
      case kTile192x256: stat_tile<typename C::T192>(a, bid, count, smem); return;
      default: stat_tile<typename C::T256>(a, bid, count, smem); return;
    }
  } else {
    stat_tile<C>(a, bid, count, smem);
  }
}

// lse = m + log s and loss = (m - l[target]) + log s of every token from the
// tiles' pairs: two terms that are never negative, and exact where the target is
// the maximum (lse less the target's logit would cancel to the rounding of lse,
// 1.5e-5 and of either sign at logits of 200). N tokens a workgroup, 1024
// / N threads a token over the tiles. Bound by latencies: 8 tokens (a row's
// pairs of one 64-byte piece) for few tokens with tiles for that many threads,
// else 64 (T = 16, 2048 tiles: 8 us, 64 tokens 25; T = 8192, 512 tiles: 16 us
// and 10; T = 40000, one tile: 22 us and 5).
template <int N>
__global__ void __launch_bounds__(1024) k_vocab_join(const float2* stat, int tiles, const float* tl, const int32_t* pos,
                                                     int T, float* loss, float* lse) {
  __shared__ float2 red[16][N];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * N + lane % N;
  const int c = t < T ? pos[t] : -1;
  float m = -INFINITY, s = 0.f;
  if (c >= 0)
#pragma unroll 4
    for (int k = threadIdx.x / N; k < tiles; k += 1024 / N) {
      const float2 v = stat[static_cast<int64_t>(k) * T + c];
      join_stat(m, s, v.x, v.y);
    }
#pragma unroll
  for (int o = N; o < 64; o <<= 1) join_stat(m, s, __shfl_xor(m, o), __shfl_xor(s, o));
  if (lane < N) red[wave][lane] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x >= N || t >= T) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) join_stat(m, s, red[w][lane].x, red[w][lane].y);
  const float log_s = __builtin_amdgcn_logf(s) * kLn2;
  lse[t] = c >= 0 ? m + log_s : 0.f;
  loss[t] = c >= 0 ? (m - tl[c]) + log_s : 0.f;
}

// Gradient of the logits of a piece in the storage type, without the common
// factor `unit`, which the products' epilogues put back in float32: a factor
// rounded with the target's entries, which outweigh the rest, would shift all
// of them alike (with g = 1 / count in bfloat16, 0.3% of dh and dw in place of
// 0.17%). p [count][ldp], zero in the columns past the vocabulary.
//
// The probabilities are off by the float lse's own half step (8e-6 of them at an lse
// of 200). Where that takes the target's p - 1 past 0, it is 0, as p is at most 1.
template <class Cfg>
__device__ __forceinline__ void dlogits_tile(const TileArgs& a, int bid, int count, char* smem) {
  int tm, tn;
  if (!vocab_place<Cfg::BM>(bid, count, a.tiles_n, tm, tn)) return;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A;
  A.rows = count;
  f32x4_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.B, m0, n0, 0, (a.d + Cfg::BK - 1) / Cfg::BK, smem, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
    const int row = m0 + tile_row<Cfg>(wm, lane, i);
    const bool in = row < count;
    const int at = in ? row : m0;  // rows past the count are not stored
    const int tcol = a.r.tgt[at] - a.v0 - n0;
    const float lse = a.r.lse[at], g = a.r.g[at];
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = g * exp_rel(acc[i][j][r], lse);
    if (__any(static_cast<unsigned>(tcol - wn * Cfg::WTN) < Cfg::WTN)) {
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (tile_col<Cfg>(wn, lane, j, r) != tcol) continue;
          const float dl = acc[i][j][r] - g;
          acc[i][j][r] = (g > 0.f && dl > 0.f) || (g < 0.f && dl < 0.f) ? 0.f : dl;  // NaN stays
        }
    }
  }
  mask_columns<Cfg>(acc, wn, lane, a.vn - n0, 0.f);
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    auto* p = static_cast<typename Elem<Cfg::ES>::type*>(a.p);
    if (m0 + row < count) tile_store8(p + static_cast<int64_t>(m0 + row) * a.ldp + n0 + col, v);
  });
}

template <class C>
__global__ void __launch_bounds__(C::NT, 1) k_vocab_dlogits(const TileArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int bid = blockIdx.x, count = *a.r.count;
  if constexpr (IsWide<C>::value) {
    switch (pick_wide(count, a.tiles_n, gridDim.x)) {
      case kTile128x256: dlogits_tile<typename C::T128>(a, bid, count, smem); return;
      case kTile192x256: dlogits_tile<typename C::T192>(a, bid, count, smem); return;
      default: dlogits_tile<typename C::T256>(a, bid, count, smem); return;
    }
  } else {
    dlogits_tile<C>(a, bid, count, smem);
  }
}

// dh: the piece's product with its rows of w, added to the earlier pieces'
// sums in float32; the last piece writes the tokens' rows. Where the tiles of
// few tokens leave CUs idle, the piece's rows are split over `splits` sets of
// workgroups with sums of their own, which k_vocab_join_splits adds up.
template <class Cfg>
__device__ __forceinline__ void dh_tile(const TileArgs& a, int bid, int nh, int count, char* smem) {
  const int tiles_h = nh / a.splits, split = bid / tiles_h;
  int tm, tn;
  if (!vocab_place<Cfg::BM>(bid % tiles_h, count, a.tiles_n, tm, tn)) return;
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A;
  A.rows = count;
  f32x4_t acc[Cfg::TM][Cfg::TN];
  const int steps = (a.vn + Cfg::BK - 1) / Cfg::BK, per = (steps + a.splits - 1) / a.splits;
  tile_product<Cfg>(A, a.B, m0, n0, split * per, min(steps, (split + 1) * per), smem, acc);
  const float unit = *a.r.unit;
  float* const sums = a.acc32 + static_cast<int64_t>(split) * a.T * a.d;
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    const int c = m0 + row, k = n0 + col;
    if (c >= count || k >= a.d) return;
    float o[8];
    float* sum = sums + static_cast<int64_t>(c) * a.d + k;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i];
    if (!a.first) {
      const float4 s0 = *reinterpret_cast<const float4*>(sum), s1 = *reinterpret_cast<const float4*>(sum + 4);
      o[0] += s0.x; o[1] += s0.y; o[2] += s0.z; o[3] += s0.w;
      o[4] += s1.x; o[5] += s1.y; o[6] += s1.z; o[7] += s1.w;
    }
    if (a.last && a.splits == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= unit;
      tile_store8(static_cast<typename Elem<Cfg::ES>::type*>(a.out) + static_cast<int64_t>(a.r.idx[c]) * a.d + k, o);
    } else {
      tile_store8(sum, o);
    }
  });
}

// Rows of dh (the counted tokens') or of a piece of dw from the splits' sums, 8
// features a thread. `rows`: of one split's sums.
template <typename T, bool DH>
__global__ void __launch_bounds__(256) k_vocab_join_splits(const TileArgs a, int rows) {
  const int chunks = a.d / 8;
  const int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const int64_t c = i / chunks;
  if (c >= (DH ? *a.r.count : rows)) return;
  const int k = static_cast<int>(i % chunks) * 8;
  float o[8] = {};
  const float* sum = a.acc32 + c * a.d + k;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s, sum += static_cast<int64_t>(rows) * a.d) {
    const float4 s0 = *reinterpret_cast<const float4*>(sum), s1 = *reinterpret_cast<const float4*>(sum + 4);
    o[0] += s0.x; o[1] += s0.y; o[2] += s0.z; o[3] += s0.w;
    o[4] += s1.x; o[5] += s1.y; o[6] += s1.z; o[7] += s1.w;
  }
  const float unit = *a.r.unit;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] *= unit;
  tile_store8(static_cast<T*>(a.out) + (DH ? static_cast<int64_t>(a.r.idx[c]) : a.v0 + c) * a.d + k, o);
}

// dw rows of a piece: the product over the counted tokens, split over sets of
// workgroups where the tiles of a small vocabulary leave CUs idle.
template <class Cfg>
__device__ __forceinline__ void dw_tile(const TileArgs& a, int bid, int count, char* smem) {
  const int tiles_m = (a.vn + Cfg::BM - 1) / Cfg::BM, tiles_w = tiles_m * a.tiles_n, split = bid / tiles_w;
  int tm, tn;
  tile_place(xcd_remap(bid % tiles_w, tiles_w), tiles_m, a.tiles_n, tm, tn);
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  TileOperand A = a.A, B = a.B;
  A.rows = count;
  B.rows = count;
  f32x4_t acc[Cfg::TM][Cfg::TN];
  const int steps = (count + Cfg::BK - 1) / Cfg::BK, per = (steps + a.splits - 1) / a.splits;
  tile_product<Cfg>(A, B, m0, n0, split * per, min(steps, (split + 1) * per), smem, acc);
  const float unit = *a.r.unit;
  float* const sums = a.acc32 + static_cast<int64_t>(split) * a.vn * a.d;
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    const int m = m0 + row, k = n0 + col;
    if (m >= a.vn || k >= a.d) return;
    if (a.splits > 1) {
      tile_store8(sums + static_cast<int64_t>(m) * a.d + k, v);
      return;
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = v[i] * unit;
    tile_store8(static_cast<typename Elem<Cfg::ES>::type*>(a.out) + static_cast<int64_t>(a.v0 + m) * a.d + k, o);
  });
}

template <class CH>
__device__ __forceinline__ void dh_part(const TileArgs& a, int bid, int nh, int count, char* smem) {
  if constexpr (IsWide<CH>::value) {
    switch (a.splits == 1 ? pick_wide(count, a.tiles_n, nh) : a.tile) {
      case kTile128x256: dh_tile<typename CH::T128>(a, bid, nh, count, smem); return;
      case kTile192x256: dh_tile<typename CH::T192>(a, bid, nh, count, smem); return;
      default: dh_tile<typename CH::T256>(a, bid, nh, count, smem); return;
    }
  } else {
    dh_tile<CH>(a, bid, nh, count, smem);
  }
}
template <class CW>
__device__ __forceinline__ void dw_part(const TileArgs& a, int bid, int count, char* smem) {
  if constexpr (IsWide<CW>::value) {
    if (a.tile == kTile128x256) dw_tile<typename CW::T128>(a, bid, count, smem);
    else dw_tile<typename CW::T256>(a, bid, count, smem);
  } else {
    dw_tile<CW>(a, bid, count, smem);
  }
}

// dh and dw of a piece: dh's nh workgroups, then dw's, in one launch where both
// take the same kind of tile, and else in two (NoTiles for the other's). One
// launch is one latency and one tail: T = 256, d = 512, V = 1000 in float, loss
// and gradients 40.6 us against 46.1. T = 8192, d = 4096, 16384 rows of w: 1.67
// ms, 1.32 PFLOP/s, operands with K as their rows through transposed LDS reads.
struct NoTiles {
  static constexpr int NT = 0, LDS = 0;
};
template <class CH, class CW>
__global__ void __launch_bounds__(CH::NT ? CH::NT : CW::NT, 1) k_vocab_grads(const TileArgs h, const TileArgs w,
                                                                             int nh) {
  __shared__ __attribute__((aligned(1024))) char smem[CH::LDS > CW::LDS ? CH::LDS : CW::LDS];
  const int bid = blockIdx.x, count = *h.r.count;
  if constexpr (CH::NT != 0) {
    if (CW::NT == 0 || bid < nh) {
      dh_part<CH>(h, bid, nh, count, smem);
      return;
    }
  }
  if constexpr (CW::NT != 0) dw_part<CW>(w, bid - nh, count, smem);
}

int tiles(int64_t n, int b) { return static_cast<int>((n + b - 1) / b); }

int pick(int64_t M, int64_t N, bool bf16) {
  if (bf16) return pick_tile(kTileCosts, kTileKinds, M, N);
  return pick_tile(kTileCostsF32, kTileKindsF32, M, N);
}
// workgroups of tile t over M x N
int pick_count(int t, int64_t M, int64_t N, bool bf16) {
  const TileCost& c = bf16 ? kTileCosts[t] : kTileCostsF32[t];
  return tiles(M, c.bm) * tiles(N, c.bn);
}
// the kernel that has the tile: the wide ones share one
int kernel_of(int t, bool bf16) { return bf16 && t > kTile128x256 ? kTile128x256 : t; }

// f(config) for the element size and kernel, K-contiguous operands or not
template <bool AKC, bool BKC, bool KTAIL, class F>
void with_tile(bool bf16, int kernel, F&& f) {
  if (!bf16) {
    switch (kernel) {
      case kTileF32: f(TileCfg<4, 32, 32, 1, 1, 2, AKC, BKC, KTAIL, 8>{}); return;
      case kTileF64: f(TileCfg<4, 64, 64, 2, 2, 3, AKC, BKC, KTAIL, 2>{}); return;
      default: f(TileCfg<4, 128, 128, 2, 4, 3, AKC, BKC, KTAIL>{}); return;
    }
  }
  switch (kernel) {
    case kTile64x2: f(TileCfg<2, 64, 64, 2, 2, 3, AKC, BKC, KTAIL, 2>{}); return;
    case kTile64: f(TileCfg<2, 64, 64, 2, 2, 4, AKC, BKC, KTAIL>{}); return;
    case kTile128: f(TileCfg<2, 128, 128, 2, 4, 4, AKC, BKC, KTAIL>{}); return;
    default: f(WideTiles<AKC, BKC, KTAIL>{}); return;
  }
}
template <class F>
void with_logits_tile(bool bf16, int kernel, int64_t d, F&& f) {
  if (d % (bf16 ? 64 : 32)) with_tile<true, true, true>(bf16, kernel, f);
  else with_tile<true, true, false>(bf16, kernel, f);
}

void gather_rows(const VocabDesc& D, bool backward, hipStream_t st) {
  const int es = D.bf16 ? 2 : 4, T = static_cast<int>(D.T);
  const RowsArgs a{D.target, D.V, T, D.rows, backward ? D.lse_in : nullptr, D.dloss, D.scale,
                   static_cast<const uint4*>(D.h), D.ldh * es / 16, static_cast<uint4*>(D.hc), D.ldhc * es / 16,
                   static_cast<uint4*>(backward ? D.dh : nullptr), static_cast<int>(D.d * es / 16)};
  // a row a wave; few tokens on as many CUs as they have fours (d = 4096, h not in
  // the cache, NW = 4 against 16: T = 1111 13.8 us, 16.5; 2048 15.5, 16.6; 4096
  // 28.6, 26.2; 8192 64.8, 53.5); every workgroup reads all targets where that costs
  // no more than a launch of counts (T = 8192: 53.5 us against 49.5 + 5.4; T = 65536,
  // d = 512: 229 us against 40.8 + 5.2)
  if (T <= 2048) {
    hipLaunchKernelGGL((k_vocab_gather<4, false>), dim3(tiles(T, 4)), dim3(256), 0, st, a, 4);
  } else if (T <= 2 * kVocabChunk) {
    hipLaunchKernelGGL((k_vocab_gather<16, false>), dim3(tiles(T, 16)), dim3(1024), 0, st, a, 16);
  } else {
    const int per = T <= 16384 ? 16 : 64;
    hipLaunchKernelGGL(k_vocab_count, dim3(tiles(T, kVocabChunk)), dim3(1024), 0, st, a);
    hipLaunchKernelGGL((k_vocab_gather<16, true>), dim3(tiles(T, per)), dim3(1024), 0, st, a, per);
  }
}

TileArgs tile_args(const VocabDesc& D) {
  TileArgs a{};
  a.r = D.rows;
  a.T = static_cast<int>(D.T);
  a.d = static_cast<int>(D.d);
  return a;
}

// Tile and splits of a product together: rounds of workgroups, each of steps /
// splits K steps, and the sums' bytes (d = 4096, V = 131072: dh of 16 tokens 225
// us, 580 unsplit; backward of 600 tokens 2.13 ms, 2.70; d = 1024, V = 32000, 64
// tokens: backward 67 us, 171; T = 65536, d = 512, V = 100: dw split, backward
// 195 us, 422). Tiles that fill the CUs a few times over are not split.
KPlan k_plan(int64_t M, int64_t N, int64_t K, bool bf16, bool no_192, int most_splits) {
  const TileCost* costs = bf16 ? kTileCosts : kTileCostsF32;
  const int kinds = bf16 ? static_cast<int>(kTileKinds) : static_cast<int>(kTileKindsF32);
  const int steps = static_cast<int>((K + (bf16 ? 63 : 31)) / (bf16 ? 64 : 32));
  KPlan best{};
  double least = INFINITY;
  for (int t = 0; t < kinds; ++t) {
    if (bf16 && no_192 && t == kTile192x256) continue;
    const int64_t n = ((M + costs[t].bm - 1) / costs[t].bm) * ((N + costs[t].bn - 1) / costs[t].bn);
    const double step = costs[t].us / (bf16 ? 32 : 1);
    for (int s = 1; s <= most_splits && (s == 1 || (steps >= 8 * s && n * s <= 4 * costs[t].slots)); ++s) {
      double us = static_cast<double>((n * s + costs[t].slots - 1) / costs[t].slots) *
                  static_cast<double>((steps + s - 1) / s) * step;
      if (s > 1) us += 4.0 + static_cast<double>(M) * static_cast<double>(N) * 8.0 * s / 4e6;
      if (us < least) {
        least = us;
        best.tile = t;
        best.splits = s;
      }
    }
  }
  return best;
}

}  // namespace

void vocab_plan(VocabDesc& D, bool lean) {
  const TileCost* t = D.bf16 ? kTileCosts : kTileCostsF32;
  auto fits = [&](int tile, int64_t M, int64_t N) { D.fits = D.fits && tiles_fit(t[tile], M, N); };
  D.fits = true;
  D.stat_tile = !lean    ? pick(D.T, D.V, D.bf16)
                : D.bf16 ? kTile128x256 + pick_tile(kTileCosts + kTile128x256, kTileKinds - kTile128x256, D.T, D.V)
                         : kTileF128;
  D.stat_tiles = tiles(D.V, t[D.stat_tile].bn);
  fits(D.stat_tile, D.T, D.V);  // the backward refuses what the forward does
  if (!D.backward) return;
  const int64_t most = std::min(D.V, D.piece), last = D.V % D.piece;
  const int splits = lean ? 1 : 16;
  D.dh_plan = k_plan(D.T, D.d, most, D.bf16, false, splits);
  D.dw_plan = k_plan(most, D.d, D.T, D.bf16, true, splits);
  fits(pick(D.T, most, D.bf16), D.T, most);
  if (last) fits(pick(D.T, last, D.bf16), D.T, last);
  fits(D.dh_plan.tile, D.T, D.d * D.dh_plan.splits);
  fits(D.dw_plan.tile, most, D.d * D.dw_plan.splits);
}

void vocab_forward(const VocabDesc& D, hipStream_t st) {
  gather_rows(D, false, st);
  const int T = static_cast<int>(D.T);
  TileArgs a = tile_args(D);
  a.A = {D.hc, D.ldhc, D.T, D.d};
  a.B = {D.w, D.ldw, D.V, D.d};
  a.vn = static_cast<int>(D.V);
  a.stat = D.stat;
  a.tl = D.tl;
  const int t = D.stat_tile;
  a.tiles_n = D.stat_tiles;
  with_logits_tile(D.bf16, kernel_of(t, D.bf16), D.d, [&](auto cfg) {
    using C = decltype(cfg);
    hipLaunchKernelGGL((k_vocab_stat<C>), dim3(pick_count(t, D.T, D.V, D.bf16)), dim3(C::NT), 0, st, a);
  });
  auto join = [&](auto kernel, int tokens) {
    hipLaunchKernelGGL(kernel, dim3(tiles(D.T, tokens)), dim3(1024), 0, st, D.stat, a.tiles_n, D.tl, D.rows.pos, T,
                       D.loss, D.lse);
  };
  if (T <= 2048 && a.tiles_n >= 128) join(k_vocab_join<8>, 8);
  else join(k_vocab_join<64>, 64);
}

void vocab_backward(const VocabDesc& D, hipStream_t st) {
  gather_rows(D, true, st);
  const int T = static_cast<int>(D.T), es = D.bf16 ? 2 : 4;
  for (int64_t v0 = 0; v0 < D.V; v0 += D.piece) {
    const int64_t vn = D.V - v0 < D.piece ? D.V - v0 : D.piece;
    const char* w = static_cast<const char*>(D.w) + v0 * D.ldw * es;
    TileArgs a = tile_args(D);
    a.v0 = static_cast<int>(v0);
    a.vn = static_cast<int>(vn);
    a.first = v0 == 0;
    a.last = v0 + vn >= D.V;
    a.p = D.p;
    a.ldp = D.piece;
    a.acc32 = D.acc;
    a.splits = D.dh_plan.splits;
    a.A = {D.hc, D.ldhc, D.T, D.d};
    a.B = {w, D.ldw, vn, D.d};
    const int t = pick(D.T, vn, D.bf16);
    with_logits_tile(D.bf16, kernel_of(t, D.bf16), D.d, [&](auto cfg) {
      using C = decltype(cfg);
      a.tiles_n = tiles(vn, C::BN);
      hipLaunchKernelGGL((k_vocab_dlogits<C>), dim3(pick_count(t, D.T, vn, D.bf16)), dim3(C::NT), 0, st, a);
    });
    // the columns of p up to the end of the last K step are zero, and so are
    // rows past an operand's end
    a.A = {D.p, D.piece, D.T, D.piece};
    a.out = D.dh;
    TileArgs b = a;
    b.B = {D.hc, D.ldhc, D.T, D.d};
    b.out = D.dw;
    b.acc32 = D.acc_w;
    b.splits = D.dw_plan.splits;
    const int th = D.dh_plan.tile, tw = D.dw_plan.tile;
    const int nh = pick_count(th, D.T, D.d, D.bf16) * a.splits, nw = pick_count(tw, vn, D.d, D.bf16) * b.splits;
    a.tile = th;
    b.tile = tw;
    const int kh = kernel_of(th, D.bf16), kw = kernel_of(tw, D.bf16);
    with_tile<true, false, false>(D.bf16, kh, [&](auto cfg) {
      using CH = decltype(cfg);
      a.tiles_n = tiles(D.d, CH::BN);
      if (kh == kw) {
        b.tiles_n = a.tiles_n;
        typedef typename Turned<CH>::type CW;
        hipLaunchKernelGGL((k_vocab_grads<CH, CW>), dim3(nh + nw), dim3(CH::NT), 0, st, a, b, nh);
      } else {
        hipLaunchKernelGGL((k_vocab_grads<CH, NoTiles>), dim3(nh), dim3(CH::NT), 0, st, a, b, nh);
      }
    });
    if (kh != kw)
      with_tile<false, false, false>(D.bf16, kw, [&](auto cfg) {
        using CW = decltype(cfg);
        b.tiles_n = tiles(D.d, CW::BN);
        hipLaunchKernelGGL((k_vocab_grads<NoTiles, CW>), dim3(nw), dim3(CW::NT), 0, st, a, b, 0);
      });
    auto join = [&](auto kernel, const TileArgs& args, int64_t rows) {
      const int64_t n = (rows * (D.d / 8) + 255) / 256, most = 1 << 20;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(std::min(n, most)), tiles(n, 1 << 20)), dim3(256), 0, st,
                         args, static_cast<int>(rows));
    };
    if (a.last && a.splits > 1) {
      if (D.bf16) join(k_vocab_join_splits<bf16_t, true>, a, D.T);
      else join(k_vocab_join_splits<float, true>, a, D.T);
    }
    if (b.splits > 1) {
      if (D.bf16) join(k_vocab_join_splits<bf16_t, false>, b, vn);
      else join(k_vocab_join_splits<float, false>, b, vn);
    }
  }
}

}  // namespace poetx
