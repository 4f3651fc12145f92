// Log probabilities of given tokens under softmax(h w^T / temperature), the
// entropy of each row's distribution and its most likely tokens, and the
// gradient of the first two, without the [T][V] logits:
//
//   forward   per tile of h w^T: each row's maximum m, the sum of exponentials
//             e^x, x = (l - m) / temperature, and the sum u of e^x x; joined over the
//             tiles, logprob = (l[target] - m) / temperature - log s and entropy = log s
//             - u / s, whose terms are all of one sign. Of the sum s the maximum's own
//             e^0 is left out, s = 1 + q, and log s taken as log1p(q): for rows that
//             are sure of a token q, logprob and entropy go towards 0 together, and
//             1 + q in float32 would leave 6e-8 of them
//   top       the logits of some tokens at a time are kept, in 16 bits below the
//             float maximum of their group of columns: the k largest lie in the k
//             groups of the largest maxima, and what reaches the k-th maximum, a few
//             more than k, is formed again, in double
//   backward  vocab_loss.hip's, with the tiles' gradient
//             dl = a ([v = target] - p) - b p (log p + H)
//             with log p = (l - m) / temperature - log s, and 1 - p of the target as
//             -expm1(log p), for the same rows
#include "vocab_tiles.hpp"

#include <algorithm>
#include <type_traits>

namespace poetx {
namespace {

constexpr float kFloatMax = 3.4028234663852886e38f;

// A row's sums over a tile, and the maxima of the tile's groups of columns.
struct __attribute__((aligned(16))) TileRec {
  float m, q, u, pad;
  float most[4];
};

static_assert(sizeof(TileRec) == kTokenRec, "records of the workspace");

struct TokenArgs {
  TileArgs t;
  float inv_temp, c;  // factor of the logits, and of their powers of two
  const int32_t* count;  // counted rows, or null: T, in their places
  const int64_t* target; // in their places: targets, or null
  int row0;              // first compact row of the launch
  int rows;              // and rows it may have
  float* statu;
  TileRec* rec;     // with alternatives: [rows][tiles]
  uint16_t* codes;  // [rows][ldl] logits of the rows
  int64_t ldl;
  int group;        // columns of a group: a wave's
  int groups;       // groups of a tile
  // selection, join
  const void* h;
  int64_t ldh;
  const void* w;
  int64_t ldw;
  int V, top;
  float* logprob;
  float* entropy;
  float2* stat;
  int64_t* top_ids;
  float* top_logprobs;
};

// rows of this launch that hold tokens
__device__ __forceinline__ int token_rows(const TokenArgs& a) {
  return min(a.rows, (a.count ? *a.count : a.t.T) - a.row0);
}

// Rows in their places: whether token t is counted, and its target, or a column that
// no tile has.
__device__ __forceinline__ bool given_counts(const TokenArgs& a, int t) {
  return !a.target || (a.target[t] >= 0 && a.target[t] < a.t.vn);
}
__device__ __forceinline__ int given_column(const TokenArgs& a, int t) {
  return given_counts(a, t) ? static_cast<int>(a.target[t]) : -(1 << 30);
}

// Joins sums over disjoint sets of columns, x in powers of two below the set's
// largest logit m: 1 + q of e^x and u of e^x x. An empty set is (-inf, -1, 0).
__device__ __forceinline__ void join_token(float& m, float& q, float& u, float m2, float q2, float u2, float c) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;
  const float d1 = (m - ref) * c, d2 = (m2 - ref) * c;
  const float f1 = __builtin_amdgcn_exp2f(d1), f2 = __builtin_amdgcn_exp2f(d2);
  // 2^-200 is 0: where the distance is that large, or infinite, nothing is left
  u = f1 * (u + fmaxf(d1, -200.f) * (1.f + q)) + f2 * (u2 + fmaxf(d2, -200.f) * (1.f + q2));
  // (a NaN logit leaves its mark in the sums; fmaxf drops it)
  q = m >= m2 ? q + f2 * (1.f + q2) : q2 + f1 * (1.f + q);
  m = top;
}

// Two logits' distances below their group's maximum in 16 bits: the upper halves
// of the (negative) floats next nearer to 0. A difference of two floats may be rounded
// away from 0 (1e-6 - 100 is -100), by half a step at most: taken one step back, the
// code is no further below the maximum than the logit is, and nearer by less than 2^-7 +
// 2^-23 of it. Zeros, infinities and NaN stay.
__device__ __forceinline__ uint32_t code_pair(float lo, float hi) {
  constexpr float kBack = 0x1.fffffep-1f;  // 1 - 2^-24: rounds to the next float towards 0
  return (__float_as_uint(lo * kBack) >> 16) | (__float_as_uint(hi * kBack) & 0xffff0000u);
}
// 32 columns lie as four lanes hold them, eight codes each: the column of code p,
// and the code of a column.
__device__ __forceinline__ int code_column(int p) { return (p & ~31) + (p >> 2 & 1) * 16 + (p >> 3 & 3) * 4 + (p & 3); }
__device__ __forceinline__ int column_code(int col) { return (col & ~31) + (col >> 2 & 3) * 8 + (col >> 4 & 1) * 4 + (col & 3); }

// A tile's statistics; with KEEP its logits and their groups' maxima, too.
template <class Cfg, bool KEEP>
__device__ __forceinline__ void token_stat_tile(const TokenArgs& a, int m0, int tn, int count, char* smem) {
  const int n0 = tn * Cfg::BN;
  TileOperand A = a.t.A;
  A.rows = count;
  f32x4_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.t.B, m0, n0, 0, (a.t.d + Cfg::BK - 1) / Cfg::BK, smem, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
  float2* red = reinterpret_cast<float2*>(smem);  // [WN][BM] maximum and sums
  float* redu = reinterpret_cast<float*>(red + Cfg::WN * Cfg::BM);
  // the first K group's waves hold the sums
  if (wave < Cfg::NW) {
    mask_columns<Cfg>(acc, wn, lane, a.t.vn - n0, -INFINITY);
#pragma unroll
    for (int i = 0; i < Cfg::TM; ++i) {
      const int row = tile_row<Cfg>(wm, lane, i);
      if (a.logprob) {
        const int at = a.row0 + m0 + row;
        const int tcol = m0 + row >= count ? -1 : a.target ? given_column(a, at) - n0 : a.t.r.tgt[at] - n0;
        if (__any(static_cast<unsigned>(tcol - wn * Cfg::WTN) < Cfg::WTN)) {
#pragma unroll
          for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (tile_col<Cfg>(wn, lane, j, r) == tcol) a.t.tl[at] = acc[i][j][r];
        }
      }
      float m = acc[i][0][0], s = 0.f, q = 0.f, u = 0.f;
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float ref = m == -INFINITY ? 0.f : fminf(m, kFloatMax);
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[i][j][r] -= ref;
          const float x = acc[i][j][r] * a.c, e = __builtin_amdgcn_exp2f(x);
          s += e;
          q += __builtin_amdgcn_fractf(e);   // without the maximum's 1
          u = fmaf(e, fmaxf(x, -200.f), u);  // 2^-200 is 0: no 0 * infinity
        }
      if constexpr (KEEP) {
        if (m0 + row < count) {
          uint16_t* const to = a.codes + (m0 + row) * a.ldl + n0 + wn * Cfg::WTN + (lane >> 4) * 8;
#pragma unroll
          for (int j = 0; j < Cfg::TN; j += 2) {
            const tg_u32x4_t v = {code_pair(acc[i][j][0], acc[i][j][1]), code_pair(acc[i][j][2], acc[i][j][3]),
                                  code_pair(acc[i][j + 1][0], acc[i][j + 1][1]), code_pair(acc[i][j + 1][2], acc[i][j + 1][3])};
            *reinterpret_cast<tg_u32x4_t*>(to + j * 16) = v;
          }
        }
      }
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      q += __shfl_xor(q, 16);
      q += __shfl_xor(q, 32);
      u += __shfl_xor(u, 16);
      u += __shfl_xor(u, 32);
      q += rintf(s - q) - 1.f;  // all but one of those that are the maximum
      if (lane < 16) {
        red[wn * Cfg::BM + row] = make_float2(m, q);
        redu[wn * Cfg::BM + row] = u;
      }
    }
  }
  __syncthreads();
  const int row = threadIdx.x;
  if (row < Cfg::BM && m0 + row < count) {
    float2 v = red[row];
    float u = redu[row];
    TileRec rec;
    if constexpr (KEEP) {
#pragma unroll
      for (int w = 0; w < 4; ++w) rec.most[w] = w < Cfg::WN ? red[w * Cfg::BM + row].x : -INFINITY;
    }
#pragma unroll
    for (int w = 1; w < Cfg::WN; ++w) {
      const float2 v2 = red[w * Cfg::BM + row];
      join_token(v.x, v.y, u, v2.x, v2.y, redu[w * Cfg::BM + row], a.c);
    }
    if constexpr (KEEP) {
      rec.m = v.x;
      rec.q = v.y;
      rec.u = u;
      a.rec[static_cast<int64_t>(m0 + row) * a.t.tiles_n + tn] = rec;
    } else {
      const int64_t at = static_cast<int64_t>(tn) * a.t.T + m0 + row;
      a.t.stat[at] = v;
      a.statu[at] = u;
    }
  }
}

// Workgroups of a launch for `rows` rows of which any number may count.
int token_tiles(int tile, int64_t rows, int64_t vn, bool bf16) {
  if (kernel_of(tile, bf16) != kTile128x256 || !bf16) return pick_count(tile, rows, vn, bf16);
  return tiles(vn, 256) * (static_cast<int>(rows / 256) + kMixedRows);
}

template <class C, bool KEEP>
__global__ void __launch_bounds__(C::NT, 1) k_token_stat(const TokenArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int count = token_rows(a);
  if (count <= 0) return;
  int m0, tn;
  if constexpr (IsWide<C>::value) {
    switch (mixed_tile(blockIdx.x, count, a.t.tiles_n, gridDim.x, 0.f, m0, tn)) {
      case 64: token_stat_tile<typename C::T64, KEEP>(a, m0, tn, count, smem); return;
      case 128: token_stat_tile<typename C::T128, KEEP>(a, m0, tn, count, smem); return;
      case 192: token_stat_tile<typename C::T192, KEEP>(a, m0, tn, count, smem); return;
      case 256: token_stat_tile<typename C::T256, KEEP>(a, m0, tn, count, smem); return;
    }
  } else if (vocab_place<C::BM>(blockIdx.x, count, a.t.tiles_n, m0, tn)) {
    token_stat_tile<C, KEEP>(a, m0 * C::BM, tn, count, smem);
  }
}

// --- the most likely tokens ------------------------------------------------------

// Keys in the order of the logits; NaN as -inf, and so every logit's above 0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t u = __float_as_uint(l == l ? l + 0.f : -INFINITY);  // + 0: -0 as 0
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

struct SelectLds {
  int hist[256];
  int sums[2][16];
  uint32_t prefix;
  int need;
};

// The K-th largest of n >= K keys, eight bits of it a pass.
template <int NT, class Key>
__device__ __forceinline__ uint32_t kth_largest(int n, int K, SelectLds& s, Key&& key) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t prefix = 0, mask = 0;
  int need = K;  // of the keys that share the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += NT) s.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += NT) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&s.hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (wave == 0) {
      // lane l: bins 255 - 4 l .. 252 - 4 l, from the largest down
      int c[4], sum = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) sum += c[b] = s.hist[255 - 4 * lane - b];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (before < need && before + c[b] >= need) {
          s.prefix = prefix | static_cast<uint32_t>(255 - 4 * lane - b) << shift;
          s.need = need - before;
        }
        before += c[b];
      }
    }
    __syncthreads();
    prefix = s.prefix;
    need = s.need;
    mask |= 255u << shift;
  }
  return prefix;
}

// Of the columns 0 .. n - 1 those of kind 2, and the first `most` of kind 1, numbered in
// their order: put(number, column). Returns how many there are.
template <int NT, class Kind, class Put>
__device__ __forceinline__ int number_columns(int n, int most, SelectLds& s, Kind&& kind, Put&& put) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned long long below = (1ull << lane) - 1;
  int alike = 0, all = 0;  // before this round of NT columns
  for (int i0 = 0; i0 < n; i0 += NT) {
    const int k = i0 + tid < n ? kind(i0 + tid) : 0;
    const unsigned long long one = __ballot(k == 1);
    if (lane == 0) s.sums[0][wave] = __popcll(one);
    __syncthreads();
    int rank = alike + __popcll(one & below);
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      rank += w < wave ? s.sums[0][w] : 0;
      alike += s.sums[0][w];
    }
    const bool take = k == 2 || (k == 1 && rank < most);
    const unsigned long long in = __ballot(take);
    if (lane == 0) s.sums[1][wave] = __popcll(in);
    __syncthreads();
    int to = all + __popcll(in & below);
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      to += w < wave ? s.sums[1][w] : 0;
      all += s.sums[1][w];
    }
    if (take) put(to, i0 + tid);
  }
  __syncthreads();
  return all;
}

// products exact (bfloat16's in float), their sum in double
__device__ __forceinline__ double dot16(uint4 a, uint4 b, double s, bf16_t) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s += static_cast<double>(__uint_as_float(x[i] << 16) * __uint_as_float(y[i] << 16));
    s += static_cast<double>(__uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u));
  }
  return s;
}
__device__ __forceinline__ double dot16(uint4 a, uint4 b, double s, float) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s = fma(static_cast<double>(__uint_as_float(x[i])), static_cast<double>(__uint_as_float(y[i])), s);
  return s;
}

// log of the sum and entropy of a row from its joined sums
struct RowOut {
  float log_s, entropy;
};
__device__ __forceinline__ RowOut row_out(float q, float u) {
  const float log_s = log1pf(q);
  return {log_s, log_s - u / (1.f + q) * kLn2};
}

// A code's logit, or a little more: its group's maximum and the distance below it
// (that of a NaN is not negative; beside an infinite maximum it is infinite itself).
// `share`: 1, or kShare for a key that the logit is not below. The sum is of floats
// that the logit, a float itself, lies between, and so does its rounding.
constexpr float kShare = 1.f + 0x1p-7f + 0x1p-15f;  // times 8 bits exact
__device__ __forceinline__ uint32_t code_key(float most, uint32_t code, float share = 1.f) {
  const float d = __uint_as_float(code << 16) * share;
  const float base = most == -INFINITY ? 0.f : fminf(most, kFloatMax);
  return logit_key(d <= 0.f || d == INFINITY ? base + d : -INFINITY);
}

// A row's outputs and its `top` most likely tokens, one workgroup a row.
//
// The K = top + kTopSpare largest float logits lie in the K groups of the largest
// maxima. The maxima fall into 128 slots; the K-th largest slot, found bit by bit by
// counting, is a lower bound of the K-th largest logit, and what reaches it, a few
// more than K, are the candidates: their logits are formed again in double, which
// float's rounding does not order, and ranked.
//
// Where more than kCandidates reach it, the bound is the K-th largest of the codes' own
// lower bounds, found digit by digit. It is no less than the K-th largest maximum: what
// reaches it lies in the fewer than K groups with a larger one, under 64 K codes (of a
// group with a logit far above the others all may reach it), which are taken kCandidates
// at a time, with the best of those before. Or its float logit is the bound itself: of
// these the kCandidates of the lowest index are taken.
constexpr int kSlots = 128, kGroupList = 256, kCandidates = 512;

// v op'd over the wave, in every lane; op commutes. Within rows of 16 lanes by moves
// of the vector unit, which take a tenth of a shuffle's time.
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  const int x = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
  const long long x = __double_as_longlong(v);
  const int lo = static_cast<int>(x), hi = static_cast<int>(x >> 32);
  const unsigned lo2 = __builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xf, 0xf, true);
  const long long hi2 = __builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xf, 0xf, true);
  return __longlong_as_double(hi2 << 32 | lo2);
}
template <class V, class Op>
__device__ __forceinline__ V over_wave(V v, Op&& op) {
  v = op(v, dpp_move<0xb1>(v));   // lane ^ 1
  v = op(v, dpp_move<0x4e>(v));   // lane ^ 2
  v = op(v, dpp_move<0x141>(v));  // the other four of eight
  v = op(v, dpp_move<0x140>(v));  // the other eight of sixteen
  v = op(v, __shfl_xor(v, 16));
  return op(v, __shfl_xor(v, 32));
}
template <class V>
__device__ __forceinline__ V sum_wave(V v) {
  return over_wave(v, [](V a, V b) { return a + b; });
}

// join_token over the wave: the maximum first, so that each lane takes its own step
// to it once; one lane that has it adds q and the others 1 + q.
__device__ __forceinline__ void join_wave(float& m, float& q, float& u, float c) {
  const float top = over_wave(m, [](float a, float b) { return fmaxf(a, b); });
  const float d = (m - (top == -INFINITY ? 0.f : top)) * c, f = __builtin_amdgcn_exp2f(d);
  const unsigned long long has = __ballot(m == top);
  const bool first = (threadIdx.x & 63) == __ffsll(has) - 1;
  u = sum_wave(f * (u + fmaxf(d, -200.f) * (1.f + q)));
  q = sum_wave(first ? q : f * (1.f + q));
  m = top;
}

template <int NT, class T>
__global__ void __launch_bounds__(NT, NT == 1024 ? 4 : 6) k_token_select(const TokenArgs a) {
  constexpr int NW = NT / 64, KEPT = 2, HROW = 1024;
  static_assert(NT >= kSlots && NT >= kTopMost, "a thread a slot, and an alternative");
  __shared__ SelectLds s;
  __shared__ uint4 hrow[HROW];
  __shared__ int groups[kGroupList];
  __shared__ __attribute__((aligned(16))) uint32_t keys[kSlots];
  __shared__ int ids[kCandidates];
  __shared__ double exact[kCandidates];
  __shared__ float4 red[NW];
  __shared__ int counts[2];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = a.row0 + r;  // a compact row, and a token, which is cleared if it is not counted
  const int tiles = a.t.tiles_n;
  const TileRec* const rec = a.rec + static_cast<int64_t>(r) * tiles;
  const uint16_t* const codes = a.codes + r * a.ldl;
  const uint4* const h = reinterpret_cast<const uint4*>(static_cast<const T*>(a.h) + c * a.ldh);
  const int chunks = a.t.d / (16 / static_cast<int>(sizeof(T)));

  // all of a row's loads at once, whether it holds a token or not
  TileRec x[KEPT];
#pragma unroll
  for (int q = 0; q < KEPT; ++q) {
    x[q].m = -INFINITY;
    x[q].q = -1.f;
    x[q].u = 0.f;
    if (tid + q * NT < tiles) x[q] = rec[tid + q * NT];
  }
  const bool uncounted = a.t.r.pos ? a.t.r.pos[c] < 0 : !given_counts(a, c);
  const int t = a.t.r.idx ? a.t.r.idx[c] : c, count = token_rows(a);
  const float given = a.logprob ? a.t.tl[c] : 0.f;
  for (int i = tid; i < min(chunks, HROW); i += NT) hrow[i] = h[i];
  if (tid < kSlots) keys[tid] = 0;
  if (tid == 0) counts[0] = counts[1] = 0;
  if (uncounted) {
    if (tid < a.top) {
      a.top_ids[static_cast<int64_t>(c) * a.top + tid] = -1;
      a.top_logprobs[static_cast<int64_t>(c) * a.top + tid] = 0.f;
    }
    if (tid == 0) {
      a.logprob[c] = a.entropy[c] = 0.f;
      a.stat[c] = make_float2(0.f, 0.f);
    }
  }
  if (r >= count || (uncounted && !a.t.r.pos)) return;
  const int K = min(a.top + kTopSpare, a.V), G = (a.V + a.group - 1) / a.group;

  // f(group, key of its maximum) for the groups of tile k
  auto groups_of = [&](int k, const TileRec& v, auto&& f) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (g < a.groups && k * a.groups + g < G) f(k * a.groups + g, logit_key(v.most[g]));
  };
  auto all_groups = [&](auto&& f) {
#pragma unroll
    for (int q = 0; q < KEPT; ++q)
      if (tid + q * NT < tiles) groups_of(tid + q * NT, x[q], f);
    for (int k = tid + KEPT * NT; k < tiles; k += NT) groups_of(k, rec[k], f);
  };
  auto most_of = [&](int g) { return rec[g / a.groups].most[g % a.groups]; };
  // f(column, its group's maximum, code) for the eight codes of a group from p on
  auto codes_of = [&](int g, int p, auto&& f) {
    const float top = most_of(g);
    const uint4 v = *reinterpret_cast<const uint4*>(codes + g * a.group + p);
    const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int col = g * a.group + code_column(p + q);
      if (col < a.V) f(col, top, y[q >> 1] >> (q & 1) * 16 & 0xffffu);
    }
  };
  const int shift = a.group == 64 ? 3 : 2;  // eights of a group
  // Few groups: their maxima alone would bound little or nothing, the slots take
  // the codes of all (T = 6947, V = 284, 20 alternatives, 512 threads a row: 538 us by
  // groups, 118 so).
  const bool fine = G < 4 * K;
  __syncthreads();
  if (fine) {
    for (int i = tid; i < G << shift; i += NT)
      codes_of(i >> shift, (i & ((1 << shift) - 1)) * 8, [&](int col, float top, uint32_t code) {
        atomicMax(&keys[col & (kSlots - 1)], code_key(top, code, kShare));
      });
  } else {
    all_groups([&](int g, uint32_t key) { atomicMax(&keys[g & (kSlots - 1)], key); });
  }
  float m = x[0].m, sum = x[0].q, u = x[0].u;
#pragma unroll
  for (int q = 1; q < KEPT; ++q) join_token(m, sum, u, x[q].m, x[q].q, x[q].u, a.c);
  for (int k = tid + KEPT * NT; k < tiles; k += NT) join_token(m, sum, u, rec[k].m, rec[k].q, rec[k].u, a.c);
  join_wave(m, sum, u, a.c);
  if (lane == 0) red[wave] = make_float4(m, sum, u, 0.f);
  __syncthreads();

  // the K-th largest slot to 18 bits, downwards: every wave counts the slots for itself
  uint32_t tau = 0;
  {
    static_assert(kSlots == 128 && kTopMost + kTopSpare <= kSlots, "two slots a lane");
    const uint2 v = *reinterpret_cast<const uint2*>(keys + lane * 2);
#pragma unroll
    for (int b = 31; b >= 14; --b) {
      const uint32_t next = tau | 1u << b;
      const int n = __popcll(__ballot(v.x >= next)) + __popcll(__ballot(v.y >= next));
      tau = n >= K ? next : tau;
    }
  }
  if (!fine)
    all_groups([&](int g, uint32_t key) {
      if (key < tau) return;
      const int at = atomicAdd(&counts[0], 1);
      if (at < kGroupList) groups[at] = g;
    });
  __syncthreads();
  const int ng = fine ? G : counts[0];
  if (fine || ng <= kGroupList)
    for (int i = tid; i < ng << shift; i += NT)
      codes_of(fine ? i >> shift : groups[i >> shift], (i & ((1 << shift) - 1)) * 8, [&](int col, float top, uint32_t code) {
        if (code_key(top, code) < tau) return;
        const int at = atomicAdd(&counts[1], 1);
        if (at < kCandidates) ids[at] = col;
      });
  __syncthreads();
  int n = counts[1], kept = 0;
  const bool many = (!fine && ng > kGroupList) || n > kCandidates;
  auto key_of = [&](int i, float share) {
    const int g = i / a.group;
    return code_key(most_of(g), codes[g * a.group + column_code(i % a.group)], share);
  };
  if (many) tau = kth_largest<NT>(a.V, K, s, [&](int i) { return key_of(i, kShare); });
  // candidate i's rank among n, and the largest logit of them
  auto rank_of = [&](int i, int n, double& most) {
    const double v = exact[i], order = v == v ? v : -INFINITY;
    const int id = ids[i];
    int rank = 0;
    most = -INFINITY;
    for (int k = 0; k < n; ++k) {
      const double w = exact[k] == exact[k] ? exact[k] : -INFINITY;
      rank += w > order || (w == order && ids[k] < id);
      most = w > most ? w : most;
    }
    return rank;
  };
  const uint4* const from = chunks <= HROW ? hrow : h;
  for (int done = 0;;) {
    int all = 0;
    if (many) {
      const int room = kCandidates - kept;
      all = number_columns<NT>(
          a.V, kCandidates, s,
          [&](int i) {
            const uint32_t most = key_of(i, 1.f);
            return most < tau ? 0 : most == tau && key_of(i, kShare) == tau ? 1 : 2;
          },
          [&](int at, int i) {
            if (at >= done && at < done + room) ids[kept + at - done] = i;
          });
      n = kept + min(all - done, room);
      done += room;
    }
    // two candidates a wave at a time, up to 8 or 4 KB of each in flight: few rows are bound by
    // latency, many by bandwidth (T = 8192, V = 131072: 5.4 TB/s of w's rows)
    for (int k = kept + wave; k < n; k += 2 * NW) {
      const int k2 = k + NW < n ? k + NW : k;
      const uint4* const w0 = reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + ids[k] * a.ldw);
      const uint4* const w1 = reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + ids[k2] * a.ldw);
      double v0 = 0, v1 = 0;
      int i = lane;
      auto step = [&](auto batch) {
        constexpr int B = decltype(batch)::value;
        for (; i + (B - 1) * 64 < chunks; i += B * 64) {
          uint4 y0[B], y1[B];
#pragma unroll
          for (int q = 0; q < B; ++q) {
            y0[q] = w0[i + q * 64];
            y1[q] = w1[i + q * 64];
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int q = 0; q < B; ++q) {
            const uint4 z = from[i + q * 64];
            v0 = dot16(z, y0[q], v0, T{});
            v1 = dot16(z, y1[q], v1, T{});
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      step(std::integral_constant<int, NT == 1024 ? 8 : 4>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 1>{});
      v0 = sum_wave(v0);
      v1 = sum_wave(v1);
      if (lane == 0) {
        exact[k] = v0;
        exact[k2] = v1;
      }
    }
    if (!many || done >= all) break;
    // the best of this batch and of those before, to the front
    constexpr int OWN = (kCandidates + NT - 1) / NT;
    __syncthreads();
    double v[OWN];
    int id[OWN], rank[OWN];
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      const int i = min(tid + q * NT, n - 1);
      v[q] = exact[i];
      id[q] = ids[i];
      double most;
      rank[q] = tid + q * NT < n ? rank_of(i, n, most) : a.top;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < OWN; ++q) {
      if (rank[q] >= a.top) continue;
      exact[rank[q]] = v[q];
      ids[rank[q]] = id[q];
    }
    kept = min(n, a.top);
  }
  const float4 part = lane < NW ? red[lane] : make_float4(-INFINITY, -1.f, 0.f, 0.f);
  m = part.x, sum = part.y, u = part.z;
  join_wave(m, sum, u, a.c);
  const RowOut o = row_out(sum, u);
  if (tid == 0) {
    a.stat[t] = make_float2(m, o.log_s);
    a.entropy[t] = o.entropy;
    if (a.logprob) a.logprob[t] = (given - m) * a.inv_temp - o.log_s;
  }
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    double most;
    const int rank = rank_of(i, n, most);
    if (rank >= a.top) continue;
    const int64_t at = static_cast<int64_t>(t) * a.top + rank;
    // The maximum that log s is taken from is a float sum, off by its rounding; the log of
    // all exponentials is off by the maximum's share of that.
    const double m64 = m, lp = ((exact[i] - m64) + (m64 - most) / (1.0 + sum)) * a.inv_temp - o.log_s;
    a.top_ids[at] = ids[i];
    a.top_logprobs[at] = lp > 0 ? 0.f : static_cast<float>(lp);  // NaN stays
  }
}

// logprob, entropy, and maximum and log s of every token from the tiles' sums. N tokens a
// workgroup, 1024 / N threads a token over the tiles.
template <int N>
__global__ void __launch_bounds__(1024) k_token_join(const TokenArgs a) {
  __shared__ float2 red[16][N];
  __shared__ float redu[16][N];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, T = a.t.T;
  const int t = blockIdx.x * N + lane % N;
  const int c = t >= T ? -1 : a.t.r.pos ? a.t.r.pos[t] : given_counts(a, t) ? t : -1;
  float m = -INFINITY, s = -1.f, u = 0.f;
  if (c >= 0)
#pragma unroll 4
    for (int k = threadIdx.x / N; k < a.t.tiles_n; k += 1024 / N) {
      const int64_t at = static_cast<int64_t>(k) * T + c;
      const float2 v = a.t.stat[at];
      join_token(m, s, u, v.x, v.y, a.statu[at], a.c);
    }
#pragma unroll
  for (int o = N; o < 64; o <<= 1) {
    const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o), u2 = __shfl_xor(u, o);
    join_token(m, s, u, m2, s2, u2, a.c);
  }
  if (lane < N) {
    red[wave][lane] = make_float2(m, s);
    redu[wave][lane] = u;
  }
  __syncthreads();
  if (threadIdx.x >= N || t >= T) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) join_token(m, s, u, red[w][lane].x, red[w][lane].y, redu[w][lane], a.c);
  const RowOut o = row_out(s, u);
  a.stat[t] = c >= 0 ? make_float2(m, o.log_s) : make_float2(0.f, 0.f);
  a.entropy[t] = c >= 0 ? o.entropy : 0.f;
  if (a.logprob) a.logprob[t] = c >= 0 ? (a.t.tl[c] - m) * a.inv_temp - o.log_s : 0.f;
}

// --- gradient ----------------------------------------------------------------------

// Gradient of the logits of a piece in the storage type, in units of the largest
// gradient and without the factor 1 / temperature, both of which the products'
// epilogues put back in float32: dl = p (g - b (log p + H)) - g [v = target] with g =
// -a, and the target's p - 1 as expm1(log p).
//
// A tile of another kind than the forward's sums in another order, and the largest logit
// is off the forward's maximum by the rounding of both, 1.5e-5 at 300: more than all of 1
// - p in a row that is sure of its token. There the distance is known without it: where
// the other exponentials are under e^0.22 - 1 = 0.25 together, the other logits are at
// least 1.4 below the maximum, and what is within 0.7 of it is the maximum itself, at a
// distance of 0. In other rows no logit passes the maximum.
template <class Cfg>
__device__ __forceinline__ void token_dlogits_tile(const TokenArgs& a, int m0, int tn, int count, char* smem) {
  const int n0 = tn * Cfg::BN;
  TileOperand A = a.t.A;
  A.rows = count;
  f32x4_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(A, a.t.B, m0, n0, 0, (a.t.d + Cfg::BK - 1) / Cfg::BK, smem, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
    const int row = m0 + tile_row<Cfg>(wm, lane, i);
    const int at = row < count ? row : m0;  // rows past the count are not stored
    const int tcol = a.t.r.tgt[at] - a.t.v0 - n0;
    const float2 st = a.t.r.stat[at];
    const float g = a.t.r.g[at];
    const float b = a.t.r.gent ? a.t.r.gent[at] : 0.f, H = a.t.r.gent ? a.t.r.ent[at] : 0.f;
    const bool given = __any(static_cast<unsigned>(tcol - wn * Cfg::WTN) < Cfg::WTN);
    float target = 0.f;
    if (given) {
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tile_col<Cfg>(wn, lane, j, r) == tcol) target = acc[i][j][r];
    }
    const float near = st.y < 0.22f ? -0.7f / a.inv_temp : 0.f;
    auto log_p = [&](float l) {
      const float below = l - st.x;
      return fmaf(below > near ? 0.f : below, a.inv_temp, -st.y);  // NaN stays
    };
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float lp = log_p(acc[i][j][r]), p = __builtin_amdgcn_exp2f(lp * kLog2e);
        acc[i][j][r] = p * (g - b * (fmaxf(lp, -200.f) + H));  // e^-200 is 0: no 0 * infinity
      }
    if (given) {
      const float lp = log_p(target), p = __builtin_amdgcn_exp2f(lp * kLog2e);
      const float dl = g * expm1f(lp) - b * p * (fmaxf(lp, -200.f) + H);
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tile_col<Cfg>(wn, lane, j, r) == tcol) {
            acc[i][j][r] = dl;
            // what its rounding takes off, for the products' epilogues
            // (the first K group's waves hold the sums)
            if (Cfg::ES == 2 && row < count && wave < Cfg::NW) {
              const float off = dl - bf16_to_f32(f32_to_bf16(dl));
              a.t.r.resid[row] = fabsf(off) < INFINITY ? off : 0.f;
            }
          }
    }
  }
  mask_columns<Cfg>(acc, wn, lane, a.t.vn - n0, 0.f);
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    auto* p = static_cast<typename Elem<Cfg::ES>::type*>(a.t.p);
    if (m0 + row < count) tile_store8(p + static_cast<int64_t>(m0 + row) * a.t.ldp + n0 + col, v);
  });
}

template <class C>
__global__ void __launch_bounds__(C::NT, 1) k_token_dlogits(const TokenArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int count = *a.t.r.count;
  int m0, tn;
  if constexpr (IsWide<C>::value) {
    switch (mixed_tile(blockIdx.x, count, a.t.tiles_n, gridDim.x, 0.f, m0, tn)) {
      case 64: token_dlogits_tile<typename C::T64>(a, m0, tn, count, smem); return;
      case 128: token_dlogits_tile<typename C::T128>(a, m0, tn, count, smem); return;
      case 192: token_dlogits_tile<typename C::T192>(a, m0, tn, count, smem); return;
      case 256: token_dlogits_tile<typename C::T256>(a, m0, tn, count, smem); return;
    }
  } else if (vocab_place<C::BM>(blockIdx.x, count, a.t.tiles_n, m0, tn)) {
    token_dlogits_tile<C>(a, m0 * C::BM, tn, count, smem);
  }
}

}  // namespace

void token_forward(const VocabDesc& D, hipStream_t st) {
  const int es = D.bf16 ? 2 : 4;
  TokenArgs a{};
  a.t = tile_args(D);
  const char* h = static_cast<const char*>(D.h);
  int64_t ldh = D.ldh;
  const int t = D.stat_tile, kernel = kernel_of(t, D.bf16);
  const int64_t chunk = D.chunk ? D.chunk : D.T;
  // Where all rows' tiles are one round, fewer rows cost as much: they stay in their
  // places, and the launch that gathers the counted ones, 5 us, is saved.
  const bool one_round = chunk >= D.T && pick_count(t, D.T, D.V, D.bf16) <= 256;
  // Rows too far apart for a tile's offsets are gathered, counted or not.
  if ((D.target && !one_round) || D.ldh > kVocabStride) {
    vocab_gather(D, false, st);
    h = static_cast<const char*>(D.hc);
    ldh = D.ldhc;
    a.count = D.rows.count;
  } else {
    a.t.r = {};
    a.target = D.target;
  }
  a.t.B = {D.w, D.ldw, D.V, D.d};
  a.t.vn = static_cast<int>(D.V);
  a.t.stat = D.stat;
  a.t.tl = D.tl;
  a.t.tiles_n = D.stat_tiles;
  a.inv_temp = D.inv_temp;
  a.c = D.inv_temp * kLog2e;
  a.statu = D.statu;
  a.rec = static_cast<TileRec*>(D.rec);
  a.codes = D.codes;
  a.ldl = D.ldl;
  a.h = h;
  a.ldh = ldh;
  a.w = D.w;
  a.ldw = D.ldw;
  a.V = static_cast<int>(D.V);
  a.top = D.top;
  a.logprob = D.logprob;
  a.entropy = D.entropy;
  a.stat = D.row_stat;
  a.top_ids = D.top_ids;
  a.top_logprobs = D.top_logprobs;
  a.group = D.bf16 && kernel == kTile128x256 ? 64 : 32;  // a wave's columns
  a.groups = (D.bf16 ? kTileCosts[t].bn : kTileCostsF32[t].bn) / a.group;
  for (int64_t r0 = 0; r0 < D.T; r0 += chunk) {
    const int64_t rows = std::min(chunk, D.T - r0);
    a.row0 = static_cast<int>(r0);
    a.rows = static_cast<int>(rows);
    a.t.A = {h + r0 * ldh * es, ldh, rows, D.d};
    with_logits_tile(D.bf16, kernel, D.d, [&](auto cfg) {
      using C = decltype(cfg);
      const dim3 grid(token_tiles(t, rows, D.V, D.bf16));
      if (D.top) hipLaunchKernelGGL((k_token_stat<C, true>), grid, dim3(C::NT), 0, st, a);
      else hipLaunchKernelGGL((k_token_stat<C, false>), grid, dim3(C::NT), 0, st, a);
    });
    if (!D.top) continue;
    auto select = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, dim3(rows), dim3(threads), 0, st, a); };
    // a row's chain of latencies is shorter over more threads, and more rows are on their
    // way with fewer (512 against 256, 5 alternatives, the whole call: 600 rows of V = 284
    // 19.2 us, 18.6; 2000 35.6, 26.0; 8000 of V = 8000, d = 1024 251, 196)
    const int threads = rows <= 256 ? 1024 : rows <= 512 ? 512 : 256;
    if (D.bf16) {
      if (threads == 1024) select(k_token_select<1024, bf16_t>, threads);
      else if (threads == 512) select(k_token_select<512, bf16_t>, threads);
      else select(k_token_select<256, bf16_t>, threads);
    } else {
      if (threads == 1024) select(k_token_select<1024, float>, threads);
      else if (threads == 512) select(k_token_select<512, float>, threads);
      else select(k_token_select<256, float>, threads);
    }
  }
  if (D.top) return;
  const int T = static_cast<int>(D.T);
  // as k_vocab_join's: by latencies
  if (T <= 2048 && D.stat_tiles >= 128)
    hipLaunchKernelGGL((k_token_join<8>), dim3(tiles(T, 8)), dim3(1024), 0, st, a);
  else
    hipLaunchKernelGGL((k_token_join<64>), dim3(tiles(T, 64)), dim3(1024), 0, st, a);
}

void token_dlogits(const VocabDesc& D, TileArgs& t, hipStream_t st) {
  const int tile = pick(D.T, t.vn, D.bf16);
  with_logits_tile(D.bf16, kernel_of(tile, D.bf16), D.d, [&](auto cfg) {
    using C = decltype(cfg);
    t.tiles_n = tiles(t.vn, C::BN);
    TokenArgs a{};
    a.t = t;
    a.inv_temp = D.inv_temp;
    hipLaunchKernelGGL((k_token_dlogits<C>), dim3(token_tiles(tile, D.T, t.vn, D.bf16)), dim3(C::NT), 0, st, a);
  });
}

}  // namespace poetx
