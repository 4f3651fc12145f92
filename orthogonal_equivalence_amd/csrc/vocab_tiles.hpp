// What the operators over a vocabulary share (vocab_loss.hip, token_logprobs.hip):
// the tiles of h w^T over the counted tokens' rows, and which tile a product takes.
#pragma once

#include "model_kernels.hpp"
#include "tile_gemm.hpp"

namespace poetx {

constexpr float kLn2 = 0.6931471805599453f;

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
  float post;      // dh, dw: factor behind the logits (1 / temperature), times the unit maybe past float32
  float beside;    // dh: us of dw's tiles in the same launch, were their K as long as kTileCosts'
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
  typedef TileCfg<2, 64, 256, 2, 4, 3, AKC, BKC, KTAIL> T64;
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

// Counted rows in tiles of 256 rows and, behind them, the last 0 to 1023 in smaller
// tiles: rounds of large tiles alone leave most CUs idle in the last one.
struct MixedTiles {
  int rows256;       // rows of tiles of 256 rows
  int bm, rows_bm;   // the others' rows, and rows of them
};
constexpr int kMixedRows = 3;  // rows of tiles that a launch has room for beyond those of 256 rows
// us of a tile of 64 .. 256 rows by 256 columns, as in kTileCosts
constexpr float kMixedCosts[4] = {24.f, 35.f, 46.5f, 57.f};

// The cheapest of the mixes whose tiles fit the launch: of two classes of tiles,
// the larger first, each CU taking the next as it gets free. Sixteen lanes try one
// each, their times with the lane's number in the low bits. `beside`: us of other
// tiles behind them, which fill the CUs that they leave.
__device__ __forceinline__ MixedTiles mix_tiles(int count, int tiles_n, int most, float beside) {
  constexpr int kCus = 256;
  const int lane = threadIdx.x & 15, kind = lane & 3;
  const int a = (count >> 8) - (lane >> 2), rest = count - (a << 8);
  // rows of 64 over rows of 64 (kind + 1): small numbers, divided by multiplication
  const int b = (((rest + 63) >> 6) + kind) * (kind == 0 ? 65536 : kind == 1 ? 32768 : kind == 2 ? 21846 : 16384) >> 16;
  const int n1 = a * tiles_n, n2 = b * tiles_n;
  float us = 3e38f;
  if (a >= 0 && n1 + n2 <= most) {
    const float c1 = kMixedCosts[3];
    const float c2 = kind == 0 ? kMixedCosts[0] : kind == 1 ? kMixedCosts[1] : kind == 2 ? kMixedCosts[2] : c1;
    const float up = static_cast<float>((n1 + kCus - 1) / kCus) * c1;
    const float all = (static_cast<float>(n1) * c1 + static_cast<float>(n2) * c2 + beside) / kCus;
    if (beside > 0.f) us = fmaxf(n1 ? up : static_cast<float>((n2 + kCus - 1) / kCus) * c2, all);
    else if (n1 % kCus == 0) us = up + static_cast<float>((n2 + kCus - 1) / kCus) * c2;
    else us = fmaxf(up, all + (n2 ? 0.5f * c2 : 0.f));
  }
  uint32_t best = (__float_as_uint(us) & ~15u) | lane;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) best = min(best, static_cast<uint32_t>(__shfl_xor(static_cast<int>(best), o)));
  const int l = __builtin_amdgcn_readfirstlane(best) & 15, bm64 = (l & 3) + 1;
  MixedTiles m;
  m.rows256 = (count >> 8) - (l >> 2);
  m.bm = 64 * bm64;
  m.rows_bm = (count - m.rows256 * 256 + m.bm - 1) / m.bm;
  return m;
}

// Workgroup bid's tile of the counted rows among the mixed ones: its rows, 0 past
// the last tile, its first row and its column tile.
__device__ __forceinline__ int mixed_tile(int bid, int count, int tiles_n, int most, float beside, int& m0,
                                          int& tn) {
  const MixedTiles m = mix_tiles(count, tiles_n, most, beside);
  const int n256 = m.rows256 * tiles_n, rest = m.rows_bm * tiles_n;
  const bool large = bid < n256;
  if (bid >= n256 + rest) return 0;
  int tm;
  const int n = large ? n256 : rest;
  tile_place(xcd_remap(large ? bid : bid - n256, n), large ? m.rows256 : m.rows_bm, tiles_n, tm, tn);
  m0 = large ? tm * 256 : m.rows256 * 256 + tm * m.bm;
  return large ? 256 : m.bm;
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

inline int tiles(int64_t n, int b) { return static_cast<int>((n + b - 1) / b); }

inline int pick(int64_t M, int64_t N, bool bf16) {
  if (bf16) return pick_tile(kTileCosts, kTileKinds, M, N);
  return pick_tile(kTileCostsF32, kTileKindsF32, M, N);
}
// workgroups of tile t over M x N
inline int pick_count(int t, int64_t M, int64_t N, bool bf16) {
  const TileCost& c = bf16 ? kTileCosts[t] : kTileCostsF32[t];
  return tiles(M, c.bm) * tiles(N, c.bn);
}
// the kernel that has the tile: the wide ones share one
inline int kernel_of(int t, bool bf16) { return bf16 && t > kTile128x256 ? kTile128x256 : t; }

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

inline TileArgs tile_args(const VocabDesc& D) {
  TileArgs a{};
  a.r = D.rows;
  a.T = static_cast<int>(D.T);
  a.d = static_cast<int>(D.d);
  a.post = D.inv_temp;
  return a;
}

}  // namespace poetx
