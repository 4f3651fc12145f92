// Tile engine of the operators around the layer: C[M][N] = sum_k A[m][k]
// B[n][k] in bfloat16 or float (float32 sums) or int8 (int32 sums), one BM x BN
// tile of C per workgroup, left in registers for an epilogue of the caller's.
//
//  * Operands go global -> LDS with buffer loads that write LDS directly, 128
//    bytes of K (64 bfloat16, 32 float, 128 int8) a step, NS stages. The
//    buffer's record count ends at the operand's last byte, so rows past the
//    end read as zero without an address select; with KTAIL, 16-byte chunks
//    past the end of K get an offset outside the buffer for the same effect
//    (what lies between rows may be anything, NaN too).
//  * LDS rows of a K-contiguous operand are 128 bytes, chunk c of row r in
//    slot c ^ (r & 7): a fragment's 16-byte reads then never meet in a bank
//    (conflicts 0.1% of the LDS cycles; with the order for 32-row fragments,
//    which also turns with r / 8, 50%, though large products, bound by power,
//    took the same time).
//  * An operand stored with K as its rows (A[k][m], B[k][n]) lies in LDS as it
//    does in memory. bfloat16 is read with ds_read_b64_tr_b16, which hands
//    every lane four consecutive k of its own column, float word by word;
//    row_swizzle keeps the rows that one read touches on different banks.
//  * 16 x 16 matrix instructions with 64 bytes of K (v_mfma_f32_16x16x32_bf16):
//    under sustained load the chip's power limit, not the issue rate, bounds a
//    large product, and they read and write the sums half as often as the 32 x
//    32 ones. 8192 x 4096 x 16384 in bfloat16, a second of launches: 0.76 ms
//    (1.45 PFLOP/s) against 0.82 ms; both 0.57 to 0.59 ms on all-zero inputs,
//    where the chip does not throttle.
//  * A K step has four phases: the two halves of a wave's rows for each 64
//    bytes of K. Every phase reads the next one's fragments while its products
//    run, across the barrier too: it comes before the last phase, whose
//    fragments are in registers by then, and a stage's loads are issued in the
//    last phase before it and the two after it, two products, one read and one
//    load in turn. (One barrier at the top with the reads behind it: 0.87 ms.
//    Four waves of 128 x 128 in place of eight of 128 x 64: 0.84 ms or more.
//    Half steps in a ring of five slots: 0.89 ms. Wave priorities: 4% slower.)
//  * The MFMA takes B's fragment first: a lane then holds, for one row m (lane
//    % 16), groups of four consecutive columns n, and a row's reduction over
//    columns stays within a lane and its partners lane ^ 16, lane ^ 32.
#pragma once

#include "common.hpp"

namespace poetx {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned int tg_u32x4_t __attribute__((ext_vector_type(4)));

// Tiles of a product: it takes the one whose rounds over the CUs cost least. A
// round's time, measured with every slot taken, in us; it grows with K alike
// for all (but for the first loads and the epilogue, a larger share of a short K). 1- and 2-byte products, as the int8 product at 32 K steps (m =
// 4096): small tiles are chains of latencies, and more of them at once hide
// each other's (64 x 64 over two groups of waves, or two workgroups a CU).
enum TileKind { kTile64x2, kTile64, kTile128, kTile128x256, kTile192x256, kTile256, kTileKinds };
struct TileCost {
  int bm, bn, slots;
  double us;
};
constexpr TileCost kTileCosts[kTileKinds] = {{64, 64, 256, 11.2},   {64, 64, 512, 16.8},   {128, 128, 256, 22.0},
                                             {128, 256, 256, 35.0}, {192, 256, 256, 46.5}, {256, 256, 256, 57.0}};
// float products, per K step: nearly in proportion to the tile, as the matrix
// instructions bound all of them.
enum TileKindF32 { kTileF32, kTileF64, kTileF128, kTileKindsF32 };
constexpr TileCost kTileCostsF32[kTileKindsF32] = {{32, 32, 256, 0.17}, {64, 64, 256, 0.60}, {128, 128, 256, 2.03}};

// index of the cheapest of n tiles for an M x N product
inline int pick_tile(const TileCost* tiles, int n, int64_t M, int64_t N) {
  int best = -1;
  double least = 0;
  for (int i = 0; i < n; ++i) {
    const TileCost& t = tiles[i];
    const int64_t count = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    const double us = static_cast<double>((count + t.slots - 1) / t.slots) * t.us;
    if (best < 0 || us < least) {
      best = i;
      least = us;
    }
  }
  return best;
}

// A launch's threads in one dimension stay below 2^32: whether the chosen
// tile's workgroups (of at most 512, two products at most) do.
inline bool tiles_fit(const TileCost& t, int64_t M, int64_t N) {
  return ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn) < (int64_t(1) << 22);
}

// One operand: rows of K (K-contiguous), or rows of columns with K down.
// `rows`: rows of the stored matrix, `cols`: its row length, `ld`: row
// stride, both in elements.
struct TileOperand {
  const void* p;
  int64_t ld;
  int64_t rows;
  int64_t cols;
};

// ES: element bytes. AKC / BKC: operand K-contiguous. WM x WN waves.
// NS: stages; the loads of NS - 1 K steps are in flight. KG: groups of WM x WN
// waves that take K steps in turn, each with stages of its own; their sums
// are joined at the end and left with the first group.
template <int ES_, int BM_, int BN_, int WM_, int WN_, int NS_, bool AKC_, bool BKC_, bool KTAIL_, int KG_ = 1>
struct TileCfg {
  static constexpr int ES = ES_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_, KG = KG_;
  static constexpr bool AKC = AKC_, BKC = BKC_, KTAIL = KTAIL_;
  static constexpr int NW = WM * WN, NT = 64 * NW * KG;  // waves of a group, threads
  static constexpr int BK = 128 / ES;              // K of a step
  static constexpr int WTM = BM / WM, WTN = BN / WN;
  static constexpr int TM = WTM / 16, TN = WTN / 16, H = TM / 2;  // 16 x 16 tiles of a wave, row tiles of a phase
  static constexpr int ABYTES = BM * 128, BBYTES = BN * 128, STAGE = ABYTES + BBYTES;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KB loads a wave
  static constexpr int SLAB = WTN + 8;             // epilogue slab row, floats
  static constexpr int SLABS = NW * 32 * SLAB * 4;
  static constexpr int RING = NS * STAGE;
  static constexpr int JOIN = (KG - 1) * BM * BN * 4;
  static_assert(BM % (16 * WM) == 0 && TM % 2 == 0 && BN % (16 * WN) == 0, "16 x 16 tiles in two halves");
  static constexpr int LDS = KG * RING > SLABS ? (KG * RING > JOIN ? KG * RING : JOIN) : (SLABS > JOIN ? SLABS : JOIN);
  static_assert((AKC || BM * ES >= 128) && (BKC || BN * ES >= 128), "rows of K of whole bank quarters");
  static_assert(ES != 1 || (AKC && BKC), "no transposed reads of bytes");
  static_assert(LA >= 1 && LB >= 1 && LDS <= 160 * 1024, "tile");
};

template <int ES>
struct TileAcc {
  typedef f32x4_t type;
};
template <>
struct TileAcc<1> {
  typedef i32x4_t type;
};

template <int ES>
struct TileFrag {
  typedef bf16x8_t type;
};
template <>
struct TileFrag<1> {
  typedef i32x4_t type;
};
template <>
struct TileFrag<4> {
  typedef f32x4_t type;
};
// sixteen k of a float fragment: four products of four
__device__ __forceinline__ f32x4_t tile_mfma(f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4_t tile_mfma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ i32x4_t tile_mfma(i32x4_t a, i32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void tg_wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Slot of chunk c in row r of K of a tile of BT columns: c ^ row_swizzle(r).
// A transposed read takes 32 bytes each of rows 0 to 3 and 8 to 11 (then 16 to
// 19 and 24 to 27) at a time: eight different 32-byte pieces of the 256-byte
// bank window, which holds one row, or two of 128 bytes. A float read takes 64
// bytes each of rows 0, 4, 8 and 12.
template <int BT, int ES>
__device__ __forceinline__ int row_swizzle(int r) {
  if constexpr (ES == 4) return BT >= 64 ? ((r >> 2) & 3) << 2 : ((r >> 2) & 1) << 2;
  else if constexpr (BT * ES == 128) return (((r >> 1) & 1) << 2) ^ (((r >> 3) & 1) << 1);
  else return ((r & 3) << 2) ^ (((r >> 3) & 1) << 1);
}

// Slot of chunk c in row r of a K-contiguous tile: c ^ chunk_swizzle(r), for
// fragments of FR rows.
template <int FR>
__device__ __forceinline__ int chunk_swizzle(int r) {
  return FR == 16 ? r & 7 : (r & 7) ^ ((r >> 3) & 1);
}

// The loads of one operand tile: per-lane byte offsets from the tile's first
// byte, and the tile's buffer.
template <int BT, int L, bool KC, int ES, bool KTAIL, int FR = 16>
struct TileLoader {
  const char* base;     // first byte of the tile's stored rows at k = 0
  int64_t left;         // bytes from there to the operand's end
  int64_t kstep;        // bytes a K step advances
  uint32_t voff[L];
  uint32_t vtail[KC && KTAIL ? L : 1];  // the same in the step that K ends in: chunks past it outside the buffer
  int tail;                              // that step

  __device__ __forceinline__ void init(const TileOperand& o, int row0, int k0, int wave, int lane) {
    const int64_t ldb = o.ld * ES;
    const int kend = static_cast<int>((o.cols - k0) * ES % 128);
    tail = kend ? static_cast<int>((o.cols - k0) * ES / 128) : -1;
    if constexpr (KC) {
      base = static_cast<const char*>(o.p) + row0 * ldb + static_cast<int64_t>(k0) * ES;
      left = (o.rows - 1 - row0) * ldb + (o.cols - k0) * ES;
      kstep = 128;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int r = (wave * L + i) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ chunk_swizzle<FR>(r);
        voff[i] = static_cast<uint32_t>(r * ldb) + c * 16;
        if constexpr (KTAIL) vtail[i] = c * 16 < kend ? voff[i] : 0xfffffff0u;
      }
    } else {
      constexpr int RB = BT * ES, CH = RB / 16, RPI = 64 / CH;
      base = static_cast<const char*>(o.p) + k0 * ldb + static_cast<int64_t>(row0) * ES;
      left = (o.rows - 1 - k0) * ldb + (o.cols - row0) * ES;
      kstep = 128 / ES * ldb;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int r = (wave * L + i) * RPI + lane / CH;
        const int c = (lane % CH) ^ row_swizzle<BT, ES>(r);
        voff[i] = static_cast<uint32_t>(r * ldb) + c * 16;
      }
    }
  }

  // load i of K step `it` into the operand's tile at `lds`
  __device__ __forceinline__ void load(int i, int it, char* lds, int wave) const {
    const int64_t adv = it * kstep;
    const int64_t rem = left - adv;
    const uint32_t num = rem <= 0 ? 0u : (rem > 0x7fffffff ? 0x7fffffffu : static_cast<uint32_t>(rem));
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base + adv), 0, static_cast<int>(num), 0x00020000);
    uint32_t v = voff[i];
    if constexpr (KC && KTAIL) v = it == tail ? vtail[i] : v;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * L + i) * 1024), 16, static_cast<int>(v), 0, 0, 0);
  }
};

// Transposed-read address (bytes in the operand's tile) of a lane for the
// 16-column fragment at column `col0`, first 32 rows of K: lane group G reads
// rows 8 G .. 8 G + 7, its lane i addressing row i / 4, column 4 (i % 4).
template <int BT>
__device__ __forceinline__ uint32_t tr_addr(int col0, int lane) {
  const int li = lane & 15;
  const int r = 8 * (lane >> 4) + (li >> 2);
  const int col = col0 + 4 * (li & 3);
  return static_cast<uint32_t>(r * BT * 2 + (((col >> 3) ^ row_swizzle<BT, 2>(r)) << 4) + (col & 7) * 2);
}

// bfloat16 fragments by transposed reads, rows +4 in the second read of each;
// an asm block waits for its own results (as builtins the reads would wait for
// the direct loads in flight).
typedef unsigned long long tr_u64;
typedef unsigned long long tr_u64x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bf16x8_t tr_frag(tr_u64 lo, tr_u64 hi) {
  return __builtin_bit_cast(bf16x8_t, tr_u64x2{lo, hi});
}
#define POETX_TR(lo, hi, ad, off) \
  "ds_read_b64_tr_b16 %" #lo ", %" #ad "\n ds_read_b64_tr_b16 %" #hi ", %" #ad " offset:%" #off "\n"
template <int BT>
__device__ __forceinline__ void tr_read(const uint32_t* a, uint32_t off, bf16x8_t (&f)[1]) {
  tr_u64 r[2];
  asm volatile(POETX_TR(0, 1, 2, 3) "s_waitcnt lgkmcnt(0)"
               : "=&v"(r[0]), "=&v"(r[1])
               : "v"(a[0] + off), "n"(4 * BT * 2)
               : "memory");
  f[0] = tr_frag(r[0], r[1]);
}
template <int BT>
__device__ __forceinline__ void tr_read(const uint32_t* a, uint32_t off, bf16x8_t (&f)[2]) {
  tr_u64 r[4];
  asm volatile(POETX_TR(0, 1, 4, 6) POETX_TR(2, 3, 5, 6) "s_waitcnt lgkmcnt(0)"
               : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
               : "v"(a[0] + off), "v"(a[1] + off), "n"(4 * BT * 2)
               : "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i) f[i] = tr_frag(r[2 * i], r[2 * i + 1]);
}
template <int BT>
__device__ __forceinline__ void tr_read(const uint32_t* a, uint32_t off, bf16x8_t (&f)[4]) {
  tr_u64 r[8];
  asm volatile(POETX_TR(0, 1, 8, 12) POETX_TR(2, 3, 9, 12) POETX_TR(4, 5, 10, 12) POETX_TR(6, 7, 11, 12)
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]),
                 "=&v"(r[7])
               : "v"(a[0] + off), "v"(a[1] + off), "v"(a[2] + off), "v"(a[3] + off), "n"(4 * BT * 2)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = tr_frag(r[2 * i], r[2 * i + 1]);
}
// four fragments each of two operands under one wait
template <int BTA, int BTB>
__device__ __forceinline__ void tr_read(const uint32_t* a, uint32_t offa, bf16x8_t (&fa)[4], const uint32_t* b,
                                        uint32_t offb, bf16x8_t (&fb)[4]) {
  tr_u64 r[8], s[8];
  asm volatile(POETX_TR(0, 1, 16, 24) POETX_TR(2, 3, 17, 24) POETX_TR(4, 5, 18, 24) POETX_TR(6, 7, 19, 24)
               POETX_TR(8, 9, 20, 25) POETX_TR(10, 11, 21, 25) POETX_TR(12, 13, 22, 25) POETX_TR(14, 15, 23, 25)
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]),
                 "=&v"(r[7]), "=&v"(s[0]), "=&v"(s[1]), "=&v"(s[2]), "=&v"(s[3]), "=&v"(s[4]), "=&v"(s[5]),
                 "=&v"(s[6]), "=&v"(s[7])
               : "v"(a[0] + offa), "v"(a[1] + offa), "v"(a[2] + offa), "v"(a[3] + offa), "v"(b[0] + offb),
                 "v"(b[1] + offb), "v"(b[2] + offb), "v"(b[3] + offb), "n"(4 * BTA * 2), "n"(4 * BTB * 2)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fa[i] = tr_frag(r[2 * i], r[2 * i + 1]);
    fb[i] = tr_frag(s[2 * i], s[2 * i + 1]);
  }
}
#undef POETX_TR

// Address of a lane's column in the fragment of float rows at column col0:
// rows 16 kk + 4 (lane / 16) + e, e = 0..3, of K group kk; the rows' slots do
// not depend on kk or e.
template <int BT>
__device__ __forceinline__ uint32_t row_addr_f32(int col0, int lane) {
  const int r = 4 * (lane >> 4), col = col0 + (lane & 15);
  return static_cast<uint32_t>(r * BT * 4 + (((col >> 2) ^ row_swizzle<BT, 4>(r)) << 4) + (col & 3) * 4);
}
template <int BT, int N>
__device__ __forceinline__ void row_read(const char* tile, const uint32_t* a, int kk, f32x4_t (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) f[i][e] = *reinterpret_cast<const float*>(tile + a[i] + (kk * 16 + e) * BT * 4);
}

// The wave's TM x TN tiles of 16 x 16 of the workgroup's tile at (m0, n0),
// over K steps [it0, it1). lds: Cfg::LDS bytes, free again for the caller when
// this returns (after its barrier).
template <class Cfg>
__device__ __forceinline__ void tile_product(const TileOperand& A, const TileOperand& B, int m0, int n0,
                                             int it0, int it1, char* lds,
                                             typename TileAcc<Cfg::ES>::type (&acc)[Cfg::TM][Cfg::TN]) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN, H = Cfg::H, LA = Cfg::LA, LB = Cfg::LB;
  const int lane = threadIdx.x & 63;
  const int gwave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = gwave % Cfg::NW, group = gwave / Cfg::NW;
  char* const smem = lds + group * Cfg::RING;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;

  TileLoader<Cfg::BM, LA, Cfg::AKC, Cfg::ES, Cfg::KTAIL> la;
  TileLoader<Cfg::BN, LB, Cfg::BKC, Cfg::ES, Cfg::KTAIL> lb;
  la.init(A, m0, 0, wave, lane);
  lb.init(B, n0, 0, wave, lane);

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = 0;
  if (it0 >= it1) {
    __syncthreads();
    return;
  }

  // fragment addresses: K group kk of a K-contiguous row is chunk 4 kk +
  // lane / 16 (64 bytes of K)
  const int lrow = lane & 15;
  const int sw = chunk_swizzle<16>(lrow);
  int koff[2];
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) koff[kk] = lrow * 128 + (((4 * kk + (lane >> 4)) ^ sw) << 4);
  const int abase = wm * Cfg::WTM * 128, bbase = Cfg::ABYTES + wn * Cfg::WTN * 128;
  uint32_t acol[Cfg::AKC ? 1 : TM], bcol[Cfg::BKC ? 1 : TN];
  if constexpr (!Cfg::AKC) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int col = wm * Cfg::WTM + i * 16;
      acol[i] = Cfg::ES == 2 ? tr_addr<Cfg::BM>(col, lane) : row_addr_f32<Cfg::BM>(col, lane);
    }
  }
  if constexpr (!Cfg::BKC) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = wn * Cfg::WTN + j * 16;
      bcol[j] = Cfg::ABYTES + (Cfg::ES == 2 ? tr_addr<Cfg::BN>(col, lane) : row_addr_f32<Cfg::BN>(col, lane));
    }
  }

  // half h of the rows' fragments for K group kk, and the columns' fragments
  typedef typename TileFrag<Cfg::ES>::type Frag;
  auto read_a = [&](const char* st, int kk, int h, Frag(&f)[H]) {
    const uint32_t sb = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(st));
    if constexpr (Cfg::AKC) {
#pragma unroll
      for (int i = 0; i < H; ++i) f[i] = *reinterpret_cast<const Frag*>(st + abase + (h * H + i) * 16 * 128 + koff[kk]);
    } else if constexpr (Cfg::ES == 2) {
      tr_read<Cfg::BM>(acol + h * H, sb + kk * 32 * Cfg::BM * 2, f);
    } else {
      row_read<Cfg::BM, H>(st, acol + h * H, kk, f);
    }
  };
  auto read_b = [&](const char* st, int kk, Frag(&f)[TN]) {
    const uint32_t sb = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(st));
    if constexpr (Cfg::BKC) {
#pragma unroll
      for (int j = 0; j < TN; ++j) f[j] = *reinterpret_cast<const Frag*>(st + bbase + j * 16 * 128 + koff[kk]);
    } else if constexpr (Cfg::ES == 2) {
      tr_read<Cfg::BN>(bcol, sb + kk * 32 * Cfg::BN * 2, f);
    } else {
      row_read<Cfg::BN, TN>(st, bcol, kk, f);
    }
  };
  auto read_ab = [&](const char* st, int kk, Frag(&fa)[H], Frag(&fb)[TN]) {
    if constexpr (Cfg::ES == 2 && !Cfg::AKC && !Cfg::BKC && H == 4 && TN == 4) {
      const uint32_t sb = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(st));
      tr_read<Cfg::BM, Cfg::BN>(acol, sb + kk * 32 * Cfg::BM * 2, fa, bcol, sb + kk * 32 * Cfg::BN * 2, fb);
    } else {
      read_b(st, kk, fb);
      read_a(st, kk, 0, fa);
    }
  };

  // The loads of a stage: N3 in the last phase of the step that frees its slot,
  // the others in the next step's first. Steps past the last load the last slice
  // again, into slots that are idle by then, so that the same number of loads is
  // always in flight.
  constexpr int L = LA + LB, N3 = (L + 1) / 2;
  auto step_of = [&](int it) { return min(it + group, it1 - 1); };
  auto load = [&](int i, int pf, char* to) {
    if (i < LA) la.load(i, pf, to, wave);
    else lb.load(i - LA, pf, to + Cfg::ABYTES, wave);
  };
#pragma unroll
  for (int s = 0; s < Cfg::NS; ++s)
#pragma unroll
    for (int i = 0; i < (s < Cfg::NS - 1 ? L : N3); ++i) load(i, step_of(it0 + s * Cfg::KG), smem + s * Cfg::STAGE);
  tg_wait_vm<(Cfg::NS - 2) * L + N3>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frag af[2][H], bf[2][TN];
  read_ab(smem, 0, af[0], bf[0]);

  int cur = 0;
  for (int it = it0; it < it1; it += Cfg::KG) {
    const bool mine = Cfg::KG == 1 || it + group < it1;  // a group may have no step left
    char* const st = smem + cur * Cfg::STAGE;
    char* const prev = smem + (cur == 0 ? Cfg::NS - 1 : cur - 1) * Cfg::STAGE;
    cur = cur == Cfg::NS - 1 ? 0 : cur + 1;
    const char* const nxt = smem + cur * Cfg::STAGE;
    const int pf = step_of(it + (Cfg::NS - 1) * Cfg::KG), pf2 = step_of(it + Cfg::NS * Cfg::KG);
#pragma unroll
    for (int ph = 0; ph < 4; ++ph) {
      const int kk = ph >> 1, h = ph & 1;
      __builtin_amdgcn_sched_barrier(0);
      if (ph == 3) {
        // this stage's reads are done and the next stage's loads (the oldest)
        // have landed, in every wave after the barrier; a bare one
        // (__syncthreads would wait for the younger loads too)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        tg_wait_vm<(Cfg::NS - 2) * L>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < N3; ++i) load(i, pf2, st);
        read_ab(nxt, 0, af[0], bf[0]);
      } else {
        constexpr int N0 = L - N3;
        const int first = ph == 0 ? N3 : L, last = ph == 0 ? N3 + N0 : L;
#pragma unroll
        for (int i = 0; i < L; ++i)
          if (i >= first && i < last) load(i, pf, prev);
        if (ph == 0) read_a(st, 0, 1, af[1]);
        else if (ph == 1) read_ab(st, 1, af[0], bf[1]);
        else read_a(st, 1, 1, af[1]);
      }
#pragma unroll
      for (int i = 0; i < H; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (mine) acc[h * H + i][j] = tile_mfma(bf[kk][j], af[h][i], acc[h * H + i][j]);
      if constexpr (H * TN >= 12) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, (H * TN + 4) / 8, 0);  // products
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);           // LDS reads
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);           // loads
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the last loads must land before the caller uses the LDS
  tg_wait_vm<0>();
  __syncthreads();
  if constexpr (Cfg::KG > 1) {
    // [group - 1][wave][tile][lane], 16 bytes a lane
    typedef typename TileAcc<Cfg::ES>::type Acc;
    Acc* const join = reinterpret_cast<Acc*>(lds) + wave * TM * TN * 64 + lane;
    constexpr int GROUP = Cfg::NW * TM * TN * 64;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (group > 0) join[(group - 1) * GROUP + (i * TN + j) * 64] = acc[i][j];
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < Cfg::KG; ++g)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] += join[(g - 1) * GROUP + (i * TN + j) * 64];
    }
    __syncthreads();
  }
}

// Row and column (of the workgroup's tile) of register r of tile (i, j) of a lane
template <class Cfg>
__device__ __forceinline__ int tile_row(int wm, int lane, int i) {
  return wm * Cfg::WTM + i * 16 + (lane & 15);
}
template <class Cfg>
__device__ __forceinline__ int tile_col(int wn, int lane, int j, int r) {
  return wn * Cfg::WTN + j * 16 + (lane >> 4) * 4 + r;
}

// Hands the wave's values, as float, row by row through its LDS slab to
// out(row, col, v[8]): 8 consecutive columns of a row of the workgroup's
// tile, whole lines of a row in consecutive lanes.
template <class Cfg, class Out>
__device__ __forceinline__ void tile_rows(const typename TileAcc<Cfg::ES>::type (&acc)[Cfg::TM][Cfg::TN], char* smem,
                                          Out&& out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave >= Cfg::NW) return;  // the first group holds the sums
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
  float* slab = reinterpret_cast<float*>(smem) + wave * 32 * Cfg::SLAB;
  constexpr int CPR = Cfg::WTN / 8, CPL = 32 * CPR / 64;
#pragma unroll
  for (int i = 0; i < Cfg::TM / 2; ++i) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < Cfg::TN; ++j) {
        const auto& v = acc[2 * i + u][j];
        *reinterpret_cast<float4*>(slab + (u * 16 + (lane & 15)) * Cfg::SLAB + j * 16 + (lane >> 4) * 4) =
            make_float4(static_cast<float>(v[0]), static_cast<float>(v[1]), static_cast<float>(v[2]), static_cast<float>(v[3]));
      }
    // the slab is the wave's own: its LDS accesses complete in order
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int ch = lane + c * 64;
      const int row = ch / CPR, col = (ch % CPR) * 8;
      const float4 a = *reinterpret_cast<const float4*>(slab + row * Cfg::SLAB + col);
      const float4 b = *reinterpret_cast<const float4*>(slab + row * Cfg::SLAB + col + 4);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      out(wm * Cfg::WTM + i * 32 + row, wn * Cfg::WTN + col, v);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// Tile (tm, tn) of index pid: groups of 4 tile rows walked column by column,
// so that neighbouring pids share operand panels.
__device__ __forceinline__ void tile_place(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 4;
  const int group = GM * tiles_n;
  const int first = (pid / group) * GM;
  const int size = min(tiles_m - first, GM);
  tm = first + (pid % group) % size;
  tn = (pid % group) / size;
}

__device__ __forceinline__ void tile_store8(bf16_t* p, const float (&v)[8]) {
  const tg_u32x4_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                        pack_bf16x2(v[6], v[7])};
  __builtin_nontemporal_store(w, reinterpret_cast<tg_u32x4_t*>(p));
}
__device__ __forceinline__ void tile_store8(float* p, const float (&v)[8]) {
  const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
  __builtin_nontemporal_store(a, reinterpret_cast<f32x4_t*>(p));
  __builtin_nontemporal_store(b, reinterpret_cast<f32x4_t*>(p + 4));
}

}  // namespace poetx
