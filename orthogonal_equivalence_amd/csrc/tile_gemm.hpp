// Tile engine of the operators around the layer: C[M][N] = sum_k A[m][k]
// B[n][k] in bfloat16 or float (float32 sums) or int8 (int32 sums), one BM x BN
// tile of C per workgroup, left in registers for an epilogue of the caller's.
//
//  * Operands go global -> LDS with buffer loads that write LDS directly, 128
//    bytes of K (64 bfloat16, 32 float, 128 int8) a step, NS stages, one barrier a
//    step, a later stage's loads spread over the current stage's MFMAs. The
//    buffer's record count ends at the operand's last byte, so rows past the
//    end read as zero without an address select; with KTAIL, 16-byte chunks
//    past the end of K get an offset outside the buffer for the same effect
//    (what lies between rows may be anything, NaN too).
//  * LDS rows of a K-contiguous operand are 128 bytes, chunk c of row r in
//    slot c ^ (r & 7) ^ ((r >> 3) & 1): the 32 rows of a fragment read fall on
//    all banks evenly.
//  * An operand stored with K as its rows (A[k][m], B[k][n]) lies in LDS as it
//    does in memory. bfloat16 is read with ds_read_b64_tr_b16, which hands
//    every lane four consecutive k of its own column; chunk c of row r is in
//    slot c ^ 4 (r & 3) (row_swizzle), so the four rows of a read fall in four
//    different 64-byte quarters of the banks. float is read word by word, the two halves
//    of a wave four rows apart; slot c ^ 8 ((r >> 2) & 1) keeps their banks
//    apart.
//  * The MFMA takes B's fragment first: a lane then holds, for one row m
//    (lane % 32), groups of four consecutive columns n, and a row's reduction
//    over columns stays within a lane and its partner lane ^ 32.
#pragma once

#include "common.hpp"

namespace poetx {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned int tg_u32x4_t __attribute__((ext_vector_type(4)));

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
  static constexpr int TM = WTM / 32, TN = WTN / 32;
  static constexpr int ABYTES = BM * 128, BBYTES = BN * 128, STAGE = ABYTES + BBYTES;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KB loads a wave
  static constexpr int SLAB = WTN + 8;             // epilogue slab row, floats
  static constexpr int SLABS = NW * 32 * SLAB * 4;
  static constexpr int RING = NS * STAGE;
  static constexpr int JOIN = (KG - 1) * BM * BN * 4;
  static constexpr int LDS = KG * RING > SLABS ? (KG * RING > JOIN ? KG * RING : JOIN) : (SLABS > JOIN ? SLABS : JOIN);
  static_assert((AKC || BM * ES >= 128) && (BKC || BN * ES >= 128), "rows of K of whole bank quarters");
  static_assert(ES != 1 || (AKC && BKC), "no transposed reads of bytes");
  static_assert(LA >= 1 && LB >= 1 && LDS <= 160 * 1024, "tile");
};

template <int ES>
struct TileAcc {
  typedef f32x16_t type;
};
template <>
struct TileAcc<1> {
  typedef i32x16_t type;
};

template <int ES>
struct TileQuad {
  typedef f32x4_t type;
};
template <>
struct TileQuad<1> {
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
// eight k of a float fragment: four products of two
__device__ __forceinline__ f32x16_t tile_mfma(f32x4_t a, f32x4_t b, f32x16_t c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x16_t tile_mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ i32x16_t tile_mfma(i32x4_t a, i32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void tg_wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Slot of chunk c in row r of K of a tile of BT columns: c ^ row_swizzle(r),
// the same for rows 4 (bfloat16) or 8 (float) further on. Rows of 128 bytes
// come two to a 256-byte bank window, wider ones one or less.
template <int BT, int ES>
__device__ __forceinline__ int row_swizzle(int r) {
  if constexpr (ES == 4) return BT >= 64 ? ((r >> 2) & 1) << 3 : 0;
  else if constexpr (BT * ES == 128) return ((r >> 1) & 1) << 2;
  else return (r & 3) << 2;
}

// The loads of one operand tile: per-lane byte offsets from the tile's first
// byte, and the tile's buffer.
template <int BT, int L, bool KC, int ES, bool KTAIL>
struct TileLoader {
  const char* base;     // first byte of the tile's stored rows at k = 0
  int64_t left;         // bytes from there to the operand's end
  int64_t kstep;        // bytes a K step advances
  uint32_t voff[L];
  uint32_t kchunk[KC && KTAIL ? L : 1];  // byte of K of the lane's chunk

  __device__ __forceinline__ void init(const TileOperand& o, int row0, int k0, int wave, int lane) {
    const int64_t ldb = o.ld * ES;
    if constexpr (KC) {
      base = static_cast<const char*>(o.p) + row0 * ldb + static_cast<int64_t>(k0) * ES;
      left = (o.rows - 1 - row0) * ldb + (o.cols - k0) * ES;
      kstep = 128;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int r = (wave * L + i) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ (r & 7) ^ ((r >> 3) & 1);
        voff[i] = static_cast<uint32_t>(r * ldb) + c * 16;
        if constexpr (KTAIL) kchunk[i] = c * 16;
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

  // load i of K step `it` into the operand's tile at `lds`; kleft: bytes of K
  // from the step's start (KTAIL)
  __device__ __forceinline__ void load(int i, int it, int64_t kleft, char* lds, int wave) const {
    const int64_t adv = it * kstep;
    const int64_t rem = left - adv;
    const uint32_t num = rem <= 0 ? 0u : (rem > 0x7fffffff ? 0x7fffffffu : static_cast<uint32_t>(rem));
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base + adv), 0, static_cast<int>(num), 0x00020000);
    uint32_t v = voff[i];
    if constexpr (KC && KTAIL) v = kchunk[i] < kleft ? v : 0xfffffff0u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * L + i) * 1024), 16, static_cast<int>(v), 0, 0, 0);
  }
};

// Transposed-read address (bytes in the operand's tile) of a lane for the
// 32-column fragment at column `col0`, first 16 rows of K.
template <int BT>
__device__ __forceinline__ uint32_t tr_addr(int col0, int lane) {
  const int grp = lane >> 4, li = lane & 15;
  const int r = 8 * (grp >> 1) + (li >> 2);
  const int col = col0 + 16 * (grp & 1) + 4 * (li & 3);
  return static_cast<uint32_t>(r * BT * 2 + (((col >> 3) ^ row_swizzle<BT, 2>(r)) << 4) + (col & 7) * 2);
}

// One, two or four bfloat16 fragments by transposed reads; each asm block
// waits for its own results (as builtins the reads would wait for the direct
// loads in flight).
template <int BT>
__device__ __forceinline__ void tr_read(const uint32_t (&a)[1], uint32_t off, bf16x8_t (&f)[1]) {
  typedef unsigned long long u64;
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  u64 r[2];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %2\n ds_read_b64_tr_b16 %1, %2 offset:%3\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1])
      : "v"(a[0] + off), "n"(4 * BT * 2)
      : "memory");
  f[0] = __builtin_bit_cast(bf16x8_t, u64x2{r[0], r[1]});
}
template <int BT>
__device__ __forceinline__ void tr_read(const uint32_t (&a)[2], uint32_t off, bf16x8_t (&f)[2]) {
  typedef unsigned long long u64;
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  u64 r[4];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4\n ds_read_b64_tr_b16 %1, %4 offset:%6\n"
      "ds_read_b64_tr_b16 %2, %5\n ds_read_b64_tr_b16 %3, %5 offset:%6\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
      : "v"(a[0] + off), "v"(a[1] + off), "n"(4 * BT * 2)
      : "memory");
  f[0] = __builtin_bit_cast(bf16x8_t, u64x2{r[0], r[1]});
  f[1] = __builtin_bit_cast(bf16x8_t, u64x2{r[2], r[3]});
}
template <int BT>
__device__ __forceinline__ void tr_read(const uint32_t (&a)[4], uint32_t off, bf16x8_t (&f)[4]) {
  typedef unsigned long long u64;
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  u64 r[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n ds_read_b64_tr_b16 %1, %8 offset:%12\n"
      "ds_read_b64_tr_b16 %2, %9\n ds_read_b64_tr_b16 %3, %9 offset:%12\n"
      "ds_read_b64_tr_b16 %4, %10\n ds_read_b64_tr_b16 %5, %10 offset:%12\n"
      "ds_read_b64_tr_b16 %6, %11\n ds_read_b64_tr_b16 %7, %11 offset:%12\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
      : "v"(a[0] + off), "v"(a[1] + off), "v"(a[2] + off), "v"(a[3] + off), "n"(4 * BT * 2)
      : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __builtin_bit_cast(bf16x8_t, u64x2{r[2 * i], r[2 * i + 1]});
}

// Address of a lane's column in the fragment of float rows at column col0:
// rows 8 kk + 4 (lane / 32) + e, e = 0..3, of K group kk. The rows' slots are
// those of row 4 (lane / 32) in every group.
template <int BT>
__device__ __forceinline__ uint32_t row_addr_f32(int col0, int lane) {
  const int half = lane >> 5, col = col0 + (lane & 31);
  return static_cast<uint32_t>(half * 4 * BT * 4 + (((col >> 2) ^ row_swizzle<BT, 4>(half * 4)) << 4) + (col & 3) * 4);
}
template <int BT, int N>
__device__ __forceinline__ void row_read(const char* tile, const uint32_t (&a)[N], int kk, f32x4_t (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) f[i][e] = *reinterpret_cast<const float*>(tile + a[i] + (kk * 8 + e) * BT * 4);
}

// The wave's TM x TN tiles of 32 x 32 of the workgroup's tile at (m0, n0),
// over K steps [it0, it1) of a K of `K` elements. smem: Cfg::LDS bytes, free
// again for the caller when this returns (after its barrier).
template <class Cfg>
__device__ __forceinline__ void tile_product(const TileOperand& A, const TileOperand& B, int m0, int n0, int64_t K,
                                             int it0, int it1, char* lds,
                                             typename TileAcc<Cfg::ES>::type (&acc)[Cfg::TM][Cfg::TN]) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN, LA = Cfg::LA, LB = Cfg::LB;
  const int lane = threadIdx.x & 63;
  const int gwave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = gwave % Cfg::NW, group = gwave / Cfg::NW;
  char* const smem = lds + group * Cfg::RING;
  const int wm = wave % Cfg::WM, wn = wave / Cfg::WM;
  const int64_t Kb = K * Cfg::ES;

  TileLoader<Cfg::BM, LA, Cfg::AKC, Cfg::ES, Cfg::KTAIL> la;
  TileLoader<Cfg::BN, LB, Cfg::BKC, Cfg::ES, Cfg::KTAIL> lb;
  la.init(A, m0, 0, wave, lane);
  lb.init(B, n0, 0, wave, lane);

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  if (it0 >= it1) {
    __syncthreads();
    return;
  }

  // fragment addresses: K group kk of a K-contiguous row is chunk 2 kk +
  // lane / 32 (32 bytes of K)
  const int lrow = lane & 31;
  const int sw = (lrow & 7) ^ ((lrow >> 3) & 1);
  int koff[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) koff[kk] = lrow * 128 + (((2 * kk + (lane >> 5)) ^ sw) << 4);
  const int abase = wm * Cfg::WTM * 128, bbase = Cfg::ABYTES + wn * Cfg::WTN * 128;
  uint32_t acol[Cfg::AKC ? 1 : TM], bcol[Cfg::BKC ? 1 : TN];
  if constexpr (!Cfg::AKC) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int col = wm * Cfg::WTM + i * 32;
      acol[i] = Cfg::ES == 2 ? tr_addr<Cfg::BM>(col, lane) : row_addr_f32<Cfg::BM>(col, lane);
    }
  }
  if constexpr (!Cfg::BKC) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = wn * Cfg::WTN + j * 32;
      bcol[j] = Cfg::ABYTES + (Cfg::ES == 2 ? tr_addr<Cfg::BN>(col, lane) : row_addr_f32<Cfg::BN>(col, lane));
    }
  }

  typedef typename TileFrag<Cfg::ES>::type Frag;
  auto read = [&](const char* st, int kk, Frag(&fa)[TM], Frag(&fb)[TN]) {
    const uint32_t sb = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(st));
    if constexpr (Cfg::AKC) {
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = *reinterpret_cast<const Frag*>(st + abase + i * 32 * 128 + koff[kk]);
    } else if constexpr (Cfg::ES == 2) {
      tr_read<Cfg::BM>(acol, sb + kk * 16 * Cfg::BM * 2, fa);
    } else {
      row_read<Cfg::BM, TM>(st, acol, kk, fa);
    }
    if constexpr (Cfg::BKC) {
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = *reinterpret_cast<const Frag*>(st + bbase + j * 32 * 128 + koff[kk]);
    } else if constexpr (Cfg::ES == 2) {
      tr_read<Cfg::BN>(bcol, sb + kk * 16 * Cfg::BN * 2, fb);
    } else {
      row_read<Cfg::BN, TN>(st, bcol, kk, fb);
    }
  };

  // steps past the last load the last slice again, into stages that are idle
  // by then, so that the same number of loads is always in flight
#pragma unroll
  for (int s = 0; s < Cfg::NS - 1; ++s) {
    const int pf = min(it0 + s * Cfg::KG + group, it1 - 1);
    const int64_t kleft = Kb - static_cast<int64_t>(pf) * 128;
#pragma unroll
    for (int i = 0; i < LA; ++i) la.load(i, pf, kleft, smem + s * Cfg::STAGE, wave);
#pragma unroll
    for (int i = 0; i < LB; ++i) lb.load(i, pf, kleft, smem + s * Cfg::STAGE + Cfg::ABYTES, wave);
  }

  int cur = 0;
  for (int it = it0; it < it1; it += Cfg::KG) {
    // this step's loads are the oldest; a bare barrier (__syncthreads would
    // wait for the younger ones too)
    tg_wait_vm<(Cfg::NS - 2) * (LA + LB)>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const char* st = smem + cur * Cfg::STAGE;
    char* nxt = smem + (cur == 0 ? Cfg::NS - 1 : cur - 1) * Cfg::STAGE;
    cur = cur == Cfg::NS - 1 ? 0 : cur + 1;
    const int pf = min(it + (Cfg::NS - 1) * Cfg::KG + group, it1 - 1);
    const bool mine = Cfg::KG == 1 || it + group < it1;  // a group may have no step left
    const int64_t kleft = Kb - static_cast<int64_t>(pf) * 128;
    Frag af[2][TM], bf[2][TN];
    read(st, 0, af[0], bf[0]);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      constexpr int L = LA + LB;
      const int first = L == 8 ? (kk == 0 ? 0 : kk == 1 ? 2 : kk == 2 ? 5 : 8) : kk * L / 4;
      const int last = L == 8 ? (kk == 0 ? 2 : kk == 1 ? 5 : 8) : (kk + 1) * L / 4;
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (i >= first && i < last) {
          if (i < LA) la.load(i, pf, kleft, nxt, wave);
          else lb.load(i - LA, pf, kleft, nxt + Cfg::ABYTES, wave);
        }
      // the next group's fragments are on their way while this group's
      // products run
      if (kk < 3) read(st, kk + 1, af[(kk + 1) & 1], bf[(kk + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          if (mine) acc[i][j] = tile_mfma(bf[kk & 1][j], af[kk & 1][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the last loads must land before the caller uses the LDS
  tg_wait_vm<0>();
  __syncthreads();
  if constexpr (Cfg::KG > 1) {
    // [group - 1][wave][tile][quad of registers][lane], 16 bytes a lane
    typedef typename TileQuad<Cfg::ES>::type Quad;
    Quad* const join = reinterpret_cast<Quad*>(lds) + wave * TM * TN * 256 + lane;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (group > 0)
            join[(group - 1) * Cfg::NW * TM * TN * 256 + (i * TN + j) * 256 + q * 64] =
                Quad{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < Cfg::KG; ++g)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const Quad v = join[(g - 1) * Cfg::NW * TM * TN * 256 + (i * TN + j) * 256 + q * 64];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
            }
    }
    __syncthreads();
  }
}

// Row and column (of the workgroup's tile) of register r of tile (i, j) of a lane
template <class Cfg>
__device__ __forceinline__ int tile_row(int wm, int lane, int i) {
  return wm * Cfg::WTM + i * 32 + (lane & 31);
}
template <class Cfg>
__device__ __forceinline__ int tile_col(int wn, int lane, int j, int r) {
  return wn * Cfg::WTN + j * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
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
  for (int i = 0; i < Cfg::TM; ++i) {
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(slab + (lane & 31) * Cfg::SLAB + j * 32 + q * 8 + (lane >> 5) * 4) =
            make_float4(static_cast<float>(acc[i][j][4 * q]), static_cast<float>(acc[i][j][4 * q + 1]),
                        static_cast<float>(acc[i][j][4 * q + 2]), static_cast<float>(acc[i][j][4 * q + 3]));
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

// Tile (tm, tn) of index pid: groups of 8 tile rows walked column by column,
// so that neighbouring pids share operand panels.
__device__ __forceinline__ void tile_place(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 8;
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
