// int8 product with one scale per token and output: z[t][c] = xs[t] ws[c]
// sum_k xq[t][k] wt[c][k], exact int32 sums on the matrix cores, the scales
// in the epilogue.
//
// Many tokens are bound by the matrix cores and by the LDS that feeds them
// (tile_gemm.hpp): T = 8192, m = 4096, n = 14336 in 390 us, 2.47 POP/s, where the
// library's plain product reaches 2.1 to 2.3. In between, the K loop of a tile
// is a chain of latencies that no other workgroup shares (T = 777, m = 2064, n =
// 5136: 22 us, 147 tiles of 128 x 256 on 256 CUs; 192 x 128 would take 20 us there
// and lose at every other of 14 sizes tried; T = 96, m = 13824, n = 5120: 32 us for
// 14 us of bytes). Few tokens are bound by the n m bytes of the weight
// (k_linear_i8_few: T = 1, m = 4096, n = 14336 11 us, 5.3 TB/s, with the weight in
// the last-level cache, and 14.3 us, 4.1 TB/s, from memory).
#include "model_kernels.hpp"
#include "tile_gemm.hpp"

namespace poetx {
namespace {

struct I8Args {
  TileOperand x, w;
  const float* xs;
  const float* ws;
  void* z;
  int64_t ldz;
  int T, n, m;
};

template <class Cfg, typename O>
__global__ void __launch_bounds__(Cfg::NT, 1) k_linear_i8(const I8Args a, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) char smem[Cfg::LDS];
  int tm, tn;
  tile_place(xcd_remap(blockIdx.x, gridDim.x), tiles_m, tiles_n, tm, tn);
  const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
  i32x4_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(a.x, a.w, m0, n0, 0, (a.m + Cfg::BK - 1) / Cfg::BK, smem, acc);
  O* z = static_cast<O*>(a.z);
  tile_rows<Cfg>(acc, smem, [&](int row, int col, const float(&v)[8]) {
    const int t = m0 + row, c = n0 + col;
    if (t >= a.T || c >= a.n) return;
    const float s = a.xs[t];
    const float4 w0 = *reinterpret_cast<const float4*>(a.ws + c), w1 = *reinterpret_cast<const float4*>(a.ws + c + 4);
    const float o[8] = {v[0] * s * w0.x, v[1] * s * w0.y, v[2] * s * w0.z, v[3] * s * w0.w,
                        v[4] * s * w1.x, v[5] * s * w1.y, v[6] * s * w1.z, v[7] * s * w1.w};
    tile_store8(z + t * a.ldz + c, o);
  });
}

template <class Cfg>
void launch(const I8Args& a, bool bf16, hipStream_t st) {
  const int tm = (a.T + Cfg::BM - 1) / Cfg::BM, tn = (a.n + Cfg::BN - 1) / Cfg::BN;
  if (bf16) hipLaunchKernelGGL((k_linear_i8<Cfg, bf16_t>), dim3(tm * tn), dim3(Cfg::NT), 0, st, a, tm, tn);
  else hipLaunchKernelGGL((k_linear_i8<Cfg, float>), dim3(tm * tn), dim3(Cfg::NT), 0, st, a, tm, tn);
}

template <int BM, int BN, int WM, int WN, int NS, int KG>
void launch_tail(const I8Args& a, bool bf16, hipStream_t st) {
  if (a.m % 128) launch<TileCfg<1, BM, BN, WM, WN, NS, true, true, true, KG>>(a, bf16, st);
  else launch<TileCfg<1, BM, BN, WM, WN, NS, true, true, false, KG>>(a, bf16, st);
}

// Up to 32 TT tokens: a workgroup computes 32 OB outputs, its NW waves taking
// 128-byte pieces of K in turn (a row's next NW pieces are read at the same
// time). Bound by the weight's bytes, which are read once (58.9 MB with the codes
// at T = 1, 4096 x 14336, for 58.7 of weight). A wave streams its
// pieces of weights and codes through an LDS ring of its own, D pieces deep, with
// direct loads of whole 128-byte lines, and waits for nothing but its own loads:
// no barrier until the waves' sums are joined.
template <int OB, int TT, int NW, int D>
struct FewCfg {
  static constexpr int L = 4 * (OB + TT);           // 1 KB loads of a piece
  static constexpr int PIECE = L * 1024;
  static constexpr int RING = NW * D * PIECE;
  static constexpr int SUMS = NW * TT * 32 * (32 * OB + 4) * 4;
  static constexpr int LDS = RING > SUMS ? RING : SUMS;
  static_assert(LDS <= 160 * 1024 && (D - 1) * L <= 63, "ring");
};

// Waits until no more than the last k pieces' loads (of L each, k up to K, the
// same for a whole wave) are in flight.
template <int L, int K>
__device__ __forceinline__ void wait_pieces(int k) {
  if constexpr (K > 0) {
    if (k < K) {
      wait_pieces<L, K - 1>(k);
      return;
    }
  }
  tg_wait_vm<K * L>();
}

template <int OB, int TT, int NW, int D, typename O>
__global__ void __launch_bounds__(64 * NW) k_linear_i8_few(const I8Args a) {
  using C = FewCfg<OB, TT, NW, D>;
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 32 * OB;
  char* ring = smem + wave * D * C::PIECE;

  TileLoader<32 * OB, 4 * OB, true, 1, true, 32> lw;
  TileLoader<32 * TT, 4 * TT, true, 1, true, 32> lx;
  lw.init(a.w, n0, 0, 0, lane);
  lx.init(a.x, 0, 0, 0, lane);
  const int pieces = (a.m + 127) / 128;
  // none past the last piece, where a row's bytes would run on into the next row
  auto load = [&](int p, char* to) {
    if (p >= pieces) return;
#pragma unroll
    for (int i = 0; i < 4 * OB; ++i) lw.load(i, p, to, 0);
#pragma unroll
    for (int i = 0; i < 4 * TT; ++i) lx.load(i, p, to + 4096 * OB, 0);
  };

  i32x16_t acc[TT][OB];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int o = 0; o < OB; ++o)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[t][o][i] = 0;
  const int r = lane & 31, half = lane >> 5;
  const int sw = chunk_swizzle<32>(r);

#pragma unroll
  for (int s = 0; s < D - 1; ++s) load(wave + s * NW, ring + s * C::PIECE);
  int cur = 0;
  for (int p = wave; p < pieces; p += NW) {
    // the slot read in the last turn is free once its reads are done
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    load(p + (D - 1) * NW, ring + (cur == 0 ? D - 1 : cur - 1) * C::PIECE);
    wait_pieces<C::L, D - 1>((pieces - 1 - p) / NW);
    const char* st = ring + cur * C::PIECE;
    cur = cur == D - 1 ? 0 : cur + 1;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int off = r * 128 + (((2 * kk + half) ^ sw) << 4);
      i32x4_t wf[OB], xf[TT];
#pragma unroll
      for (int o = 0; o < OB; ++o) wf[o] = *reinterpret_cast<const i32x4_t*>(st + o * 4096 + off);
#pragma unroll
      for (int t = 0; t < TT; ++t) xf[t] = *reinterpret_cast<const i32x4_t*>(st + (OB + t) * 4096 + off);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int o = 0; o < OB; ++o)
          acc[t][o] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[o], xf[t], acc[t][o], 0, 0, 0);
    }
  }
  tg_wait_vm<0>();
  __syncthreads();

  // sums [wave][token][output]
  constexpr int ROW = 32 * OB + 4;
  int* part = reinterpret_cast<int*>(smem);
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int o = 0; o < OB; ++o)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<i32x4_t*>(part + ((wave * TT + t) * 32 + r) * ROW + o * 32 + q * 8 + half * 4) =
            i32x4_t{acc[t][o][4 * q], acc[t][o][4 * q + 1], acc[t][o][4 * q + 2], acc[t][o][4 * q + 3]};
  __syncthreads();
  O* z = static_cast<O*>(a.z);
  for (int e = threadIdx.x; e < min(a.T, 32 * TT) * 32 * OB; e += 64 * NW) {
    const int t = e / (32 * OB), c = e % (32 * OB);
    if (n0 + c >= a.n) continue;
    int s = 0;
#pragma unroll
    for (int v = 0; v < NW; ++v) s += part[(v * TT * 32 + t) * ROW + c];
    store_from_f32(z + t * a.ldz + n0 + c, static_cast<float>(s) * a.xs[t] * a.ws[n0 + c]);
  }
}

template <int OB, int TT, int NW, int D>
void launch_few(const I8Args& a, bool bf16, hipStream_t st) {
  const dim3 grid((a.n + 32 * OB - 1) / (32 * OB));
  if (bf16) hipLaunchKernelGGL((k_linear_i8_few<OB, TT, NW, D, bf16_t>), grid, dim3(64 * NW), 0, st, a);
  else hipLaunchKernelGGL((k_linear_i8_few<OB, TT, NW, D, float>), grid, dim3(64 * NW), 0, st, a);
}

}  // namespace

bool linear_i8(const LinearI8Desc& d, hipStream_t st) {
  const I8Args a{{d.xq, d.m, d.T, d.m}, {d.wt, d.m, d.n, d.m}, d.xs, d.ws, d.z, d.ldz,
                 static_cast<int>(d.T), static_cast<int>(d.n), static_cast<int>(d.m)};
  // Few tokens: one ring a wave. 64 outputs a workgroup where 32 would make
  // more than one round over the 256 CUs (64 outputs against 32 at T = 1, weight in
  // the cache: m = 4096, n = 14336 11.1 us, 14.3; m = 13824, n = 5120 14.8, 12.4; not
  // in the cache: 14.4, 14.6; 22.8, 15.6). 33 to 64 tokens with that many outputs go
  // to the tiles (T = 64, tiles against rings, same shapes: in the cache 13.2 us, 19.3;
  // 26.4, 18.8; not in it 16.5, 21.4; 36.7, 27.7).
  if (a.T <= 32) {
    if (a.n > 256 * 32) launch_few<2, 1, 4, 2>(a, d.out_bf16, st);
    else launch_few<1, 1, 4, 4>(a, d.out_bf16, st);
    return true;
  }
  if (a.T <= 64 && a.n <= 256 * 32) {
    launch_few<1, 2, 4, 3>(a, d.out_bf16, st);
    return true;
  }
  const int tile = pick_tile(kTileCosts, kTileKinds, a.T, a.n);
  if (!tiles_fit(kTileCosts[tile], a.T, a.n)) return false;
  switch (tile) {
    case kTile64x2: launch_tail<64, 64, 2, 2, 3, 2>(a, d.out_bf16, st); break;
    case kTile64: launch_tail<64, 64, 2, 2, 4, 1>(a, d.out_bf16, st); break;
    case kTile128: launch_tail<128, 128, 2, 4, 4, 1>(a, d.out_bf16, st); break;
    case kTile128x256: launch_tail<128, 256, 2, 4, 3, 1>(a, d.out_bf16, st); break;
    case kTile192x256: launch_tail<192, 256, 2, 4, 2, 1>(a, d.out_bf16, st); break;
    default: launch_tail<256, 256, 2, 4, 2, 1>(a, d.out_bf16, st); break;
  }
  return true;
}

}  // namespace poetx
