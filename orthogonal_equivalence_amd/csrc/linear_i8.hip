// int8 product with one scale per token and output: z[t][c] = xs[t] ws[c]
// sum_k xq[t][k] wt[c][k], exact int32 sums on v_mfma_i32_32x32x32_i8, the
// scales in the epilogue.
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
  i32x16_t acc[Cfg::TM][Cfg::TN];
  tile_product<Cfg>(a.x, a.w, m0, n0, a.m, 0, (a.m + Cfg::BK - 1) / Cfg::BK, smem, acc);
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

}  // namespace

size_t linear_i8_part_bytes(int64_t, int64_t, int64_t) { return 0; }

void linear_i8(const LinearI8Desc& d, hipStream_t st) {
  const I8Args a{{d.xq, d.m, d.T, d.m}, {d.wt, d.m, d.n, d.m}, d.xs, d.ws, d.z, d.ldz,
                 static_cast<int>(d.T), static_cast<int>(d.n), static_cast<int>(d.m)};
  if (d.m % 128) launch<TileCfg<1, 256, 256, 2, 4, true, true, true>>(a, d.out_bf16, st);
  else launch<TileCfg<1, 256, 256, 2, 4, true, true, false>>(a, d.out_bf16, st);
}

}  // namespace poetx
