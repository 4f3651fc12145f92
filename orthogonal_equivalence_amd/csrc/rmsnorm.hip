// RMS norm of the residual stream: s = x + res, y = s * rstd * gain with
// rstd = 1 / sqrt(mean(s^2) + eps), y in the activation type or as int8 rows
// with one scale per token; and its backward.
//
// All of it is bound by HBM: a row is read once, held in registers as float
// across its reductions and written once. A row belongs to TPR threads (from 8
// to sixteen waves), each with CH chunks of 8 consecutive features, 16 bytes of
// bfloat16 a load; rows too wide for that are read again per pass. (The backward of
// rows of 8200 to 24576 features needs more than its 128 registers a thread: 25 to 379
// lie in scratch memory, and T = 4096, n = 13824 takes 216 us for 89 us of bytes.)
// Measured in
// bfloat16 with the residual (a large copy reaches 5.1 TB/s, more where the
// last-level cache holds the data): T = 8192, n = 4096 forward 41 us (6.5
// TB/s), int8 rows 39 us, backward 42 us and 5 us for dgain; T = 4096, n =
// 5120 forward 31 us, backward 31 us; one row of 4096 3.5 us.
#include "common.hpp"
#include "model_kernels.hpp"

namespace poetx {
namespace {

constexpr float kTinyRow = 0x1p-100f;  // rows below this count as zero when quantised

// 8 features as they lie in memory
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void widen(const Raw8<bf16_t>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  widen(load_raw(p), v);
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// int8 code of v / scale: ties to even, NaN to 0.
__device__ __forceinline__ uint32_t code8(float v, float inv) {
  const float r = fminf(fmaxf(rintf(v * inv), -127.f), 127.f);
  return static_cast<uint32_t>(v * inv == v * inv ? static_cast<int>(r) : 0) & 0xffu;
}
__device__ __forceinline__ void store_codes8(int8_t* p, const float (&v)[8], float inv) {
  uint2 w = make_uint2(0u, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w.x |= code8(v[i], inv) << (8 * i);
    w.y |= code8(v[4 + i], inv) << (8 * i);
  }
  *reinterpret_cast<uint2*>(p) = w;
}

// Sum / maximum of one value per thread over the TPR threads of a row. The
// maximum is taken on the bits of |v|, where NaN is larger than infinity and
// therefore stays. `red`: two words a wave and call, in turn (`turn` counts
// the calls), so that one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int& turn) {
  static_assert(TPR <= 64 || TPR >= 256, "a row over several waves has the workgroup to itself");
#pragma unroll
  for (int o = TPR < 64 ? TPR / 2 : 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* r = red[turn & 1];
    ++turn;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += r[i];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ float row_absmax(float v, float (*red)[16], int& turn) {
  uint32_t m = __float_as_uint(v);
#pragma unroll
  for (int o = TPR < 64 ? TPR / 2 : 32; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o)));
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* r = red[turn & 1];
    ++turn;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = __uint_as_float(m);
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, __float_as_uint(r[i]));
  }
  return __uint_as_float(m);
}
__device__ __forceinline__ float absmax_bits(float m, float v) {
  return __uint_as_float(max(__float_as_uint(m), __float_as_uint(v) & 0x7fffffffu));
}

// scale and its inverse of a row with largest magnitude a
__device__ __forceinline__ void row_scale(float a, float& scale, float& inv) {
  const bool zero = a < kTinyRow;  // false for NaN
  scale = zero ? 1.f : a / 127.f;
  inv = zero ? 0.f : 127.f / a;
}

template <typename T>
struct NormArgs {
  const T* x;
  int64_t ldx;
  const T* res;
  int64_t ldr;
  const float* gain;
  float eps;
  T* h;
  T* y;
  float* rstd;
  int8_t* q;
  float* scale;
  int64_t T_;
  int64_t n;
};

// NORM: the norm (else the rows are only quantised); Q8: int8 rows out.
// CH > 0: CH chunks a thread in registers. CH = 0: any width, the row read
// once per pass (each element is read and written by one thread, so h may
// still be x or res).
template <typename T, int TPR, int CH, bool NORM, bool Q8>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_norm_fwd(const NormArgs<T> a) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;  // rows of a workgroup
  __shared__ float red[2][16];
  int turn = 0;
  const int t = threadIdx.x % TPR;
  const int64_t row = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * RPW + threadIdx.x / TPR;
  if (row >= a.T_) return;  // a row's threads together; a row over several waves has the workgroup to itself
  const T* x = a.x + row * a.ldx;
  const T* r = a.res ? a.res + row * a.ldr : nullptr;
  const int chunks = static_cast<int>(a.n / 8);

  if constexpr (CH > 0) {
    // all loads of the row at once, the gains too where they fit beside it
    constexpr bool kGainEarly = NORM && CH <= 3;
    Raw8<T> rx[CH], rr[CH];
    float s[CH][8], ge[kGainEarly ? CH : 1][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = c * TPR + t;
      if (k < chunks) {
        rx[c] = load_raw(x + static_cast<int64_t>(k) * 8);
        if (r) rr[c] = load_raw(r + static_cast<int64_t>(k) * 8);
        if constexpr (kGainEarly) load8(a.gain + static_cast<int64_t>(k) * 8, ge[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (c * TPR + t < chunks) {
        widen(rx[c], s[c]);
        if (r) {
          float u[8];
          widen(rr[c], u);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[c][i] += u[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[c][i] = 0.f;
      }
    }
    if constexpr (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += s[c][i] * s[c][i];
      ss = row_sum<TPR>(ss, red, turn);
      const float rs = 1.f / sqrtf(ss / static_cast<float>(a.n) + a.eps);
      if (a.rstd && t == 0) a.rstd[row] = rs;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = c * TPR + t;
        if (k < chunks) {
          if (a.h) store8(a.h + row * a.n + static_cast<int64_t>(k) * 8, s[c]);
          float g[8];
          if constexpr (kGainEarly) {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = ge[c][i];
          } else {
            load8(a.gain + static_cast<int64_t>(k) * 8, g);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s[c][i] = s[c][i] * rs * g[i];
          if constexpr (!Q8) store8(a.y + row * a.n + static_cast<int64_t>(k) * 8, s[c]);
        }
      }
    }
    if constexpr (Q8) {
      float m = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = absmax_bits(m, s[c][i]);
      float scale, inv;
      row_scale(row_absmax<TPR>(m, red, turn), scale, inv);
      if (t == 0) a.scale[row] = scale;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = c * TPR + t;
        if (k < chunks) store_codes8(a.q + row * a.n + static_cast<int64_t>(k) * 8, s[c], inv);
      }
    }
  } else {
    auto sum8 = [&](int k, float (&s)[8]) {
      load8(x + static_cast<int64_t>(k) * 8, s);
      if (r) {
        float u[8];
        load8(r + static_cast<int64_t>(k) * 8, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += u[i];
      }
    };
    float rs = 1.f;
    if constexpr (NORM) {
      float ss = 0.f;
      for (int k = t; k < chunks; k += TPR) {
        float s[8];
        sum8(k, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += s[i] * s[i];
      }
      ss = row_sum<TPR>(ss, red, turn);
      rs = 1.f / sqrtf(ss / static_cast<float>(a.n) + a.eps);
      if (a.rstd && t == 0) a.rstd[row] = rs;
    }
    auto norm8 = [&](int k, float (&s)[8]) {
      if constexpr (NORM) {
        float g[8];
        load8(a.gain + static_cast<int64_t>(k) * 8, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = s[i] * rs * g[i];
      }
    };
    float inv = 0.f;
    if constexpr (Q8) {
      float m = 0.f;
      for (int k = t; k < chunks; k += TPR) {
        float s[8];
        sum8(k, s);
        norm8(k, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = absmax_bits(m, s[i]);
      }
      float scale;
      row_scale(row_absmax<TPR>(m, red, turn), scale, inv);
      if (t == 0) a.scale[row] = scale;
    }
    for (int k = t; k < chunks; k += TPR) {
      float s[8];
      sum8(k, s);
      if (NORM && a.h) store8(a.h + row * a.n + static_cast<int64_t>(k) * 8, s);
      norm8(k, s);
      if constexpr (Q8) store_codes8(a.q + row * a.n + static_cast<int64_t>(k) * 8, s, inv);
      else store8(a.y + row * a.n + static_cast<int64_t>(k) * 8, s);
    }
  }
}

template <typename T>
struct NormBwdArgs {
  const T* dy;
  int64_t lddy;
  const T* h;
  const float* rstd;
  const float* gain;
  const T* dh;
  int64_t lddh;
  T* dx;
  float* part;  // [groups][n], or null
  int64_t T_;
  int64_t n;
  int groups;
};

// Rows g, g + groups, ... of row group g; the group's share of dgain stays in
// registers (CH > 0) or in its own row of `part` (CH = 0) until the last row.
template <typename T, int TPR, int CH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_norm_bwd(const NormBwdArgs<T> a) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[2][16];
  int turn = 0;
  const int t = threadIdx.x % TPR;
  const int g = static_cast<int>(blockIdx.x) * RPW + static_cast<int>(threadIdx.x) / TPR;
  if (g >= a.groups) return;
  const int chunks = static_cast<int>(a.n / 8);
  const float inv_n = 1.f / static_cast<float>(a.n);

  if constexpr (CH > 0) {
    float gn[CH][8], acc[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = c * TPR + t;
#pragma unroll
      for (int i = 0; i < 8; ++i) gn[c][i] = acc[c][i] = 0.f;
      if (k < chunks) load8(a.gain + static_cast<int64_t>(k) * 8, gn[c]);
    }
    // the next row's loads are in flight while a row is reduced and written
    Raw8<T> rdy[CH], rh[CH], rdh[CH];
    float rs_next = 0.f;
    auto fetch = [&](int64_t row) {
      if (row >= a.T_) return;
      rs_next = a.rstd[row];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = c * TPR + t;
        if (k < chunks) {
          rdy[c] = load_raw(a.dy + row * a.lddy + static_cast<int64_t>(k) * 8);
          rh[c] = load_raw(a.h + row * a.n + static_cast<int64_t>(k) * 8);
          if (a.dh) rdh[c] = load_raw(a.dh + row * a.lddh + static_cast<int64_t>(k) * 8);
        }
      }
    };
    fetch(g);
    for (int64_t row = g; row < a.T_; row += a.groups) {
      const float rs = rs_next;
      float dy[CH][8], u[CH][8], d[CH][8];
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (c * TPR + t < chunks) {
          widen(rdy[c], dy[c]);
          widen(rh[c], u[c]);
          if (a.dh) widen(rdh[c], d[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dy[c][i] = u[c][i] = 0.f;
        }
      }
      fetch(row + a.groups);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[c][i] *= rs;
          acc[c][i] += dy[c][i] * u[c][i];
          dy[c][i] *= gn[c][i];
          dot += dy[c][i] * u[c][i];
        }
      const float mean = row_sum<TPR>(dot, red, turn) * inv_n;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = c * TPR + t;
        if (k < chunks) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = rs * (dy[c][i] - u[c][i] * mean);
          if (a.dh) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += d[c][i];
          }
          store8(a.dx + row * a.n + static_cast<int64_t>(k) * 8, v);
        }
      }
    }
    if (a.part) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int k = c * TPR + t;
        if (k < chunks) store8(a.part + static_cast<int64_t>(g) * a.n + static_cast<int64_t>(k) * 8, acc[c]);
      }
    }
  } else {
    for (int64_t row = g; row < a.T_; row += a.groups) {
      const float rs = a.rstd[row];
      const T* dyr = a.dy + row * a.lddy;
      const T* hr = a.h + row * a.n;
      float dot = 0.f;
      for (int k = t; k < chunks; k += TPR) {
        float dy[8], u[8], gn[8], acc[8];
        load8(dyr + static_cast<int64_t>(k) * 8, dy);
        load8(hr + static_cast<int64_t>(k) * 8, u);
        load8(a.gain + static_cast<int64_t>(k) * 8, gn);
        float* p = a.part ? a.part + static_cast<int64_t>(g) * a.n + static_cast<int64_t>(k) * 8 : nullptr;
        if (p && row != g) {
          load8(p, acc);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] *= rs;
          acc[i] += dy[i] * u[i];
          dot += dy[i] * gn[i] * u[i];
        }
        if (p) store8(p, acc);
      }
      const float mean = row_sum<TPR>(dot, red, turn) * inv_n;
      for (int k = t; k < chunks; k += TPR) {
        float dy[8], u[8], gn[8], v[8];
        load8(dyr + static_cast<int64_t>(k) * 8, dy);
        load8(hr + static_cast<int64_t>(k) * 8, u);
        load8(a.gain + static_cast<int64_t>(k) * 8, gn);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = rs * (dy[i] * gn[i] - u[i] * rs * mean);
        if (a.dh) {
          float d[8];
          load8(a.dh + row * a.lddh + static_cast<int64_t>(k) * 8, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += d[i];
        }
        store8(a.dx + row * a.n + static_cast<int64_t>(k) * 8, v);
      }
    }
  }
}

// out[j] = sum over the groups, in a fixed order: 32 columns a workgroup, row
// lane r of 32 over groups r, r + 32, .. (16 loads in flight), then a tree over
// the row lanes.
__global__ void __launch_bounds__(1024) k_dgain_sum(const float* part, int groups, int64_t n, float* out) {
  __shared__ float s[32][33];
  const int col = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + col;
  float v = 0.f;
  if (j < n) {
    for (int k = r; k < groups; k += 512) {
      float u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int g = k + i * 32;
        u[i] = g < groups ? part[static_cast<int64_t>(g) * n + j] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) v += u[i];
    }
  }
  s[r][col] = v;
  __syncthreads();
  v = s[col][r];  // row lane `col` of column `r`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor(v, o);
  const int64_t to = static_cast<int64_t>(blockIdx.x) * 32 + r;
  if (col == 0 && to < n) out[to] = v;
}

// n workgroups of up to 1024 threads in two dimensions: the threads of one stay
// below 2^32
dim3 row_grid(int64_t n) {
  constexpr int64_t kMost = int64_t(1) << 21;
  return dim3(static_cast<unsigned>(n < kMost ? n : kMost), static_cast<unsigned>((n + kMost - 1) / kMost));
}

template <typename T, bool NORM, bool Q8>
void launch_fwd(const NormArgs<T>& a, hipStream_t st) {
  const int64_t chunks = a.n / 8;
#define POETX_NORM_FWD(TPR, CH)                                                                          \
  {                                                                                                      \
    constexpr int rpw = TPR < 256 ? 256 / TPR : 1;                                                       \
    hipLaunchKernelGGL((k_norm_fwd<T, TPR, CH, NORM, Q8>), row_grid((a.T_ + rpw - 1) / rpw),              \
                       dim3(TPR < 256 ? 256 : TPR), 0, st, a);                                           \
    return;                                                                                              \
  }
  // Few rows leave CUs idle, so a wide row gets sixteen waves (T = 48, n =
  // 13824 with int8 rows: 12.1 us on four waves).
  const bool few = a.T_ < 512;
  if (chunks <= 8) POETX_NORM_FWD(8, 1)
  if (chunks <= 16) POETX_NORM_FWD(16, 1)
  if (chunks <= 32) POETX_NORM_FWD(32, 1)
  if (chunks <= 64) POETX_NORM_FWD(64, 1)
  if (chunks <= 128) POETX_NORM_FWD(64, 2)
  if (chunks <= 256) POETX_NORM_FWD(256, 1)
  if (chunks <= 512) POETX_NORM_FWD(256, 2)
  if (chunks <= 768 && !few) POETX_NORM_FWD(256, 3)
  if (chunks <= 1024 && !few) POETX_NORM_FWD(256, 4)
  if (chunks <= 1024) POETX_NORM_FWD(1024, 1)
  if (chunks <= 2048) POETX_NORM_FWD(1024, 2)
  if (chunks <= 4096) POETX_NORM_FWD(1024, 4)
  POETX_NORM_FWD(1024, 0)
#undef POETX_NORM_FWD
}

template <typename T>
void launch_bwd(const NormBwdArgs<T>& a, hipStream_t st) {
  const int64_t chunks = a.n / 8;
#define POETX_NORM_BWD(TPR, CH)                                                                    \
  {                                                                                                \
    constexpr int rpw = TPR < 256 ? 256 / TPR : 1;                                                 \
    hipLaunchKernelGGL((k_norm_bwd<T, TPR, CH>), dim3((a.groups + rpw - 1) / rpw), dim3(TPR < 256 ? 256 : TPR), \
                       0, st, a);                                                                  \
    return;                                                                                        \
  }
  if (chunks <= 8) POETX_NORM_BWD(8, 1)
  if (chunks <= 16) POETX_NORM_BWD(16, 1)
  if (chunks <= 32) POETX_NORM_BWD(32, 1)
  if (chunks <= 64) POETX_NORM_BWD(64, 1)
  if (chunks <= 128) POETX_NORM_BWD(64, 2)
  if (chunks <= 256) POETX_NORM_BWD(256, 1)
  if (chunks <= 512) POETX_NORM_BWD(256, 2)
  if (chunks <= 768) POETX_NORM_BWD(256, 3)
  if (chunks <= 1024) POETX_NORM_BWD(512, 2)
  if (chunks <= 2048) POETX_NORM_BWD(1024, 2)
  if (chunks <= 3072) POETX_NORM_BWD(1024, 3)
  POETX_NORM_BWD(1024, 0)
#undef POETX_NORM_BWD
}

}  // namespace

// Enough groups for two workgroups a CU (rows of several waves) or more, with
// at most 8 MB of partial sums up to n = 4096.
int norm_bwd_groups(int64_t T, int64_t n) {
  const int64_t most = n <= 128 ? 8192 : n <= 256 ? 4096 : n <= 1024 ? 2048 : 512;
  return static_cast<int>(T < most ? T : most);
}

void norm_forward(const NormFwdDesc& d, hipStream_t st) {
  auto run = [&](auto tag) {
    using T = decltype(tag);
    const NormArgs<T> a{static_cast<const T*>(d.x), d.ldx, static_cast<const T*>(d.res), d.ldr, d.gain, d.eps,
                        static_cast<T*>(d.h), static_cast<T*>(d.y), d.rstd, d.q, d.scale, d.T, d.n};
    if (!d.gain) launch_fwd<T, false, true>(a, st);
    else if (d.q) launch_fwd<T, true, true>(a, st);
    else launch_fwd<T, true, false>(a, st);
  };
  if (d.bf16) run(bf16_t{});
  else run(float{});
}

void norm_backward(const NormBwdDesc& d, hipStream_t st) {
  const int groups = norm_bwd_groups(d.T, d.n);
  auto run = [&](auto tag) {
    using T = decltype(tag);
    const NormBwdArgs<T> a{static_cast<const T*>(d.dy), d.lddy, static_cast<const T*>(d.h), d.rstd, d.gain,
                           static_cast<const T*>(d.dh), d.lddh, static_cast<T*>(d.dx), d.part, d.T, d.n, groups};
    launch_bwd<T>(a, st);
  };
  if (d.bf16) run(bf16_t{});
  else run(float{});
  if (d.part)
    hipLaunchKernelGGL(k_dgain_sum, dim3(static_cast<unsigned>((d.n + 31) / 32)), dim3(1024), 0, st, d.part, groups, d.n,
                       d.dgain);
}

}  // namespace poetx
