// The norm of all gradients of a model together, and their scaling by it:
//
//   norm = sqrt(sum over the tensors of x^2),  out = x min(1, max_norm / (norm + 1e-6))
//
// One pass of sums, one of scaling, both bound by memory. The tensors are cut
// into units of 16 KB, and each workgroup walks a run of consecutive units,
// across tensors, so that few large and many small ones take the same kernel.
// Squares and sums are in double: no float32 or bfloat16 value overflows or
// vanishes, and a billion of them lose nothing. Every workgroup leaves one sum;
// they are added in a fixed order, without atomics.
//
// Pointers and sizes reach the device in launch arguments: those of up to kArgs
// tensors in the sums' own, which leaves them in the workspace for the scaling, those
// of more by launches of their own before it, so that the sums are one launch.
#include "common.hpp"
#include "model_kernels.hpp"

#include <algorithm>

namespace poetx {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kArgs = 120;      // tensors of a launch: 4 KB of arguments
// Workgroups, each with a sum of its own (2.4 GB in 514 tensors, sums and scaling:
// 512 1.48 ms, 1024 1.36, 2048 1.40).
constexpr int kBlocks = 1024;

struct GradArgs {
  int count;   // tensors of this launch
  int first;   // the first of them
  GradEntry e[kArgs];
};

__device__ __forceinline__ int unit_values(const GradEntry& e) { return e.bf16 ? kGradUnit / 2 : kGradUnit / 4; }

// last tensor whose first unit is at or before u
__device__ __forceinline__ int entry_of(const GradEntry* e, int count, uint32_t u) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (e[mid].first <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum of v over the workgroup, in every thread.
__device__ __forceinline__ double sum_workgroup(double v, double* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v += red[w];
  return v;
}

__device__ __forceinline__ double square(float x) {
  const double d = x;
  return d * d;
}
__device__ __forceinline__ double squares(uint4 v, bool bf16) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  double s = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s += bf16 ? square(__uint_as_float(x[i] << 16)) + square(__uint_as_float(x[i] & 0xffff0000u))
              : square(__uint_as_float(x[i]));
  return s;
}

// Values [lo, hi) of a tensor: 16 bytes at a time where they are aligned, value by
// value before and behind; with BACK the former from the last to the first.
template <bool BACK, class V16, class V1>
__device__ __forceinline__ void walk(const void* p, int es, int64_t lo, int64_t hi, V16&& wide, V1&& one) {
  const int64_t per = 16 / es;
  const int64_t off = (16 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15)) % 16 / es;  // of the first aligned value
  const int64_t a = min(hi, off + (lo - off + per - 1 + per) / per * per - per), b = a + (hi - a) / per * per;
  for (int64_t i = lo + threadIdx.x; i < a; i += kThreads) one(i);
  if constexpr (BACK) {
#pragma unroll 4
    for (int64_t i = b - (threadIdx.x + 1) * per; i >= a; i -= kThreads * per) wide(i);
  } else {
#pragma unroll 4
    for (int64_t i = a + threadIdx.x * per; i < b; i += kThreads * per) wide(i);
  }
  for (int64_t i = b + threadIdx.x; i < hi; i += kThreads) one(i);
}

__device__ __forceinline__ void store_table(const GradArgs& a, GradEntry* table) {
  for (int i = threadIdx.x; i < a.count; i += kThreads) table[a.first + i] = a.e[i];
}
__global__ void __launch_bounds__(kThreads) k_grad_table(const GradArgs a, GradEntry* table) { store_table(a, table); }

// This workgroup's share of the units, f(entry, lo, hi) for its part of every
// tensor; with BACK from the last one to the first.
template <bool BACK, class F>
__device__ __forceinline__ void walk_share(const GradEntry* e, int count, uint32_t units, F&& f) {
  const uint32_t u0 = static_cast<uint32_t>(static_cast<uint64_t>(units) * blockIdx.x / gridDim.x);
  const uint32_t u1 = static_cast<uint32_t>(static_cast<uint64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  for (int k = entry_of(e, count, BACK ? u1 - 1 : u0);; k += BACK ? -1 : 1) {
    const GradEntry x = e[k];
    const uint32_t from = max(u0, x.first), to = k + 1 < count ? min(u1, e[k + 1].first) : u1;
    const int64_t per = unit_values(x);
    f(x, static_cast<int64_t>(from - x.first) * per, min(x.n, static_cast<int64_t>(to - x.first) * per));
    if (BACK ? x.first <= u0 : to >= u1) return;
  }
}

__device__ __forceinline__ double sum_squares(const GradEntry& e, int64_t lo, int64_t hi) {
  double sum = 0;
  if (e.bf16) {
    const bf16_t* p = static_cast<const bf16_t*>(e.g);
    walk<false>(p, 2, lo, hi, [&](int64_t i) { sum += squares(*reinterpret_cast<const uint4*>(p + i), true); },
                [&](int64_t i) { sum += square(bf16_to_f32(p[i])); });
  } else {
    const float* p = static_cast<const float*>(e.g);
    walk<false>(p, 4, lo, hi, [&](int64_t i) { sum += squares(*reinterpret_cast<const uint4*>(p + i), false); },
                [&](int64_t i) { sum += square(p[i]); });
  }
  return sum;
}

// The workgroups' sums, of the tensors in the arguments (and then in the table), or
// of those in the table.
template <bool ARGS>
__global__ void __launch_bounds__(kThreads) k_grad_sums(const GradArgs a, GradEntry* table, int count, uint32_t units,
                                                        double* part) {
  __shared__ double red[kThreads / 64];
  if (ARGS && blockIdx.x == 0) store_table(a, table);
  double sum = 0;
  walk_share<false>(ARGS ? a.e : table, count, units,
                    [&](const GradEntry& e, int64_t lo, int64_t hi) { sum += sum_squares(e, lo, hi); });
  sum = sum_workgroup(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double sum_parts(const double* part, int parts, double* red) {
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return sum_workgroup(s, red);
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const double* part, int parts, float* norm) {
  __shared__ double red[kThreads / 64];
  const double s = sum_parts(part, parts, red);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <class T>
__device__ __forceinline__ void scale_values(const GradEntry& e, int64_t lo, int64_t hi, float first, float f) {
  const T* g = static_cast<const T*>(e.g);
  T* out = static_cast<T*>(e.out);
  constexpr int es = sizeof(T);
  if ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(out)) & 15) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) store_from_f32(out + i, load_as_f32(g + i) * first * f);
    return;
  }
  walk<true>(g, es, lo, hi,
       [&](int64_t i) {
         uint4 v = *reinterpret_cast<const uint4*>(g + i);
         uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
         for (int j = 0; j < 4; ++j)
           x[j] = es == 2 ? pack_bf16x2(__uint_as_float(x[j] << 16) * first * f, __uint_as_float(x[j] & 0xffff0000u) * first * f)
                          : __float_as_uint(__uint_as_float(x[j]) * first * f);
         const u32x4_t y = {x[0], x[1], x[2], x[3]};
         __builtin_nontemporal_store(y, reinterpret_cast<u32x4_t*>(out + i));
       },
       [&](int64_t i) { store_from_f32(out + i, load_as_f32(g + i) * first * f); });
}

// The norm and the scaled values. Each workgroup takes the share that it took of
// the sums, from the end, as what was read last may still lie in the last-level
// cache, and stores past that cache (sums and scaling of 2.4 and 0.41 GB: 1.36 ms and
// 232 us; from the front 1.39 and 269; through the cache 1.39 and 252).
__global__ void __launch_bounds__(kThreads) k_grad_scale(const GradEntry* table, int count, uint32_t units,
                                                         const double* part, double max_norm, float* norm) {
  __shared__ double red[kThreads / 64];
  const double size = sqrt(sum_parts(part, gridDim.x, red)), q = max_norm / (size + 1e-6);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(size);
  // a factor below float's normal numbers in two, of which the first takes no bits of values
  // whose products are normal
  const float first = q < 0x1p-126 ? 0x1p-126f : 1.f;
  const float f = q > 1.0 ? 1.f : static_cast<float>(q / first);  // NaN stays
  walk_share<true>(table, count, units, [&](const GradEntry& e, int64_t lo, int64_t hi) {
    if (f == 1.f && e.out == e.g) return;
    if (e.bf16) scale_values<bf16_t>(e, lo, hi, first, f);
    else scale_values<float>(e, lo, hi, first, f);
  });
}

}  // namespace

int64_t grad_parts(int64_t count) { return count ? kBlocks : 0; }

void grad_norm(const GradDesc& d, hipStream_t st) {
  const int count = static_cast<int>(d.count);
  uint32_t units = 0;
  GradArgs a{};
  for (int i = 0; i < count; ++i) {
    if (a.count == kArgs) {
      hipLaunchKernelGGL(k_grad_table, dim3(1), dim3(kThreads), 0, st, a, d.table);
      a.first = i;
      a.count = 0;
    }
    a.e[a.count++] = {d.g[i], d.out ? d.out[i] : nullptr, d.n[i], units, d.bf16(i)};
    units += static_cast<uint32_t>(grad_units(d.n[i], d.bf16(i)));
  }
  const unsigned blocks = std::min<uint32_t>(std::max(units, 1u), kBlocks);
  if (count > kArgs) {
    hipLaunchKernelGGL(k_grad_table, dim3(1), dim3(kThreads), 0, st, a, d.table);
    hipLaunchKernelGGL((k_grad_sums<false>), dim3(blocks), dim3(kThreads), 0, st, GradArgs{}, d.table, count, units, d.part);
  } else if (count > 0) {
    hipLaunchKernelGGL((k_grad_sums<true>), dim3(blocks), dim3(kThreads), 0, st, a, d.table, count, units, d.part);
  }
  if (d.out)
    hipLaunchKernelGGL(k_grad_scale, dim3(blocks), dim3(kThreads), 0, st, d.table, count, units, d.part,
                       static_cast<double>(d.max_norm), d.norm);
  else
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(kThreads), 0, st, d.part, static_cast<int>(count ? blocks : 0), d.norm);
}

}  // namespace poetx
