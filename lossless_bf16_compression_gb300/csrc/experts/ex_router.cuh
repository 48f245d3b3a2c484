// ex_router.cuh -- what the router's kernels share: rows in registers, sums over them, scores; and their launchers.
//
// A token's row of logits lies in the registers of W neighbouring lanes, N to a lane, so a warp works on 32 / W tokens at
// a time: with few experts, a warp for each token would spend its instructions on lanes that hold nothing (32768 x 64 with
// eight chosen: 16.4 us by whole warps, 8.0 by eight lanes each, at the time).
#pragma once

#include <type_traits>

#include "ex_common.cuh"
#include "zc_router.h"

namespace zc {
namespace ex {

struct RouterShape {
  size_t tokens;
  int experts, k, type, score, normalize;
  float scale;
};

cudaError_t launch_route(const RouterShape& s, const void* logits, size_t pitch, float* weights, int* ids,
                         cudaStream_t stream);
cudaError_t launch_route_grad(const RouterShape& s, const float* d_weights, const int* ids, const float* d_loss,
                              const float* slope, const void* logits, size_t pitch, void* d_logits, size_t d_pitch,
                              const DeviceInfo& dev, cudaStream_t stream);
size_t balance_workspace(size_t tokens, int experts);
cudaError_t launch_balance(const RouterShape& s, const void* logits, size_t pitch, const int* ids, float* loss, int* counts,
                           float* slope, void* workspace, cudaStream_t stream);

// ------------------------------------------------------------------ rows in registers

constexpr float kInf = __builtin_inff();

template <int B>
struct Word;
template <>
struct Word<2> { using type = unsigned short; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };

template <typename T>
__device__ __forceinline__ T lowest();
template <>
__device__ __forceinline__ __nv_bfloat16 lowest() { return __ushort_as_bfloat16(0xFF80); }
template <>
__device__ __forceinline__ __half lowest() { return __ushort_as_half(0xFC00); }
template <>
__device__ __forceinline__ float lowest() { return -kInf; }

// Up to N W values, V neighbours to a lane and N / V times W V values, the V by one load where every row starts and ends on
// a whole vector of them (Whole).  Which lane holds what does not depend on that, so results do not either.
template <typename T_, int N_, int W_, bool Whole_>
struct Row {
  using T = T_;
  static constexpr int N = N_, W = W_;
  static constexpr bool Whole = Whole_;
  static constexpr int V = N * sizeof(T) <= 16 ? N : 16 / sizeof(T);
  using Vector = typename Word<V * sizeof(T)>::type;
  T v[N];

  __device__ __forceinline__ static int lane() { return threadIdx.x % W; }
  __device__ __forceinline__ static int column(int i) { return (i / V * W + lane()) * V + i % V; }
  // Values past the row's end are -infinity.
  __device__ __forceinline__ void load(const T* row, int experts) {
    union {
      Vector w;
      T v[V];
    } u;
#pragma unroll
    for (int i = 0; i < N; i += V) {
#pragma unroll
      for (int j = 0; j < V; ++j) u.v[j] = lowest<T>();
      if (Whole) {
        if (column(i) < experts) u.w = *reinterpret_cast<const Vector*>(row + column(i));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (column(i + j) < experts) u.v[j] = row[column(i + j)];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[i + j] = u.v[j];
    }
  }
  __device__ __forceinline__ void store(T* row, int experts) const {
    union {
      Vector w;
      T v[V];
    } u;
#pragma unroll
    for (int i = 0; i < N; i += V) {
#pragma unroll
      for (int j = 0; j < V; ++j) u.v[j] = v[i + j];
      if (Whole) {
        if (column(i) < experts) *reinterpret_cast<Vector*>(row + column(i)) = u.w;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (column(i + j) < experts) row[column(i + j)] = v[i + j];
      }
    }
  }
};

// ------------------------------------------------------------------ over a token's lanes

template <int W>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = W / 2; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  return v;
}
// The sum over the first `n` lanes, in all of those (lanes behind hold 0, or have no use for it).
template <int W>
__device__ __forceinline__ float slots_sum(float v, int n) {
#pragma unroll
  for (int d = 1; d < W; d *= 2) {
    if (d >= n) break;
    v += __shfl_xor_sync(~0u, v, d);
  }
  return v;
}
// The larger value; NaN if there is one.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int W>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (W == 32) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int d = W / 2; d > 0; d /= 2) v = larger(v, __shfl_xor_sync(~0u, v, d));
    return v;
  }
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  if constexpr (W == 32) {
    return __reduce_max_sync(~0u, v);
  } else {
#pragma unroll
    for (int d = W / 2; d > 0; d /= 2) v = max(v, __shfl_xor_sync(~0u, v, d));
    return v;
  }
}
template <int W>
__device__ __forceinline__ int row_min(int v) {
  if constexpr (W == 32) {
    return __reduce_min_sync(~0u, v);
  } else {
#pragma unroll
    for (int d = W / 2; d > 0; d /= 2) v = min(v, __shfl_xor_sync(~0u, v, d));
    return v;
  }
}

// ------------------------------------------------------------------ scores

// A sigmoid and one less it, from one exponential of a negative number.
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid(float x) {
  const float z = expf(-fabsf(x)), r = __fdividef(1.0f, 1.0f + z);
  return x > 0 ? Sigmoid{r, z * r} : Sigmoid{z * r, r};
}
// sigmoid(x) e^-m, m the smaller of 0 and the row's largest logit: a row of very low logits does not vanish before it is
// divided by its sum.
__device__ __forceinline__ Sigmoid scaled_sigmoid(float x, float m) {
  Sigmoid v = sigmoid(x);
  if (m < 0) v.s = expf(x - m) * v.rest;
  return v;
}

// ------------------------------------------------------------------ which instance

// f(row type) for rows of `experts` values at these places; `narrow`: tokens may share a warp.
template <typename F>
cudaError_t by_row(int type, int experts, bool narrow, std::initializer_list<const void*> bases,
                   std::initializer_list<size_t> pitches, F f) {
  const auto go = [&](auto t, auto n, auto w) {
    using T = decltype(t);
    constexpr int N = decltype(n)::value, W = decltype(w)::value;
    uintptr_t all = experts * sizeof(T);
    for (const void* b : bases) all |= reinterpret_cast<uintptr_t>(b);
    for (size_t p : pitches) all |= p * sizeof(T);
    if (all % (Row<T, N, W, true>::V * sizeof(T)) == 0) return f(Row<T, N, W, true>());
    return f(Row<T, N, W, false>());
  };
  const auto shape = [&](auto t) {
    constexpr std::integral_constant<int, 8> eight;
    if (narrow && experts <= 32) return go(t, eight, std::integral_constant<int, 4>());
    if (narrow && experts <= 64) return go(t, eight, std::integral_constant<int, 8>());
    if (narrow && experts <= 128) return go(t, eight, std::integral_constant<int, 16>());
    if (experts <= 256) return go(t, eight, std::integral_constant<int, 32>());
    return go(t, std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
  };
  if (type == ZC_TYPE_BF16) return shape(__nv_bfloat16());
  if (type == ZC_TYPE_FP16) return shape(__half());
  return shape(0.0f);
}
// Lanes of a token for so many experts.
inline int lanes_of(int experts) { return experts <= 32 ? 4 : experts <= 64 ? 8 : experts <= 128 ? 16 : 32; }

}  // namespace ex
}  // namespace zc
