// ex_rows.cu -- rows to their places in the order by expert and back, with weights, and the
// gradients.  The order is a permutation known from the sort, so every kernel here is driven by
// tokens: a token's row is read (or written) once and its k sorted rows once each, which is all
// the traffic there is, and every sum over j runs inside one thread in slot order (no atomics).
// Bound by HBM.
#include <initializer_list>

#include "ex_common.cuh"

namespace zc {
namespace ex {
namespace {

// A slot's row, or -1 when the slot has no expert (or its position is out of range, which sets
// the error and is never used as an address).
__device__ __forceinline__ int row_of(const int* position, size_t s, size_t slots, int kept, int* status) {
  const int p = position[s];
  if (p < 0 || static_cast<size_t>(p) >= slots) {
    set_error(status, ZC_ERR_CORRUPT);
    return -2;
  }
  return p < kept ? p : -1;
}

// rows[position[t, j]] = x[t].  One CTA a token.
template <int B>
__global__ void __launch_bounds__(256) dispatch_kernel(const uint8_t* __restrict__ x, size_t x_pitch,
                                                       uint8_t* __restrict__ rows, size_t rows_pitch, int vecs, int k,
                                                       size_t slots, const int* __restrict__ position,
                                                       const int* __restrict__ total, int* status) {
  using V = typename Bytes<B>::type;
  wait_for_previous();
  const size_t t = blockIdx.x;
  const int kept = *total;
  for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
    const V v = reinterpret_cast<const V*>(x + t * x_pitch)[c];
    for (int j = 0; j < k; ++j) {
      const int p = position[t * k + j];
      if (p < 0 || static_cast<size_t>(p) >= slots) {
        set_error(status, ZC_ERR_CORRUPT);
        continue;
      }
      reinterpret_cast<V*>(rows + p * rows_pitch)[c] = p < kept ? v : V{};
    }
  }
}

// out[t] = sum over j of weights[t, j] rows[position[t, j]].  One CTA a token.
template <typename T, int B>
__global__ void __launch_bounds__(256) combine_kernel(const uint8_t* __restrict__ rows, size_t rows_pitch,
                                                      const float* __restrict__ weights, uint8_t* __restrict__ out,
                                                      size_t out_pitch, int vecs, int k, size_t slots,
                                                      const int* __restrict__ position, const int* __restrict__ total,
                                                      int* status) {
  constexpr int N = B / sizeof(T);
  const size_t t = blockIdx.x;
  const int kept = *total;
  for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
    float acc[N] = {};
    for (int j = 0; j < k; ++j) {
      const int p = row_of(position, t * k + j, slots, kept, status);
      if (p < 0) continue;
      Pack<T, B> v;
      v.raw = reinterpret_cast<const typename Bytes<B>::type*>(rows + p * rows_pitch)[c];
      const float w = weights ? weights[t * k + j] : 1.f;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(w, to_float(v.v[i]), acc[i]);
    }
    Pack<T, B> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_float<T>(acc[i]);
    reinterpret_cast<typename Bytes<B>::type*>(out + t * out_pitch)[c] = o.raw;
  }
}

// d_rows[position[t, j]] = weights[t, j] d_out[t], d_weights[t, j] = <d_out[t], rows[...]>.
// One CTA a token.
template <typename T, int B>
__global__ void __launch_bounds__(256) combine_grad_kernel(
    const uint8_t* __restrict__ d_out, size_t d_out_pitch, const uint8_t* __restrict__ rows, size_t rows_pitch,
    const float* __restrict__ weights, uint8_t* __restrict__ d_rows, size_t d_rows_pitch, float* __restrict__ d_weights,
    int vecs, int k, size_t slots, const int* __restrict__ position, const int* __restrict__ total, int* status) {
  constexpr int N = B / sizeof(T);
  using V = typename Bytes<B>::type;
  __shared__ float sums[8];
  const size_t t = blockIdx.x;
  const int kept = *total;
  for (int j = 0; j < k; ++j) {
    const int p = position[t * k + j];
    const bool ok = p >= 0 && static_cast<size_t>(p) < slots, here = ok && p < kept;
    if (!ok) set_error(status, ZC_ERR_CORRUPT);
    const float w = here ? weights[t * k + j] : 0.f;
    float dot = 0.f;
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
      Pack<T, B> d, r, o;
      d.raw = reinterpret_cast<const V*>(d_out + t * d_out_pitch)[c];
      if (here) r.raw = reinterpret_cast<const V*>(rows + p * rows_pitch)[c];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        o.v[i] = from_float<T>(here ? w * to_float(d.v[i]) : 0.f);
        if (here) dot = fmaf(to_float(d.v[i]), to_float(r.v[i]), dot);
      }
      if (ok) reinterpret_cast<V*>(d_rows + p * d_rows_pitch)[c] = o.raw;
    }
    for (int m = 16; m; m /= 2) dot += __shfl_xor_sync(~0u, dot, m);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float s = 0.f;
      for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) s += sums[i];
      d_weights[t * k + j] = s;
    }
    __syncthreads();
  }
}

template <typename F>
cudaError_t by_type(int type, int bytes, F&& f) {
  using std::integral_constant;
  if (type == ZC_TYPE_FP32)
    return bytes == 16 ? f(float{}, integral_constant<int, 16>{}) : f(float{}, integral_constant<int, 4>{});
  const auto half = [&](auto t) {
    return bytes == 16  ? f(t, integral_constant<int, 16>{})
           : bytes == 4 ? f(t, integral_constant<int, 4>{})
                        : f(t, integral_constant<int, 2>{});
  };
  return type == ZC_TYPE_FP16 ? half(__half{}) : half(__nv_bfloat16{});
}

}  // namespace

cudaError_t launch_dispatch(const RowShape& s, const void* x, size_t x_pitch, void* rows, size_t rows_pitch,
                            const int* position, const int* offsets, int* status, cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {x, rows}, {x_pitch, rows_pitch});
  const auto run = [&](auto kernel) {
    return launch(kernel, static_cast<unsigned>(s.tokens), 256, 0, stream, true, static_cast<const uint8_t*>(x),
                  x_pitch * b, static_cast<uint8_t*>(rows), rows_pitch * b, static_cast<int>(s.hidden * b / v), s.k,
                  s.tokens * s.k, position, offsets + s.experts, status);
  };
  return v == 16 ? run(dispatch_kernel<16>) : v == 4 ? run(dispatch_kernel<4>) : run(dispatch_kernel<2>);
}

cudaError_t launch_combine(const RowShape& s, const void* rows, size_t rows_pitch, const float* weights,
                           const int* position, const int* offsets, void* out, size_t out_pitch, int* status,
                           cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {rows, out}, {rows_pitch, out_pitch});
  return by_type(s.type, v, [&](auto type, auto bytes) {
    return launch(combine_kernel<decltype(type), bytes()>, static_cast<unsigned>(s.tokens), 256, 0, stream, false,
                  static_cast<const uint8_t*>(rows), rows_pitch * b, weights, static_cast<uint8_t*>(out),
                  out_pitch * b, static_cast<int>(s.hidden * b / v), s.k, s.tokens * s.k, position,
                  offsets + s.experts, status);
  });
}

cudaError_t launch_combine_grad(const RowShape& s, const void* d_out, size_t d_out_pitch, const void* rows,
                                size_t rows_pitch, const float* weights, const int* position, const int* offsets,
                                void* d_rows, size_t d_rows_pitch, float* d_weights, int* status,
                                cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {d_out, rows, d_rows}, {d_out_pitch, rows_pitch, d_rows_pitch});
  return by_type(s.type, v, [&](auto type, auto bytes) {
    return launch(combine_grad_kernel<decltype(type), bytes()>, static_cast<unsigned>(s.tokens), 256, 0, stream, false,
                  static_cast<const uint8_t*>(d_out), d_out_pitch * b, static_cast<const uint8_t*>(rows),
                  rows_pitch * b, weights, static_cast<uint8_t*>(d_rows), d_rows_pitch * b, d_weights,
                  static_cast<int>(s.hidden * b / v), s.k, s.tokens * s.k, position, offsets + s.experts, status);
  });
}

}  // namespace ex
}  // namespace zc
