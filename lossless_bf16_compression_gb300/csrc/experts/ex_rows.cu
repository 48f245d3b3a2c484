// ex_rows.cu -- rows to their places in the order by expert and back, with weights, and the
// gradients.  The order is a permutation known from the sort, so every kernel here is driven by
// tokens: a token's row is read (or written) once and its k sorted rows once each, which is all
// the traffic there is, and every sum over j runs inside one thread in slot order (no atomics).
// Bound by HBM when there are many tokens, by two dependent loads (position, then row) when there
// are few; so a thread asks for the rows of eight slots before it uses the first.
#include <initializer_list>

#include "ex_common.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kMaxThreads = 256;
// Smaller CTAs keep an SM's loads further apart: combine of 16384 x 8 x 7168 with 256 threads 365
// us, with 128 336 us; of 4999 x 6 x 2050 53 and 41 us.
constexpr int kCombineThreads = 128;
constexpr int kBatch = 8;  // slots whose rows a thread has in flight

// A position that may be used as an address; reported otherwise.
__device__ __forceinline__ bool in_range(int p, size_t slots, int* status) {
  if (p >= 0 && static_cast<size_t>(p) < slots) return true;
  set_error(status, ZC_ERR_CORRUPT);
  return false;
}

// Vectors of a row that a thread takes, a row's threads apart.  Rows that only 4-byte (or smaller)
// vectors divide need more of them in flight.
constexpr int per_thread(int bytes) { return bytes == 16 ? 1 : 4; }

// How a row's vectors are shared out: to `parts` CTAs of `threads`.
struct Cut {
  unsigned parts, threads;
};
Cut cut_row(size_t vecs, int bytes, unsigned most_threads) {
  const unsigned u = per_thread(bytes), most = most_threads * u;
  const unsigned parts = static_cast<unsigned>((vecs + most - 1) / most);
  const unsigned each = static_cast<unsigned>((vecs + parts * u - 1) / (parts * u));
  return {parts, (each + 31) / 32 * 32};
}
// This thread's first vector.
template <int B>
__device__ __forceinline__ int first_vector(unsigned parts) {
  return static_cast<int>(blockIdx.x % parts * blockDim.x * per_thread(B) + threadIdx.x);
}
// A token's vectors as a thread holds them, and to a slot's row.
template <int B>
struct Held {
  static constexpr int U = per_thread(B);
  using V = typename Bytes<B>::type;
  V v[U];
  __device__ __forceinline__ void load(const uint8_t* row, int c, int vecs) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = c + u * static_cast<int>(blockDim.x);
      v[u] = load_if<B>(row + static_cast<size_t>(at) * B, at < vecs);
    }
  }
  __device__ __forceinline__ void store(uint8_t* row, int c, int vecs, bool zeros) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = c + u * static_cast<int>(blockDim.x);
      if (at < vecs) reinterpret_cast<V*>(row)[at] = zeros ? V{} : v[u];
    }
  }
};

// rows[position[t, j]] = x[t].  Short rows share a CTA, one token for each threadIdx.y: it only stores,
// so what bounds them is how fast CTAs start (16384 x 2 x 1024: 28 -> 22 us; the other kernels
// lose more by giving up uniform registers for a token's positions and addresses, the combine
// gradient at that size 53 -> 84 us).
template <int B>
__global__ void __launch_bounds__(kMaxThreads) dispatch_kernel(const uint8_t* __restrict__ x, size_t x_pitch,
                                                               uint8_t* __restrict__ rows, size_t rows_pitch, int vecs,
                                                               unsigned parts, size_t tokens, int k,
                                                               const int* __restrict__ position,
                                                               const int* __restrict__ total, int* status) {
  let_next_start();
  const size_t t = static_cast<size_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y, slots = tokens * k;
  const int c = first_vector<B>(parts);
  if (t >= tokens) return;
  Held<B> held;
  held.load(x + t * x_pitch, c, vecs);  // x does not come from the sort
  wait_for_previous();
  const int kept = *total;
  for (int j = 0; j < k; ++j) {
    const int p = position[t * k + j];
    if (in_range(p, slots, status)) held.store(rows + p * rows_pitch, c, vecs, p >= kept);
  }
}

// Sort and dispatch of few slots in one launch: every CTA counts, for the slots of its token, the
// slots that come before them -- slots x k comparisons, shared by its threads -- so no CTA waits
// for another.  At 64 tokens x 8 that is 16 comparisons a thread.
constexpr size_t kSmallSlots = 1024;

template <typename Id, int B>
__global__ void __launch_bounds__(kMaxThreads) small_dispatch_kernel(
    const Id* __restrict__ ids, int slots, int experts, const uint8_t* __restrict__ x, size_t x_pitch,
    uint8_t* __restrict__ rows, size_t rows_pitch, int vecs, unsigned parts, int k, int* __restrict__ position,
    int* __restrict__ offsets) {
  __shared__ short keys[kSmallSlots];
  __shared__ int place[ZC_MOE_MAX_K];
  __shared__ int bins[ZC_MOE_MAX_EXPERTS + 1];
  __shared__ int kept;
  let_next_start();
  wait_for_previous();
  const int t = static_cast<int>(blockIdx.x / parts), part = static_cast<int>(blockIdx.x % parts);
  const int c = first_vector<B>(parts), lane = threadIdx.x % 32;
  Held<B> held;
  held.load(x + t * x_pitch, c, vecs);
  const bool starts = blockIdx.x == 0;  // this CTA writes the offsets as well
  if (threadIdx.x < ZC_MOE_MAX_K) place[threadIdx.x] = 0;
  if (threadIdx.x == 0) kept = 0;
  if (starts)
    for (int i = threadIdx.x; i <= experts; i += blockDim.x) bins[i] = 0;
  __syncthreads();
  int valid = 0;
  for (int s = threadIdx.x; s < slots; s += blockDim.x) {
    const Id id = ids[s];
    const int key = id >= 0 && id < experts ? static_cast<int>(id) : experts;
    keys[s] = static_cast<short>(key);
    valid += key < experts;
    if (starts) atomicAdd(&bins[key], 1);
  }
  valid = __reduce_add_sync(~0u, valid);
  if (lane == 0 && valid) atomicAdd(&kept, valid);
  __syncthreads();
  for (int j = 0; j < k; ++j) {
    const int s = t * k + j, key = keys[s];
    int before = 0;
    for (int o = threadIdx.x; o < slots; o += blockDim.x) {
      const int other = keys[o];
      before += other < key || (other == key && o < s);
    }
    before = __reduce_add_sync(~0u, before);
    if (lane == 0 && before) atomicAdd(&place[j], before);
  }
  __syncthreads();
  if (part == 0 && static_cast<int>(threadIdx.x) < k) position[t * k + threadIdx.x] = place[threadIdx.x];
  for (int j = 0; j < k; ++j) {
    const int p = place[j];
    held.store(rows + p * rows_pitch, c, vecs, p >= kept);
  }
  if (starts && threadIdx.x < 32) {
    int before = 0;
    for (int base = 0; base <= experts; base += 32) {
      const int e = base + lane;
      const int n = e <= experts ? bins[e] : 0;
      int incl = n;
      for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(~0u, incl, d);
        if (lane >= d) incl += u;
      }
      if (e <= experts) offsets[e] = before + incl - n;
      before += __shfl_sync(~0u, incl, 31);
    }
  }
}

// out[t] = sum over j of weights[t, j] rows[position[t, j]].  A thread takes Tokens tokens that follow
// one another, with kBatch / Tokens of each one's slots at a time: eight rows in flight however few
// slots a token has.
template <typename T, int B, int Tokens, bool Weighted>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const uint8_t* __restrict__ rows, size_t rows_pitch,
                                                              const float* __restrict__ weights,
                                                              uint8_t* __restrict__ out, size_t out_pitch, int vecs,
                                                              unsigned parts, size_t tokens, int k,
                                                              const int* __restrict__ position,
                                                              const int* __restrict__ total, int* status) {
  constexpr int N = B / sizeof(T), U = per_thread(B), S = kBatch / Tokens;
  let_next_start();
  wait_for_previous();
  const size_t t0 = static_cast<size_t>(blockIdx.x / parts) * Tokens, slots = tokens * k;
  const int c = first_vector<B>(parts);
  if (c >= vecs || t0 >= tokens) return;
  const int kept = *total;
  float acc[Tokens][U][N] = {};
  for (int j0 = 0; j0 < k; j0 += S) {
    Pack<T, B> v[kBatch][U];
    float w[kBatch];
    int at[kBatch];
    bool here[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const size_t t = min(t0 + i / S, tokens - 1), s = t * k + min(j0 + i % S, k - 1);
      at[i] = position[s];
      w[i] = Weighted ? weights[s] : 1.f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      here[i] = j0 + i % S < k && t0 + i / S < tokens && in_range(at[i], slots, status) && at[i] < kept;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c + u * static_cast<int>(blockDim.x);
        v[i][u].raw = load_if<B>(rows + at[i] * rows_pitch + static_cast<size_t>(cu) * B, here[i] && cu < vecs);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e)
          acc[i / S][u][e] = here[i] ? fmaf(w[i], to_float(v[i][u].v[e]), acc[i / S][u][e]) : acc[i / S][u][e];
  }
#pragma unroll
  for (int i = 0; i < Tokens; ++i)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cu = c + u * static_cast<int>(blockDim.x);
      Pack<T, B> o;
#pragma unroll
      for (int e = 0; e < N; ++e) o.v[e] = from_float<T>(acc[i][u][e]);
      if (cu < vecs && t0 + i < tokens)
        reinterpret_cast<typename Bytes<B>::type*>(out + (t0 + i) * out_pitch)[cu] = o.raw;
    }
}

// d_rows[position[t, j]] = weights[t, j] d_out[t], d_weights[t, j] = <d_out[t], rows[...]>.  One
// CTA a token: each thread sums its vectors' products, then lanes, then warps, in a fixed order.
template <typename T, int B>
__global__ void __launch_bounds__(kMaxThreads) combine_grad_kernel(
    const uint8_t* __restrict__ d_out, size_t d_out_pitch, const uint8_t* __restrict__ rows, size_t rows_pitch,
    const float* __restrict__ weights, uint8_t* __restrict__ d_rows, size_t d_rows_pitch, float* __restrict__ d_weights,
    int vecs, size_t tokens, int k, const int* __restrict__ position, const int* __restrict__ total, int* status) {
  constexpr int N = B / sizeof(T);
  using V = typename Bytes<B>::type;
  __shared__ float sums[kBatch][kMaxThreads / 32];
  let_next_start();
  wait_for_previous();
  const size_t t = blockIdx.x, slots = tokens * k;
  const int kept = *total, warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    int at[kBatch];
    float w[kBatch], dot[kBatch];
    bool ok[kBatch], here[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const size_t s = t * k + j0 + i;
      at[i] = j0 + i < k ? position[s] : 0;
      ok[i] = j0 + i < k && in_range(at[i], slots, status);
      here[i] = ok[i] && at[i] < kept;
      w[i] = here[i] ? weights[s] : 0.f;
      dot[i] = 0.f;
    }
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
      Pack<T, B> d, r[kBatch];
      d.raw = reinterpret_cast<const V*>(d_out + t * d_out_pitch)[c];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        r[i].raw = load_if<B>(rows + at[i] * rows_pitch + static_cast<size_t>(c) * B, here[i]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        Pack<T, B> o;
        o.raw = V{};
        if (here[i]) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float g = to_float(d.v[e]);
            o.v[e] = from_float<T>(w[i] * g);
            dot[i] = fmaf(g, to_float(r[i].v[e]), dot[i]);
          }
        }
        if (ok[i]) reinterpret_cast<V*>(d_rows + at[i] * d_rows_pitch)[c] = o.raw;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      for (int m = 16; m; m /= 2) dot[i] += __shfl_xor_sync(~0u, dot[i], m);
      if (lane == 0) sums[i][warp] = dot[i];
    }
    __syncthreads();
    if (threadIdx.x < kBatch && j0 + static_cast<int>(threadIdx.x) < k) {
      float s = 0.f;
      for (int i = 0; i < warps; ++i) s += sums[threadIdx.x][i];
      d_weights[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

template <typename F>
cudaError_t by_bytes(int bytes, F&& f) {
  using std::integral_constant;
  return bytes == 16  ? f(integral_constant<int, 16>{})
         : bytes == 4 ? f(integral_constant<int, 4>{})
                      : f(integral_constant<int, 2>{});
}
template <typename F>
cudaError_t by_type(int type, int bytes, F&& f) {
  using std::integral_constant;
  if (type == ZC_TYPE_FP32)
    return bytes == 16 ? f(float{}, integral_constant<int, 16>{}) : f(float{}, integral_constant<int, 4>{});
  const auto half = [&](auto t) { return by_bytes(bytes, [&](auto b) { return f(t, b); }); };
  return type == ZC_TYPE_FP16 ? half(__half{}) : half(__nv_bfloat16{});
}

}  // namespace

cudaError_t launch_dispatch(const RowShape& s, const void* x, size_t x_pitch, void* rows, size_t rows_pitch,
                            const int* position, const int* offsets, int* status, cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {x, rows}, {x_pitch, rows_pitch});
  const size_t vecs = s.hidden * b / v;
  const Cut cut = cut_row(vecs, v, kMaxThreads);
  return by_bytes(v, [&](auto bytes) {
    const unsigned together = kMaxThreads / cut.threads;  // tokens of a CTA
    return launch(dispatch_kernel<bytes()>, static_cast<unsigned>((s.tokens + together - 1) / together) * cut.parts,
                  dim3(cut.threads, together), 0, stream, true,
                  static_cast<const uint8_t*>(x), x_pitch * b, static_cast<uint8_t*>(rows), rows_pitch * b,
                  static_cast<int>(vecs), cut.parts, s.tokens, s.k, position, offsets + s.experts, status);
  });
}

bool small_dispatch(size_t slots) { return slots > 0 && slots <= kSmallSlots; }

cudaError_t launch_small_dispatch(const RowShape& s, const void* ids, int id_bytes, const void* x, size_t x_pitch,
                                  void* rows, size_t rows_pitch, int* position, int* offsets, cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {x, rows}, {x_pitch, rows_pitch});
  const size_t vecs = s.hidden * b / v;
  const Cut cut = cut_row(vecs, v, kMaxThreads);
  const unsigned threads = cut.threads < 64 ? 64 : cut.threads;  // at least ZC_MOE_MAX_K
  return by_bytes(v, [&](auto bytes) {
    const auto go = [&](auto* p) {
      using Id = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
      return launch(small_dispatch_kernel<Id, bytes()>, static_cast<unsigned>(s.tokens) * cut.parts, threads, 0,
                    stream, true, p, static_cast<int>(s.tokens * s.k), s.experts, static_cast<const uint8_t*>(x),
                    x_pitch * b, static_cast<uint8_t*>(rows), rows_pitch * b, static_cast<int>(vecs), cut.parts, s.k,
                    position, offsets);
    };
    return id_bytes == 8 ? go(static_cast<const long long*>(ids)) : go(static_cast<const int*>(ids));
  });
}

cudaError_t launch_combine(const RowShape& s, const void* rows, size_t rows_pitch, const float* weights,
                           const int* position, const int* offsets, void* out, size_t out_pitch, int* status,
                           cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {rows, out}, {rows_pitch, out_pitch});
  const size_t vecs = s.hidden * b / v;
  const Cut cut = cut_row(vecs, v, kCombineThreads);
  const auto go = [&](auto type, auto bytes, auto tokens) {
    return launch(weights ? combine_kernel<decltype(type), bytes(), tokens(), true>
                          : combine_kernel<decltype(type), bytes(), tokens(), false>,
                  static_cast<unsigned>((s.tokens + tokens() - 1) / tokens()) * cut.parts, cut.threads, 0, stream, true,
                  static_cast<const uint8_t*>(rows), rows_pitch * b, weights, static_cast<uint8_t*>(out), out_pitch * b, static_cast<int>(vecs), cut.parts, s.tokens, s.k,
                  position, offsets + s.experts, status);
  };
  return by_type(s.type, v, [&](auto type, auto bytes) {
    // few tokens: one a thread, so that they spread over the SMs
    const bool many = s.tokens * cut.parts >= 2048;
    return many && s.k <= 2   ? go(type, bytes, std::integral_constant<int, 4>{})
           : many && s.k <= 4 ? go(type, bytes, std::integral_constant<int, 2>{})
                              : go(type, bytes, std::integral_constant<int, 1>{});
  });
}

cudaError_t launch_combine_grad(const RowShape& s, const void* d_out, size_t d_out_pitch, const void* rows,
                                size_t rows_pitch, const float* weights, const int* position, const int* offsets,
                                void* d_rows, size_t d_rows_pitch, float* d_weights, int* status,
                                cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const int v = vector_bytes(b, s.hidden, {d_out, rows, d_rows}, {d_out_pitch, rows_pitch, d_rows_pitch});
  const size_t vecs = s.hidden * b / v;
  return by_type(s.type, v, [&](auto type, auto bytes) {
    // A token's sums need all of its row, which the CTA's threads walk: with few tokens more threads
    // finish a row sooner (1 token x 8 x 7168: 12 us with 256, 16 with 128, 25 with 64), with many
    // fewer leave more CTAs to an SM (16384 x 2 x 1024: 41 us with 64, 53 with 128, 16384 x 8 x
    // 7168: 582 and 576).
    const unsigned most = s.tokens < 2048 ? 256 : vecs <= 256 ? 64 : 128;
    return launch(combine_grad_kernel<decltype(type), bytes()>, static_cast<unsigned>(s.tokens),
                  cut_row(vecs, 16, most).threads, 0, stream, true,
                  static_cast<const uint8_t*>(d_out), d_out_pitch * b, static_cast<const uint8_t*>(rows),
                  rows_pitch * b, weights, static_cast<uint8_t*>(d_rows), d_rows_pitch * b, d_weights,
                  static_cast<int>(vecs), s.tokens, s.k, position, offsets + s.experts, status);
  });
}

}  // namespace ex
}  // namespace zc
