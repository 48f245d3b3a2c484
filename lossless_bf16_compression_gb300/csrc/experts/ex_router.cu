// ex_router.cu -- a router's choice of experts, its balance loss, and their gradients.
//
// One warp to a token: the row's logits lie in registers, N to a lane, and every sum over the row is a
// sum over the warp.
#include "ex_router.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kTokenWarps = 8;  // tokens of a CTA at a time
constexpr float kInf = __builtin_inff();

// ------------------------------------------------------------------ rows in registers

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

// A row of up to 32 N values, V neighbours to a lane and N / V times 32 V values, the V by one load where
// every row starts and ends on a whole vector of them (Whole).  Which lane holds what does not depend on
// that, so results do not either.
template <typename T, int N, bool Whole>
struct Row {
  static constexpr int V = N * sizeof(T) <= 16 ? N : 16 / sizeof(T);
  using W = typename Word<V * sizeof(T)>::type;
  T v[N];

  __device__ __forceinline__ static int column(int i) {
    return (i / V * 32 + static_cast<int>(threadIdx.x % 32)) * V + i % V;
  }
  // Values past the row's end are -infinity.
  __device__ __forceinline__ void load(const T* row, int experts) {
    union {
      W w;
      T v[V];
    } u;
#pragma unroll
    for (int i = 0; i < N; i += V) {
#pragma unroll
      for (int j = 0; j < V; ++j) u.v[j] = lowest<T>();
      if (Whole) {
        if (column(i) < experts) u.w = *reinterpret_cast<const W*>(row + column(i));
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
      W w;
      T v[V];
    } u;
#pragma unroll
    for (int i = 0; i < N; i += V) {
#pragma unroll
      for (int j = 0; j < V; ++j) u.v[j] = v[i + j];
      if (Whole) {
        if (column(i) < experts) *reinterpret_cast<W*>(row + column(i)) = u.w;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (column(i + j) < experts) row[column(i + j)] = v[i + j];
      }
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// ------------------------------------------------------------------ the order of logits
//
// Logits as unsigned integers in their own order: a NaN of either sign above all, -0 equal to 0, and 0 for
// -infinity, which is never chosen.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  if (v != v) return ~0u;
  return v == -kInf ? 0u : b ^ (b >> 31 ? ~0u : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t key) {
  return __uint_as_float(key >> 31 ? key ^ 0x80000000u : ~key);
}
// The row's largest logit, NaN above all, as the same number in every lane.
__device__ __forceinline__ float row_top(uint32_t key) {
  const uint32_t top = __reduce_max_sync(~0u, key);
  return top == 0 ? -kInf : unordered(top);
}

// The score of a logit relative to a common factor: exp(x - m) for a softmax; for sigmoids sigmoid(x) e^-m with
// m <= 0, so that a row of very low logits does not vanish before it is divided by its sum.
__device__ __forceinline__ float scaled_sigmoid(float x, float m) {
  return x > 0 ? 1.0f / (1.0f + expf(-x)) : expf(x - m) / (1.0f + expf(x));
}
__device__ __forceinline__ float one_minus_sigmoid(float x) { return 1.0f / (1.0f + expf(x)); }

// ------------------------------------------------------------------ the choice

template <typename T, int N, bool Whole>
__global__ void __launch_bounds__(32 * kTokenWarps)
    route_kernel(const T* logits, size_t pitch, size_t tokens, int experts, int k, int score, int normalize, float scale,
                 float* weights, int* ids) {
  using R = Row<T, N, Whole>;
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32;
  const size_t t = static_cast<size_t>(blockIdx.x) * kTokenWarps + threadIdx.x / 32;
  if (t >= tokens) return;
  R row;
  row.load(logits + t * pitch, experts);
  uint32_t key[N], best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    key[i] = ordered(to_float(row.v[i]));
    if (key[i] > best) best = key[i], at = R::column(i);
  }
  const float top = row_top(best);

  float total = 0;  // of the whole row, where the softmax is not of the chosen alone
  if (score == ZC_SCORE_SOFTMAX && !normalize) {
#pragma unroll
    for (int i = 0; i < N; ++i) total += expf(to_float(row.v[i]) - top);
    total = warp_sum(total);
  }

  float x[2] = {-kInf, -kInf};  // what slots lane and lane + 32 hold
  int e[2] = {-1, -1};
  for (int j = 0; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(~0u, best);
    if (m == 0) break;
    const int first = __reduce_min_sync(~0u, best == m ? at : experts);
    if (lane == j % 32) {
      const int h = j / 32;
      if (h) x[1] = unordered(m), e[1] = first;
      else x[0] = unordered(m), e[0] = first;
    }
    if (best == m && at == first) {
      best = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (R::column(i) == first) key[i] = 0;
        if (key[i] > best) best = key[i], at = R::column(i);
      }
    }
  }

  float w[2];
  const float m = score == ZC_SCORE_SOFTMAX ? top : normalize ? fminf(top, 0.0f) : 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = e[h] < 0 ? 0.0f : score == ZC_SCORE_SOFTMAX ? expf(x[h] - m) : scaled_sigmoid(x[h], m);
  if (normalize) total = warp_sum(w[0] + w[1]);
  else if (score == ZC_SCORE_SIGMOID) total = 1.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    if (j < k) {
      weights[t * k + j] = e[h] < 0 ? 0.0f : scale * (w[h] / total);
      ids[t * k + j] = e[h];
    }
  }
}

// ------------------------------------------------------------------ the gradient
//
// With g the gradients of a token's weights, times scale:
//   softmax of the chosen   d_j = w_j (g_j - sum g w)
//   sigmoids over their sum d_j = w_j (1 - s_j) (g_j - sum g w)
//   sigmoids                d_j = s_j (1 - s_j) g_j
//   softmax of the row      d_i = p_i (g_i - sum g p), g_i the sum over the slots of expert i
// and of the balance loss  d_i = d_loss p_i (slope_i - sum slope p), times 1 - s_i for sigmoids.
// What belongs to chosen experts goes through a row in shared memory.

template <typename T, int N, bool Whole>
__global__ void __launch_bounds__(32 * kTokenWarps)
    route_grad_kernel(const float* d_weights, const int* ids, const float* d_loss, const float* slope, const T* logits,
                      size_t pitch, size_t tokens, int experts, int k, int score, int normalize, float scale, T* d_logits,
                      size_t d_pitch) {
  using R = Row<T, N, Whole>;
  extern __shared__ float rows[];  // a row of N x 32 to a warp, in the order of its lanes' registers
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32;
  float* mine = rows + threadIdx.x / 32 * (32 * N);
  const bool softmax = score == ZC_SCORE_SOFTMAX, whole = softmax && !normalize && d_weights != nullptr;
  const float loss = d_loss != nullptr ? *d_loss : 0.0f;
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = slope != nullptr && R::column(i) < experts ? loss * slope[R::column(i)] : 0.0f;

  const size_t step = static_cast<size_t>(gridDim.x) * kTokenWarps;
  for (size_t t = static_cast<size_t>(blockIdx.x) * kTokenWarps + threadIdx.x / 32; t < tokens; t += step) {
    const T* row = logits + t * pitch;
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = 0.0f;
    // The slots of this lane.
    float g[2] = {0, 0}, x[2] = {-kInf, -kInf};
    int e[2] = {-1, -1};
    if (d_weights != nullptr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        if (j < k) {
          e[h] = ids[t * k + j];
          g[h] = scale * d_weights[t * k + j];
          if (e[h] < 0 || e[h] >= experts) e[h] = -1;
          else x[h] = to_float(row[e[h]]);
          if (x[h] == -kInf) e[h] = -1;
        }
        if (e[h] < 0) g[h] = 0;
      }
    }
    float inner = 0, factor = 0, top = -kInf;  // of the whole row: sum of slope p (and g p), 1 / sum of scores
    if (slope != nullptr || whole) {
      R r;
      r.load(row, experts);
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) best = max(best, ordered(to_float(r.v[i])));
      top = row_top(best);
      if (top != -kInf) {
        const float m = softmax ? top : fminf(top, 0.0f);
        float sum = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = to_float(r.v[i]);
          d[i] = softmax ? expf(v - m) : scaled_sigmoid(v, m);
          sum += d[i];
          dot += a[i] * d[i];
        }
        factor = 1.0f / warp_sum(sum);
        if (whole) dot += (e[0] < 0 ? 0.0f : g[0] * expf(x[0] - top)) + (e[1] < 0 ? 0.0f : g[1] * expf(x[1] - top));
        inner = warp_sum(dot) * factor;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float v = to_float(r.v[i]);
          d[i] = d[i] * factor * (a[i] - inner);
          if (!softmax) d[i] *= one_minus_sigmoid(v);
          if (v == -kInf) d[i] = 0;
        }
      }
    }
    if (d_weights != nullptr) {
      float c[2];
      if (whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) c[h] = e[h] < 0 ? 0.0f : g[h] * expf(x[h] - top) * factor;
      } else {
        const float first = row_top(max(ordered(e[0] < 0 ? -kInf : x[0]), ordered(e[1] < 0 ? -kInf : x[1])));
        const float m = softmax ? first : normalize ? fminf(first, 0.0f) : 0.0f;
        float w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = e[h] < 0 ? 0.0f : softmax ? expf(x[h] - m) : scaled_sigmoid(x[h], m);
        float mean = 0, f = 1;
        if (normalize) {
          f = first == -kInf ? 0.0f : 1.0f / warp_sum(w[0] + w[1]);
          mean = warp_sum(g[0] * w[0] + g[1] * w[1]) * f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          c[h] = e[h] < 0 ? 0.0f : w[h] * f * (g[h] - mean);
          if (!softmax && e[h] >= 0) c[h] *= one_minus_sigmoid(x[h]);
        }
      }
      // Into the places of their experts: column c is register i of a lane.
#pragma unroll
      for (int i = 0; i < N; ++i) mine[i * 32 + lane] = d[i];
      __syncwarp();
      const auto place = [&](int col) { return (col / (32 * R::V) * R::V + col % R::V) * 32 + col / R::V % 32; };
      // (A lane without a slot has a number of its own.)
      const unsigned same = __match_any_sync(~0u, e[0] < 0 ? -1 - lane : e[0]);
      if (k <= 32 && __all_sync(~0u, (same & (same - 1)) == 0)) {
        if (e[0] >= 0) mine[place(e[0])] += c[0];
      } else {  // the same expert twice, which zc_moe_route does not choose, or many slots: one after the other
        for (int j = 0; j < k; ++j) {
          if (lane == j % 32) {
            const int h = j / 32;
            const int to = h ? e[1] : e[0];
            if (to >= 0) mine[place(to)] += h ? c[1] : c[0];
          }
          __syncwarp();
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = mine[i * 32 + lane];
      __syncwarp();
    }
    R out;
#pragma unroll
    for (int i = 0; i < N; ++i) out.v[i] = from_float<T>(d[i]);
    out.store(d_logits + t * d_pitch, experts);
  }
}

// ------------------------------------------------------------------ the balance loss
//
// Each warp keeps the sums of its tokens' probabilities in registers, a lane's own columns; a CTA's are added
// in shared memory in the order of its warps, the CTAs' by the kernel that follows, in their order.

constexpr int kBalanceWarps = 16;
constexpr int kBalanceThreads = 32 * kBalanceWarps;
constexpr int kSums = 8;  // rows of sums in shared memory
constexpr size_t kMaxParts = 152;

struct Parts {  // of each CTA: sums, counts, tokens
  float* sums;
  int *counts, *tokens;
};
__host__ __device__ inline Parts parts_of(void* workspace, size_t ctas, size_t experts) {
  float* s = static_cast<float*>(workspace);
  int* c = reinterpret_cast<int*>(s + ctas * experts);
  return {s, c, c + ctas * experts};
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Loss, counts and slopes from the sums and counts of one expert a thread (threads past the last one: zeros).
template <int Threads>
__device__ __forceinline__ void settle(const float* sums, const int* totals, int tokens, int experts, int k, float* loss,
                                       int* counts, float* slope) {
  __shared__ double parts[Threads / 32];
  const double n = tokens;
  double mine = 0;
  for (int e = threadIdx.x; e < experts; e += Threads) {
    const double c = totals[e], s = tokens > 0 ? experts * c / (k * n * n) : 0.0;
    counts[e] = totals[e];
    slope[e] = static_cast<float>(s);
    mine += s * sums[e];
  }
  mine = warp_sum(mine);
  if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0;
    for (int w = 0; w < Threads / 32; ++w) all += parts[w];
    *loss = static_cast<float>(all);
  }
}

template <typename T, int N, bool Whole>
__global__ void __launch_bounds__(kBalanceThreads)
    balance_kernel(const T* logits, size_t pitch, const int* ids, size_t tokens, int experts, int k, int score, float* loss,
                   int* counts, float* slope, void* workspace) {
  using R = Row<T, N, Whole>;
  extern __shared__ float sums[];  // [kSums][experts], then experts counts
  __shared__ int live_of[kBalanceWarps];
  int* found = reinterpret_cast<int*>(sums + kSums * experts);
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int e = threadIdx.x; e < experts; e += kBalanceThreads) found[e] = 0;
  __syncthreads();
  const size_t each = (tokens + gridDim.x - 1) / gridDim.x;
  const size_t begin = min(tokens, blockIdx.x * each), end = min(tokens, begin + each);
  for (size_t s = begin * k + threadIdx.x; s < end * k; s += kBalanceThreads) {
    const int e = ids[s];
    if (e >= 0 && e < experts) atomicAdd(&found[e], 1);
  }
  float sum[N];
  int live = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0;
  for (size_t t = begin + warp; t < end; t += kBalanceWarps) {
    R r;
    r.load(logits + t * pitch, experts);
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) best = max(best, ordered(to_float(r.v[i])));
    const float top = row_top(best);
    if (top == -kInf) continue;
    ++live;
    const float m = score == ZC_SCORE_SOFTMAX ? top : fminf(top, 0.0f);
    float p[N], total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = to_float(r.v[i]);
      p[i] = score == ZC_SCORE_SOFTMAX ? expf(v - m) : scaled_sigmoid(v, m);
      total += p[i];
    }
    const float f = 1.0f / warp_sum(total);
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] += p[i] * f;
  }
  if (lane == 0) live_of[warp] = live;
#pragma unroll
  for (int round = 0; round < kBalanceWarps / kSums; ++round) {
    if (warp / kSums == round) {
      float* to = sums + warp % kSums * experts;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = R::column(i);
        if (c < experts) to[c] = round == 0 ? sum[i] : to[c] + sum[i];
      }
    }
    __syncthreads();
  }
  int rows = 0;
  for (int w = 0; w < kBalanceWarps; ++w) rows += live_of[w];
  const bool alone = gridDim.x == 1;
  const Parts parts = parts_of(workspace, gridDim.x, experts);
  for (int e = threadIdx.x; e < experts; e += kBalanceThreads) {
    float s = 0;
    for (int w = 0; w < kSums; ++w) s += sums[w * experts + e];
    if (alone) {
      sums[e] = s;  // (read by this thread only: row 0 of column e)
    } else {
      parts.sums[blockIdx.x * static_cast<size_t>(experts) + e] = s;
      parts.counts[blockIdx.x * static_cast<size_t>(experts) + e] = found[e];
    }
  }
  if (alone) {
    __syncthreads();
    settle<kBalanceThreads>(sums, found, rows, experts, k, loss, counts, slope);
  } else if (threadIdx.x == 0) {
    parts.tokens[blockIdx.x] = rows;
  }
}

constexpr int kSettleThreads = 1024;
__global__ void __launch_bounds__(kSettleThreads) settle_kernel(void* workspace, int ctas, int experts, int k, float* loss,
                                                                int* counts, float* slope) {
  __shared__ float sums[ZC_MOE_MAX_EXPERTS];
  __shared__ int totals[ZC_MOE_MAX_EXPERTS];
  __shared__ int tokens;
  wait_for_previous();
  let_next_start();
  const Parts parts = parts_of(workspace, ctas, experts);
  for (int e = threadIdx.x; e < experts; e += kSettleThreads) {
    float s = 0;
    int c = 0;
    for (int b = 0; b < ctas; ++b) {
      s += parts.sums[static_cast<size_t>(b) * experts + e];
      c += parts.counts[static_cast<size_t>(b) * experts + e];
    }
    sums[e] = s;
    totals[e] = c;
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int b = 0; b < ctas; ++b) n += parts.tokens[b];
    tokens = n;
  }
  __syncthreads();
  settle<kSettleThreads>(sums, totals, tokens, experts, k, loss, counts, slope);
}

size_t balance_ctas(size_t tokens) {
  const size_t n = (tokens + 4 * kBalanceWarps - 1) / (4 * kBalanceWarps);
  return n < 1 ? 1 : n > kMaxParts ? kMaxParts : n;
}

// ------------------------------------------------------------------ which instance

template <typename T, typename F>
cudaError_t by_shape(int experts, std::initializer_list<const void*> bases, std::initializer_list<size_t> pitches, F f) {
  const auto go = [&](auto n) {
    uintptr_t all = experts * sizeof(T);
    for (const void* b : bases) all |= reinterpret_cast<uintptr_t>(b);
    for (size_t p : pitches) all |= p * sizeof(T);
    if (all % (Row<T, decltype(n)::value, true>::V * sizeof(T)) == 0) return f(n, std::true_type());
    return f(n, std::false_type());
  };
  if (experts <= 64) return go(std::integral_constant<int, 2>());
  if (experts <= 128) return go(std::integral_constant<int, 4>());
  if (experts <= 256) return go(std::integral_constant<int, 8>());
  return go(std::integral_constant<int, 32>());
}
template <typename F>
cudaError_t by_type(int type, F f) {
  if (type == ZC_TYPE_BF16) return f(__nv_bfloat16());
  if (type == ZC_TYPE_FP16) return f(__half());
  return f(float());
}

}  // namespace

cudaError_t launch_route(const RouterShape& s, const void* logits, size_t pitch, float* weights, int* ids,
                         cudaStream_t stream) {
  const auto grid = static_cast<unsigned>((s.tokens + kTokenWarps - 1) / kTokenWarps);
  return by_type(s.type, [&](auto t) {
    using T = decltype(t);
    return by_shape<T>(s.experts, {logits}, {pitch}, [&](auto n, auto whole) {
      return launch(ZC_KERNEL_MOE_ROUTE, route_kernel<T, decltype(n)::value, decltype(whole)::value>, grid, 32 * kTokenWarps, 0,
                    stream, static_cast<const T*>(logits), pitch, s.tokens, s.experts, s.k, s.score, s.normalize, s.scale,
                    weights, ids);
    });
  });
}

cudaError_t launch_route_grad(const RouterShape& s, const float* d_weights, const int* ids, const float* d_loss,
                              const float* slope, const void* logits, size_t pitch, void* d_logits, size_t d_pitch,
                              const DeviceInfo& dev, cudaStream_t stream) {
  const size_t ctas = (s.tokens + kTokenWarps - 1) / kTokenWarps, most = static_cast<size_t>(dev.sm_count) * 8;
  return by_type(s.type, [&](auto t) {
    using T = decltype(t);
    return by_shape<T>(s.experts, {logits, d_logits}, {pitch, d_pitch}, [&](auto n, auto whole) {
      constexpr int N = decltype(n)::value;
      return launch(ZC_KERNEL_MOE_ROUTE_GRAD, route_grad_kernel<T, N, decltype(whole)::value>,
                    static_cast<unsigned>(ctas < most ? ctas : most), 32 * kTokenWarps,
                    kTokenWarps * 32 * N * sizeof(float), stream, d_weights, ids, d_loss, slope,
                    static_cast<const T*>(logits), pitch, s.tokens, s.experts, s.k, s.score, s.normalize, s.scale,
                    static_cast<T*>(d_logits), d_pitch);
    });
  });
}

size_t balance_workspace(size_t tokens, int experts) {
  const size_t n = balance_ctas(tokens);
  return n > 1 ? n * (2 * static_cast<size_t>(experts) + 1) * 4 : 0;
}

cudaError_t launch_balance(const RouterShape& s, const void* logits, size_t pitch, const int* ids, float* loss, int* counts,
                           float* slope, void* workspace, cudaStream_t stream) {
  const int ctas = static_cast<int>(balance_ctas(s.tokens));
  const cudaError_t err = by_type(s.type, [&](auto t) {
    using T = decltype(t);
    return by_shape<T>(s.experts, {logits}, {pitch}, [&](auto n, auto whole) {
      return launch(ZC_KERNEL_MOE_BALANCE, balance_kernel<T, decltype(n)::value, decltype(whole)::value>, ctas, kBalanceThreads,
                    sizeof(float) * (kSums + 1) * s.experts, stream, static_cast<const T*>(logits), pitch, ids, s.tokens,
                    s.experts, s.k, s.score, loss, counts, slope, workspace);
    });
  });
  if (err != cudaSuccess || ctas == 1) return err;
  return launch(ZC_KERNEL_MOE_BALANCE, settle_kernel, 1, kSettleThreads, 0, stream, workspace, ctas, s.experts, s.k, loss,
                counts, slope);
}

}  // namespace ex
}  // namespace zc
