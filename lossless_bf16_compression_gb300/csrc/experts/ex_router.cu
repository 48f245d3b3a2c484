// ex_router.cu -- a router's choice of experts, its balance loss, and their gradients.
//
// One warp to a token: the row's logits lie in registers, N to a lane, and every sum over the row is a
// sum over the warp.
#include "ex_router.cuh"

#include <type_traits>

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

// ------------------------------------------------------------------ scores

// The largest value of the warp's; NaN if there is one.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

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

// ------------------------------------------------------------------ the order of logits
//
// A logit as an unsigned integer in its own order: a NaN of either sign above all, -0 equal to 0 (an addition of 0 makes
// them one), -infinity below all.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kNone = 0x007FFFFFu;  // of -infinity

// The keys that are searched for a row's largest logits.
//   16 bits: the logit's order above 0xFFFF - column: no two are equal, and equal logits go by column.
//   fp32: the order with its last bits given to the number of the lane's register, N - 1 - i.  Two logits that differ in
//   those bits alone, or not at all, may come in the wrong order: that is seen, and the row is searched again.
template <typename T, int N, bool Whole>
struct Keys {
  using R = Row<T, N, Whole>;
  static constexpr bool kUnique = sizeof(T) == 2;
  static constexpr uint32_t kLow = kUnique ? 0xFFFFu : N - 1;
  static constexpr uint32_t kLeast = sizeof(T) == 2 && std::is_same_v<T, __half> ? 0x03FFFFFFu : kNone;
  uint32_t k[N];

  __device__ __forceinline__ explicit Keys(const R& row) {
    if constexpr (kUnique) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        uint32_t w = pair_plus_zero(row.v[i], row.v[i + 1]), sign;
        asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(sign) : "r"(w));  // each half's sign, all over it
        w ^= sign | 0x80008000u;
        k[i] = w << 16 | (0xFFFFu - R::column(i));
        k[i + 1] = (w & 0xFFFF0000u) | (0xFFFFu - R::column(i + 1));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) k[i] = (ordered(row.v[i]) & ~kLow) | (N - 1 - i);
    }
  }
  __device__ __forceinline__ static uint32_t pair_plus_zero(__nv_bfloat16 a, __nv_bfloat16 b) {
    const __nv_bfloat162 r = __hadd2(__nv_bfloat162(a, b), __float2bfloat162_rn(0.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ __forceinline__ static uint32_t pair_plus_zero(__half a, __half b) {
    const __half2 r = __hadd2(__half2(a, b), __float2half2_rn(0.0f));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t best = k[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = max(best, k[i]);
    return best;
  }
  // The largest below m; 0: there is none.  (Distances from m - 1 wrap around for the others.)
  __device__ __forceinline__ uint32_t below(uint32_t m) const {
    uint32_t least = m - 1 - k[0];
#pragma unroll
    for (int i = 1; i < N; ++i) least = min(least, m - 1 - k[i]);
    return least < m ? m - 1 - least : 0u;
  }
};

// ------------------------------------------------------------------ the choice

// The k largest of a row whose search by keys was not sure, one after the other by value and column: slot lane (and
// lane + 32) gets its column.
template <typename T, int N, bool Whole>
__device__ __noinline__ int2 search_again(const T* logits, int experts, int k) {
  using R = Row<T, N, Whole>;
  const int lane = threadIdx.x % 32;
  R row;
  row.load(logits, experts);
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = ordered(to_float(row.v[i]));
  int2 e = make_int2(-1, -1);
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > best) best = key[i], at = R::column(i);
    const uint32_t m = __reduce_max_sync(~0u, best);
    if (m <= kNone) break;
    const int first = __reduce_min_sync(~0u, best == m ? at : experts);
    if (lane == j % 32) {
      if (j >= 32) e.y = first;
      else e.x = first;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (R::column(i) == first) key[i] = 0;
  }
  return e;
}

template <typename T, int N, bool Whole>
__global__ void __launch_bounds__(32 * kTokenWarps)
    route_kernel(const T* logits, size_t pitch, size_t tokens, int experts, int k, int score, int normalize, float scale,
                 float* weights, int* ids) {
  using R = Row<T, N, Whole>;
  using K = Keys<T, N, Whole>;
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32;
  const size_t t = static_cast<size_t>(blockIdx.x) * kTokenWarps + threadIdx.x / 32;
  if (t >= tokens) return;
  const T* from = logits + t * pitch;
  R row;
  row.load(from, experts);
  const K keys(row);

  int e[2] = {-1, -1};  // what slots lane and lane + 32 hold
  uint32_t best = keys.largest(), before = 0;
  bool unsure = false;
  int j = 0;
  for (; j < k; ++j) {
    const uint32_t m = __reduce_max_sync(~0u, best);
    if (m <= K::kLeast) break;
    int column;
    if (K::kUnique) {
      column = 0xFFFF - static_cast<int>(m & 0xFFFFu);
    } else {
      const unsigned who = __ballot_sync(~0u, best == m);
      const int i = N - 1 - static_cast<int>(m & K::kLow);
      column = (i / R::V * 32 + __ffs(who) - 1) * R::V + i % R::V;
      unsure |= (who & (who - 1)) != 0 || (m ^ before) <= K::kLow;
      before = m;
    }
    if (lane == (j & 31)) {
      if (j >= 32) e[1] = column;
      else e[0] = column;
    }
    if (best == m) best = keys.below(m);
  }
  if (!K::kUnique) {
    if (j == k) unsure |= (__reduce_max_sync(~0u, best) ^ before) <= K::kLow;
    if (unsure) {
      const int2 again = search_again<T, N, Whole>(from, experts, k);
      e[0] = again.x;
      e[1] = again.y;
    }
  }

  // (The chosen logits again, from the L1.)
  float x[2] = {-kInf, -kInf};
  if (e[0] >= 0) x[0] = to_float(from[e[0]]);
  if (k > 32 && e[1] >= 0) x[1] = to_float(from[e[1]]);
  const float top = __shfl_sync(~0u, x[0], 0);
  const bool softmax = score == ZC_SCORE_SOFTMAX;
  const auto value = [&](int h) {
    return e[h] < 0 ? 0.0f : softmax ? expf(x[h] - top) : scaled_sigmoid(x[h], normalize ? fminf(top, 0.0f) : 0.0f).s;
  };
  const float w0 = value(0), w1 = k > 32 ? value(1) : 0.0f;
  float total = 1.0f;
  if (normalize) {
    total = warp_sum(w0 + w1);
  } else if (softmax) {
    total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) total += expf(to_float(row.v[i]) - top);
    total = warp_sum(total);
  }
  if (lane < k) {
    weights[t * k + lane] = e[0] < 0 ? 0.0f : scale * (w0 / total);
    ids[t * k + lane] = e[0];
  }
  if (lane + 32 < k) {
    weights[t * k + lane + 32] = e[1] < 0 ? 0.0f : scale * (w1 / total);
    ids[t * k + lane + 32] = e[1];
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

constexpr int kGradCtas = 4;  // on an SM at a time, of up to eight values a lane

template <typename T, int N, bool Whole>
__global__ void __launch_bounds__(32 * kTokenWarps, N <= 8 ? kGradCtas : 1)
    route_grad_kernel(const float* d_weights, const int* ids, const float* d_loss, const float* slope, const T* logits,
                      size_t pitch, size_t tokens, int experts, int k, int score, int normalize, float scale, T* d_logits,
                      size_t d_pitch) {
  using R = Row<T, N, Whole>;
  __shared__ __align__(16) float rows[kTokenWarps][32 * N];  // a lane's registers one after the other
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32;
  float* mine = rows[threadIdx.x / 32];
  const bool softmax = score == ZC_SCORE_SOFTMAX, whole = softmax && !normalize && d_weights != nullptr, many = k > 32;
  const float loss = d_loss != nullptr ? *d_loss : 0.0f;
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = slope != nullptr && R::column(i) < experts ? loss * slope[R::column(i)] : 0.0f;

  // What a token needs is asked for while the one before it is at work: its row where all of it is read, and the slots
  // of this lane, lane and lane + 32.
  const bool dense = slope != nullptr || whole;
  R ahead;
  int id[2] = {-1, -1};
  float dw[2] = {0, 0};
  const auto ask = [&](size_t t) {
    if (dense) ahead.load(logits + t * pitch, t < tokens ? experts : 0);
    if (d_weights != nullptr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !many) break;
        const int j = lane + 32 * h;
        id[h] = -1;
        if (j < k && t < tokens) {
          id[h] = ids[t * k + j];
          dw[h] = d_weights[t * k + j];
        }
      }
    }
  };
  const size_t step = static_cast<size_t>(gridDim.x) * kTokenWarps;
  size_t t = static_cast<size_t>(blockIdx.x) * kTokenWarps + threadIdx.x / 32;
  ask(t);
  for (; t < tokens; t += step) {
    const T* row = logits + t * pitch;
    // A slot without an expert, or one that the token may not use, has e = -1 and g = 0.
    float g[2] = {0, 0}, x[2] = {-kInf, -kInf};
    int e[2] = {-1, -1};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !many) break;
      if (id[h] >= 0 && id[h] < experts) {
        x[h] = to_float(row[id[h]]);
        e[h] = id[h];
        g[h] = scale * dw[h];
      }
    }
    const R r = ahead;
    ask(t + step);
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = 0.0f;
    float factor = 0, top = -kInf;
    if (dense) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = to_float(r.v[i]);
        top = larger(top, v[i]);
      }
      top = warp_max(top);
      if (top != -kInf) {
        const float m = softmax ? top : fminf(top, 0.0f);
        float sum = 0, dot = 0, rest[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (softmax) {
            d[i] = expf(v[i] - m);
          } else {
            const Sigmoid s = scaled_sigmoid(v[i], m);
            d[i] = s.s;
            rest[i] = s.rest;
          }
          sum += d[i];
          dot += a[i] * d[i];
        }
        if (whole) dot += (e[0] < 0 ? 0.0f : g[0] * expf(x[0] - top)) + (!many || e[1] < 0 ? 0.0f : g[1] * expf(x[1] - top));
        factor = 1.0f / warp_sum(sum);
        const float inner = warp_sum(dot) * factor;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          d[i] *= factor * (a[i] - inner);
          if (!softmax) d[i] *= rest[i];
          if (v[i] == -kInf) d[i] = 0;
        }
      }
    }
    if (d_weights != nullptr) {
      float c[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (x[h] == -kInf) e[h] = -1, g[h] = 0;
      if (whole) {
        c[0] = e[0] < 0 ? 0.0f : g[0] * expf(x[0] - top) * factor;
        if (many) c[1] = e[1] < 0 ? 0.0f : g[1] * expf(x[1] - top) * factor;
      } else {
        const float first = normalize ? warp_max(larger(e[0] < 0 ? -kInf : x[0], e[1] < 0 ? -kInf : x[1])) : 0.0f;
        const float m = softmax ? first : fminf(first, 0.0f);
        float w[2] = {0, 0}, rest[2] = {1, 1};
        const auto weigh = [&](int h) {
          if (e[h] < 0) return;
          if (softmax) {
            w[h] = expf(x[h] - m);
          } else {
            const Sigmoid s = scaled_sigmoid(x[h], m);
            w[h] = s.s;
            rest[h] = s.rest;
          }
        };
        weigh(0);
        if (many) weigh(1);
        float mean = 0, f = 1;
        if (normalize) {
          const float total = warp_sum(w[0] + w[1]);
          f = total == 0 ? 0.0f : 1.0f / total;
          mean = warp_sum(g[0] * w[0] + g[1] * w[1]) * f;
        }
        c[0] = e[0] < 0 ? 0.0f : w[0] * f * (g[0] - mean) * rest[0];
        if (many) c[1] = e[1] < 0 ? 0.0f : w[1] * f * (g[1] - mean) * rest[1];
      }
      // Into the places of their experts.
      float* own = mine + lane * N;
#pragma unroll
      for (int i = 0; i < N; ++i) own[i] = d[i];
      __syncwarp();
      const auto place = [&](int col) { return col / R::V % 32 * N + col / (32 * R::V) * R::V + col % R::V; };
      // (A lane without a slot has a number of its own.)
      const unsigned same = __match_any_sync(~0u, e[0] < 0 ? -1 - lane : e[0]);
      if (!many && __all_sync(~0u, (same & (same - 1)) == 0)) {
        if (e[0] >= 0) mine[place(e[0])] += c[0];
      } else {  // the same expert twice, which zc_moe_route does not choose, or many slots: one after the other
        for (int j = 0; j < k; ++j) {
          if (lane == (j & 31)) {
            const int to = j >= 32 ? e[1] : e[0];
            if (to >= 0) mine[place(to)] += j >= 32 ? c[1] : c[0];
          }
          __syncwarp();
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = own[i];
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

// Rows that a warp takes at a time, so that their loads are in flight together, and warps of a CTA: what registers allow.
template <int N>
constexpr int rows_at_once() { return N <= 8 ? 4 : 1; }
template <int N>
constexpr int balance_warps() { return N <= 8 ? 32 : 16; }
constexpr int kSums = 8;  // rows of sums in shared memory
constexpr size_t kMaxParts = 152;
constexpr size_t kPartTokens = 128, kAlone = 512;  // tokens that one CTA takes by itself

struct Parts {  // of each CTA: sums, counts, tokens
  float* sums;
  int *counts, *tokens;
};
__host__ __device__ inline Parts parts_of(void* workspace, size_t ctas, size_t experts) {
  float* s = static_cast<float*>(workspace);
  int* c = reinterpret_cast<int*>(s + ctas * experts);
  return {s, c, c + ctas * experts};
}

// Counts and slopes of experts begin .. end - 1 from their sums and counts (of `tokens` tokens), and in thread 0 the CTA's
// part of the loss.  Slopes are rounded once: one division in 64 bits, which is slow, for all.
__device__ __forceinline__ float settle(const float* sums, const int* totals, int tokens, int begin, int end, int experts,
                                        int k, int* counts, float* slope) {
  __shared__ double unit;
  __shared__ float parts[ZC_MOE_MAX_EXPERTS / 32];
  if (threadIdx.x == 0) unit = tokens > 0 ? experts / (static_cast<double>(k) * tokens * tokens) : 0.0;
  __syncthreads();
  const int warps = (end - begin + 31) / 32;
  for (int w = threadIdx.x / 32; w < warps; w += blockDim.x / 32) {
    const int e = w * 32 + threadIdx.x % 32;
    float mine = 0;
    if (begin + e < end) {
      const float s = static_cast<float>(unit * totals[e]);
      counts[begin + e] = totals[e];
      slope[begin + e] = s;
      mine = s * sums[e];
    }
    mine = warp_sum(mine);
    if (threadIdx.x % 32 == 0) parts[w] = mine;
  }
  __syncthreads();
  float all = 0;
  if (threadIdx.x == 0)
    for (int w = 0; w < warps; ++w) all += parts[w];
  return all;
}

template <typename T, int N, bool Whole>
__global__ void __launch_bounds__(32 * balance_warps<N>())
    balance_kernel(const T* logits, size_t pitch, const int* ids, size_t tokens, int experts, int k, int score, float* loss,
                   int* counts, float* slope, void* workspace) {
  using R = Row<T, N, Whole>;
  constexpr int kRows = rows_at_once<N>(), kBalanceWarps = balance_warps<N>(), kBalanceThreads = 32 * kBalanceWarps;
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
  float sum[N];
  int live = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0;
  for (size_t first = begin; first < end; first += kBalanceWarps * kRows) {
    R r[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const size_t t = first + warp + u * kBalanceWarps;
      r[u].load(logits + t * pitch, t < end ? experts : 0);  // (behind the last: a row of nothing)
    }
    // The slots of these tokens.
    const size_t slots = min(end - first, static_cast<size_t>(kBalanceWarps * kRows)) * k;
    for (size_t s = threadIdx.x; s < slots; s += kBalanceThreads) {
      const int e = ids[first * k + s];
      if (e >= 0 && e < experts) atomicAdd(&found[e], 1);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float p[N], top = -kInf;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = to_float(r[u].v[i]);
        top = larger(top, p[i]);
      }
      top = warp_max(top);
      if (top == -kInf) continue;
      ++live;
      const float m = score == ZC_SCORE_SOFTMAX ? top : fminf(top, 0.0f);
      float total = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p[i] = score == ZC_SCORE_SOFTMAX ? expf(p[i] - m) : scaled_sigmoid(p[i], m).s;
        total += p[i];
      }
      const float f = 1.0f / warp_sum(total);
#pragma unroll
      for (int i = 0; i < N; ++i) sum[i] += p[i] * f;
    }
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
    const float all = settle(sums, found, rows, 0, experts, experts, k, counts, slope);
    if (threadIdx.x == 0) *loss = all;
  } else if (threadIdx.x == 0) {
    parts.tokens[blockIdx.x] = rows;
  }
}

// The CTAs' parts added: one cluster, each of its CTAs a share of the experts, for every expert several threads that
// read at the same time.
constexpr int kSettleThreads = 1024, kSettleCtas = 8;
__global__ void __launch_bounds__(kSettleThreads) __cluster_dims__(kSettleCtas, 1, 1)
    settle_kernel(void* workspace, int ctas, int experts, int k, float* loss, int* counts, float* slope) {
  __shared__ float sums[kSettleThreads];
  __shared__ int totals[kSettleThreads], live[32];
  __shared__ float losses[kSettleCtas];
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // (waited for before the first CTA's memory is used)
  wait_for_previous();
  let_next_start();
  const Parts parts = parts_of(workspace, ctas, experts);
  const int each = (experts + kSettleCtas - 1) / kSettleCtas, rank = blockIdx.x;
  const int begin = min(experts, rank * each), end = min(experts, begin + each);
  const int readers = min(32, kSettleThreads / each), reader = threadIdx.x / each, e = begin + threadIdx.x % each;
  float s = 0;
  int c = 0, n = 0;
  if (reader < readers && e < end) {
#pragma unroll 8
    for (int b = reader; b < ctas; b += readers) {
      s += parts.sums[static_cast<size_t>(b) * experts + e];
      c += parts.counts[static_cast<size_t>(b) * experts + e];
    }
  }
  if (threadIdx.x < ctas) n = parts.tokens[threadIdx.x];
  sums[threadIdx.x] = s;
  totals[threadIdx.x] = c;
  n = __reduce_add_sync(~0u, n);
  if (threadIdx.x % 32 == 0) live[threadIdx.x / 32] = n;
  __syncthreads();
  int tokens = 0;
  for (int w = 0; w < kSettleThreads / 32; ++w) tokens += live[w];
  if (threadIdx.x < each) {
    for (int r = 1; r < readers; ++r) {
      s += sums[r * each + threadIdx.x];
      c += totals[r * each + threadIdx.x];
    }
  }
  __syncthreads();
  if (threadIdx.x < each) {
    sums[threadIdx.x] = s;
    totals[threadIdx.x] = c;
  }
  __syncthreads();
  const float all = settle(sums, totals, tokens, begin, end, experts, k, counts, slope);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (threadIdx.x == 0) {  // into the first CTA
    const auto at = static_cast<uint32_t>(__cvta_generic_to_shared(&losses[rank]));
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.f32 [a], %1;\n\t}" ::"r"(at),
                 "f"(all)
                 : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && threadIdx.x == 0) {
    float sum = 0;
    for (int i = 0; i < kSettleCtas; ++i) sum += losses[i];
    *loss = sum;
  }
}

size_t balance_ctas(size_t tokens) {
  const size_t n = tokens <= kAlone ? 1 : (tokens + kPartTokens - 1) / kPartTokens;
  return n > kMaxParts ? kMaxParts : n;
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
  const size_t ctas = (s.tokens + kTokenWarps - 1) / kTokenWarps, most = static_cast<size_t>(dev.sm_count) * kGradCtas;
  return by_type(s.type, [&](auto t) {
    using T = decltype(t);
    return by_shape<T>(s.experts, {logits, d_logits}, {pitch, d_pitch}, [&](auto n, auto whole) {
      constexpr int N = decltype(n)::value;
      return launch(ZC_KERNEL_MOE_ROUTE_GRAD, route_grad_kernel<T, N, decltype(whole)::value>,
                    static_cast<unsigned>(ctas < most ? ctas : most), 32 * kTokenWarps, 0, stream, d_weights, ids, d_loss, slope,
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
      return launch(ZC_KERNEL_MOE_BALANCE, balance_kernel<T, decltype(n)::value, decltype(whole)::value>, ctas,
                    32 * balance_warps<decltype(n)::value>(),
                    sizeof(float) * (kSums + 1) * s.experts, stream, static_cast<const T*>(logits), pitch, ids, s.tokens,
                    s.experts, s.k, s.score, loss, counts, slope, workspace);
    });
  });
  if (err != cudaSuccess || ctas == 1) return err;
  return launch(ZC_KERNEL_MOE_BALANCE, settle_kernel, kSettleCtas, kSettleThreads, 0, stream, workspace, ctas, s.experts, s.k, loss,
                counts, slope);
}

}  // namespace ex
}  // namespace zc
