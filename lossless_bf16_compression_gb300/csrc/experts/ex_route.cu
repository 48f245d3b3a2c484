// ex_route.cu -- a router's choice: the k largest logits of each token, and their weights.
//
// The largest of a row is found k times: each lane offers the largest of its own that is left, the row's largest wins,
// and the lane that had it goes on to its next one.  Bound by instructions (integer comparisons and moves): one token 2.2 us,
// 32768 x 64 in fp32, eight chosen, 5.7, 16384 x 256 in bfloat16 6.7, in fp32 8.2 (values of 16 bits, many of them equal, 10.2).
#include "ex_router.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kWarps = 8;

// ------------------------------------------------------------------ the order of logits
//
// A logit as an unsigned integer in its own order: a NaN of either sign above all, -0 equal to 0 (an addition of 0 makes
// them one), -infinity below all.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kNone = 0x007FFFFFu;  // of -infinity

// The keys that are searched for a row's largest logits; no two of a row are equal.
//   16 bits: the logit's order above 0xFFFF - column: equal logits go by column.
//   fp32: the order with its last bits (eight for a row of 256) given to the column.  Two logits that differ in those bits
//   alone may come in the wrong order: that is seen, and the row is searched again.  (With three bits, for the lane's register
//   alone, and the lane by a vote, it happened less, but every row took longer: 16384 x 256 10.5 us.)
template <typename R>
struct Keys {
  using T = typename R::T;
  static constexpr int N = R::N;
  static constexpr bool kExact = sizeof(T) == 2;
  static constexpr uint32_t kLow = kExact ? 0xFFFFu : R::W * N - 1;
  static constexpr uint32_t kLeast = sizeof(T) == 2 && std::is_same_v<T, __half> ? 0x03FFFFFFu : kNone;
  uint32_t k[N];

  __device__ __forceinline__ explicit Keys(const R& row) {
    if constexpr (kExact) {
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
      for (int i = 0; i < N; ++i) k[i] = (ordered(row.v[i]) & ~kLow) | (kLow - R::column(i));
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
  // A lane's keys in descending order (eight of them: a network of 19 comparisons; more: as they are).
  static constexpr bool kSorted = N == 8;
  __device__ __forceinline__ void order(int a, int b) {
    const uint32_t x = k[a], y = k[b];
    k[a] = max(x, y);
    k[b] = min(x, y);
  }
  __device__ __forceinline__ void sort() {
    if constexpr (kSorted) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) order(i, i + 1);
      order(0, 2), order(1, 3), order(4, 6), order(5, 7);
      order(1, 2), order(5, 6);
      order(0, 4), order(1, 5), order(2, 6), order(3, 7);
      order(2, 4), order(3, 5);
      order(1, 2), order(3, 4), order(5, 6);
    }
  }
  __device__ __forceinline__ uint32_t largest() const {
    if (kSorted) return k[0];
    uint32_t best = k[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = max(best, k[i]);
    return best;
  }
  // The largest after m, which was this lane's (0: there is none).
  __device__ __forceinline__ uint32_t after(uint32_t m) {
    if constexpr (kSorted) {
#pragma unroll
      for (int i = 0; i < N - 1; ++i) k[i] = k[i + 1];
      k[N - 1] = 0;
      return k[0];
    } else {  // (distances from m - 1 wrap around for those that are not below m)
      uint32_t least = m - 1 - k[0];
#pragma unroll
      for (int i = 1; i < N; ++i) least = min(least, m - 1 - k[i]);
      return least < m ? m - 1 - least : 0u;
    }
  }
};

// ------------------------------------------------------------------ the choice

// The k largest of a row whose search by keys was not sure, one after the other by value and column: slot lane (and
// lane + 32) gets its column.
template <typename R>
__device__ __noinline__ int2 search_again(const typename R::T* logits, int experts, int k) {
  constexpr int N = R::N;
  const int lane = R::lane();
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
    const uint32_t m = row_max<R::W>(best);
    const int first = row_min<R::W>(best == m ? at : experts);
    if (lane == j % R::W && m > kNone) {
      if (j >= R::W) e.y = first;
      else e.x = first;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (R::column(i) == first) key[i] = 0;
  }
  return e;
}

// Slots: lane j of a token's has slot j, and slot j + 32 where a token has a whole warp.
template <typename R>
__global__ void __launch_bounds__(32 * kWarps)
    route_kernel(const typename R::T* logits, size_t pitch, size_t tokens, int experts, int k, int score, int normalize,
                 float scale, float* weights, int* ids) {
  using K = Keys<R>;
  constexpr int N = R::N, W = R::W;
  wait_for_previous();
  let_next_start();
  const int lane = R::lane();
  const size_t t = (static_cast<size_t>(blockIdx.x) * (32 * kWarps) + threadIdx.x) / W;
  const bool real = t < tokens;  // (the others of a warp take part in its exchanges)
  const typename R::T* from = logits + (real ? t : 0) * pitch;
  R row;
  row.load(from, real ? experts : 0);
  K keys(row);
  keys.sort();

  uint32_t got[2] = {0, 0}, best = keys.largest();  // the keys in this lane's slots; its largest one that is left
  if (K::kSorted && k <= N) {
    // (As many of a lane's keys go up as may still be asked for; the last may stay behind and look like one too near.)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j == k) break;
      const uint32_t m = row_max<W>(keys.k[0]);
      if (lane == j) got[0] = m;
      if (keys.k[0] == m) {
#pragma unroll
        for (int i = 0; i < N - 1 && i < N - j; ++i) keys.k[i] = keys.k[i + 1];
      }
    }
    best = keys.k[0];
  } else {
    for (int j = 0; j < k; ++j) {
      const uint32_t m = row_max<W>(best);
      if (W == 32 && m <= K::kLeast) break;
      if (lane == (j & (W - 1))) {
        if (W == 32 && j >= 32) got[1] = m;
        else got[0] = m;
      }
      if (best == m) best = keys.after(m);
    }
  }
  const bool many = W == 32 && k > 32, softmax = score == ZC_SCORE_SOFTMAX;
  int e[2];  // the columns
#pragma unroll
  for (int h = 0; h < 2; ++h) e[h] = got[h] > K::kLeast ? static_cast<int>(K::kLow - (got[h] & K::kLow)) : -1;
  float x[2];  // (the chosen logits again, from the L1)
  const auto gather = [&] {
    x[0] = e[0] >= 0 ? to_float(from[e[0]]) : -kInf;
    x[1] = many && e[1] >= 0 ? to_float(from[e[1]]) : -kInf;
  };
  gather();
  if (!K::kExact) {
    // Slots whose keys are near have to be in order by their logits, and the largest key that is left must not be near.
    const uint32_t left = row_max<W>(best);
    bool unsure = false;
    const auto check = [&](int slot, uint32_t key, float v, uint32_t next_key, float next) {
      if (slot >= k || key <= K::kLeast) return;
      unsure |= slot == k - 1 ? (key ^ left) <= K::kLow : (key ^ next_key) <= K::kLow && !(v >= next);
    };
    uint32_t next_key = __shfl_down_sync(~0u, got[0], 1, W);
    float next = __shfl_down_sync(~0u, x[0], 1, W);
    if (many) {
      const uint32_t first_key = __shfl_sync(~0u, got[1], 0);
      const float first = __shfl_sync(~0u, x[1], 0);
      if (lane == 31) next_key = first_key, next = first;
    }
    check(lane, got[0], x[0], next_key, next);
    if (many) check(lane + 32, got[1], x[1], __shfl_down_sync(~0u, got[1], 1), __shfl_down_sync(~0u, x[1], 1));
    if (__any_sync(~0u, unsure)) {
      const int2 again = search_again<R>(from, real ? experts : 0, k);
      e[0] = again.x;
      e[1] = again.y;
      gather();
    }
  }

  const float top = __shfl_sync(~0u, x[0], 0, W);
  const auto value = [&](int h) {
    return e[h] < 0 ? 0.0f : softmax ? expf(x[h] - top) : scaled_sigmoid(x[h], normalize ? fminf(top, 0.0f) : 0.0f).s;
  };
  const float w0 = value(0), w1 = many ? value(1) : 0.0f;
  float total = 1.0f;
  if (normalize) {
    total = slots_sum<W>(w0 + w1, k);
  } else if (softmax) {
    total = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) total += expf(to_float(row.v[i]) - top);
    total = row_sum<W>(total);
  }
  const float f = scale * __fdividef(1.0f, total);
  if (real && lane < k) {
    weights[t * k + lane] = e[0] < 0 ? 0.0f : f * w0;
    ids[t * k + lane] = e[0];
  }
  if (many && real && lane + 32 < k) {
    weights[t * k + lane + 32] = e[1] < 0 ? 0.0f : f * w1;
    ids[t * k + lane + 32] = e[1];
  }
}

}  // namespace

cudaError_t launch_route(const RouterShape& s, const void* logits, size_t pitch, float* weights, int* ids,
                         cudaStream_t stream) {
  return by_row(s.type, s.experts, s.k <= lanes_of(s.experts), {logits}, {pitch}, [&](auto row) {
    using R = decltype(row);
    const size_t tokens = 32 / R::W * kWarps;  // of a CTA
    return launch(ZC_KERNEL_MOE_ROUTE, route_kernel<R>, static_cast<unsigned>((s.tokens + tokens - 1) / tokens), 32 * kWarps, 0,
                  stream, static_cast<const typename R::T*>(logits), pitch, s.tokens, s.experts, s.k, s.score, s.normalize,
                  s.scale, weights, ids);
  });
}

}  // namespace ex
}  // namespace zc
