// ex_route_grad.cu -- the gradient of a router's weights and of its balance loss with respect to the logits.
//
// With g the gradients of a token's weights, times scale:
//   softmax of the chosen   d_j = w_j (g_j - sum g w)
//   sigmoids over their sum d_j = w_j (1 - s_j) (g_j - sum g w)
//   sigmoids                d_j = s_j (1 - s_j) g_j
//   softmax of the row      d_i = p_i (g_i - sum g p), g_i the sum over the slots of expert i
// and of the balance loss  d_i = d_loss p_i (slope_i - sum slope p), times 1 - s_i for sigmoids.
// What belongs to chosen experts goes through a row in shared memory, by column (by lane, eight lanes met in a bank where a
// lane has 32 values: 8192 x 1000 20.9 us, now 7.2), so that a row is written once and whole.  Bound by instructions and
// latency: 16384 x 256, eight chosen, the weights' alone 5.1 to 5.3 us (fp32: 17 MB written, 2.6 us at the copy rate), the
// balance loss's alone 6.8 in bfloat16, both 9.6; 32768 x 64 in fp32 4.2 and 7.4.  Softmax of the row: 16384 x 256 10.0 to 10.1, with the
// loss 10.5 in fp32 and 11.1 in bfloat16; 32768 x 64 6.2 and 6.6; 8192 x 1000 22.4 and 23.6.
#include "ex_router.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kWarps = 8;

// Dense: the balance loss or a softmax over the row takes part, so that all of a row is read; else only the chosen logits.
// Slots: the weights' gradients do.
template <typename R, bool Dense>
constexpr int ctas() { return R::N > 8 ? 1 : Dense ? 4 : 8; }  // on an SM at a time

// The part of a row's gradient that all of it takes part in: d_i = p_i (a_i - (sum a p + others)), others(top) what chosen
// experts add to the sum, before its division.  `top` and `factor` are the row's largest logit and one over its scores' sum.
template <typename R, typename F>
__device__ __forceinline__ void whole_row(const R& r, const float (&a)[R::N], bool softmax, F others, float (&d)[R::N], float& top,
                                          float& factor) {
  constexpr int N = R::N, W = R::W;
  float v[N], rest[N], sum = 0, dot = 0;
  top = -kInf;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = to_float(r.v[i]);
    top = larger(top, v[i]);
  }
  top = row_max<W>(top);
  const float m = top == -kInf ? 0.0f : softmax ? top : fminf(top, 0.0f);  // (a row of padding: scores of 0)
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
  dot += others(top);
  const float total = row_sum<W>(sum);
  factor = total == 0 ? 0.0f : __fdividef(1.0f, total);
  const float inner = row_sum<W>(dot) * factor;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    d[i] *= factor * (a[i] - inner);
    if (!softmax) d[i] *= rest[i];
    if (v[i] == -kInf) d[i] = 0;
  }
}

template <typename R, bool Dense, bool Slots>
__global__ void __launch_bounds__(32 * kWarps, (ctas<R, Dense>()))
    route_grad_kernel(const float* d_weights, const int* ids, const float* d_loss, const float* slope, const typename R::T* logits,
                      size_t pitch, size_t tokens, int experts, int k, int score, int normalize, float scale, typename R::T* d_logits,
                      size_t d_pitch) {
  using T = typename R::T;
  constexpr int N = R::N, W = R::W;
  __shared__ __align__(16) float rows[Slots ? 32 * kWarps * N : 1];  // by column
  wait_for_previous();
  let_next_start();
  const int lane = R::lane();
  float* mine = rows + (threadIdx.x - lane) * N;  // of the token's lanes
  const bool softmax = score == ZC_SCORE_SOFTMAX, whole = Dense && Slots && softmax && !normalize,
             many = W == 32 && k > 32;
  const float loss = d_loss != nullptr ? *d_loss : 0.0f;
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = Dense && slope != nullptr && R::column(i) < experts ? loss * slope[R::column(i)] : 0.0f;

  // What a token needs is asked for while the one before it is at work: its row where all of it is read, and the slots
  // of this lane, lane and lane + 32.
  R ahead;
  int id[2] = {-1, -1};
  float dw[2] = {0, 0};
  const auto ask = [&](size_t t) {
    if (Dense) ahead.load(logits + t * pitch, t < tokens ? experts : 0);
    if (Slots) {
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
  constexpr int kTokens = 32 / W * kWarps;  // of a CTA at a time
  const size_t step = static_cast<size_t>(gridDim.x) * kTokens;
  size_t t = static_cast<size_t>(blockIdx.x) * kTokens + threadIdx.x / W;
  ask(t);
  // (A warp goes on while it has a token: its first is the one that ends last.)
  for (; t - threadIdx.x % 32 / W < tokens; t += step) {
    const T* row = logits + t * pitch;
    // A slot without an expert has x = -infinity, e = -1 and g = 0; so has, below, one that the token may not use.
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
    if (Dense)
      whole_row(r, a, softmax, [&](float largest) {
        if (!whole) return 0.0f;
        // (Asked of x, not of e, which still names experts that the token may not use: their g may be anything.)
        return (x[0] == -kInf ? 0.0f : g[0] * expf(x[0] - largest)) + (x[1] == -kInf ? 0.0f : g[1] * expf(x[1] - largest));
      }, d, top, factor);
    if (Slots) {
      float c[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (x[h] == -kInf) e[h] = -1, g[h] = 0;
      if (whole) {
        c[0] = e[0] < 0 ? 0.0f : g[0] * expf(x[0] - top) * factor;
        if (many) c[1] = e[1] < 0 ? 0.0f : g[1] * expf(x[1] - top) * factor;
      } else {
        const float first = normalize ? row_max<W>(larger(e[0] < 0 ? -kInf : x[0], e[1] < 0 ? -kInf : x[1])) : 0.0f;
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
          const float total = slots_sum<W>(w[0] + w[1], k), dot = slots_sum<W>(g[0] * w[0] + g[1] * w[1], k);
          f = total == 0 ? 0.0f : __fdividef(1.0f, total);
          mean = dot * f;
        }
        c[0] = e[0] < 0 ? 0.0f : w[0] * f * (g[0] - mean) * rest[0];
        if (many) c[1] = e[1] < 0 ? 0.0f : w[1] * f * (g[1] - mean) * rest[1];
      }
      // Into the places of their experts.
#pragma unroll
      for (int i = 0; i < N; ++i) mine[R::column(i)] = d[i];
      __syncwarp();
      // (A lane without a slot has a number of its own, and so has each token of a warp.)
      const int token = threadIdx.x % 32 / W;
      const unsigned same = __match_any_sync(~0u, e[0] < 0 ? -1 - lane - token * W : e[0] * (32 / W) + token);
      if (!many && __all_sync(~0u, (same & (same - 1)) == 0)) {
        if (e[0] >= 0) mine[e[0]] += c[0];
      } else {  // the same expert twice, which zc_moe_route does not choose, or many slots: one after the other
        for (int j = 0; j < k; ++j) {
          if (lane == (j & (W - 1))) {
            const bool second = W == 32 && j >= 32;
            const int to = second ? e[1] : e[0];
            if (to >= 0) mine[to] += second ? c[1] : c[0];
          }
          __syncwarp();
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = mine[R::column(i)];
      __syncwarp();
    }
    R out;
#pragma unroll
    for (int i = 0; i < N; ++i) out.v[i] = from_float<T>(d[i]);
    out.store(d_logits + t * d_pitch, t < tokens ? experts : 0);
  }
}

// Where rows are long, slots few and tokens many, a warp has the slots of 32 >> log_slots tokens in its lanes at once,
// 1 << log_slots lanes for each, and then works on the tokens' rows one after the other.  (A token at a time, with all lanes
// idle but those of its slots, eight chosen of 256 in fp32: 16384 tokens 7.5 us instead of 5.2, 4096 3.4 and 3.0, 3000 the
// same; but 2048 2.7 and 2.9, 777 2.5 and 2.9: from 20 tokens for each SM on.)  Not for a softmax over the whole row, whose
// slots want the row's sum first.
constexpr int kMostShared = 16;  // slots of a token

template <typename R, bool Dense>
constexpr int shared_ctas() { return R::N > 8 ? Dense ? 1 : 4 : Dense ? 4 : 8; }

template <typename R, bool Dense>
__global__ void __launch_bounds__(32 * kWarps, (shared_ctas<R, Dense>()))
    shared_grad_kernel(const float* d_weights, const int* ids, const float* d_loss, const float* slope, const typename R::T* logits,
                       size_t pitch, size_t tokens, int experts, int k, int log_slots, int score, int normalize, float scale,
                       typename R::T* d_logits, size_t d_pitch) {
  constexpr int N = R::N;
  static_assert(R::W == 32);
  __shared__ __align__(16) float rows[32 * kWarps * N];  // by column
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, slots = 1 << log_slots, together = 32 >> log_slots;
  const int which = lane >> log_slots, j = lane & (slots - 1);  // of the tokens, and of its slots
  const bool softmax = score == ZC_SCORE_SOFTMAX;
  float* mine = rows + 32 * N * warp;
  const float loss = Dense ? *d_loss : 0.0f;
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = Dense && R::column(i) < experts ? loss * slope[R::column(i)] : 0.0f;
  int id = -1;
  float dw = 0;
  const auto ask = [&](size_t t) {
    id = -1;
    if (j < k && t < tokens) {
      id = ids[t * k + j];
      dw = d_weights[t * k + j];
    }
  };
  const size_t step = static_cast<size_t>(gridDim.x) * kWarps * together;
  size_t first = (static_cast<size_t>(blockIdx.x) * kWarps + warp) * together;
  R ahead;
  ask(first + which);
  if (Dense) ahead.load(logits + first * pitch, first < tokens ? experts : 0);
  for (; first < tokens; first += step) {
    // A slot without an expert, or one that the token may not use, has e = -1.
    float g = 0, x = -kInf;
    int e = -1;
    if (id >= 0 && id < experts) {
      x = to_float(logits[(first + which) * pitch + id]);
      g = scale * dw;
      if (x != -kInf) e = id;
    }
    ask(first + step + which);
    float top = normalize ? x : 0.0f;
    if (normalize)
      for (int d = 1; d < slots; d *= 2) top = larger(top, __shfl_xor_sync(~0u, top, d));
    float w = 0, rest = 1;
    if (e >= 0) {
      if (softmax) {
        w = expf(x - top);
      } else {
        const Sigmoid s = scaled_sigmoid(x, fminf(top, 0.0f));
        w = s.s;
        rest = s.rest;
      }
    } else {
      g = 0;
    }
    float mean = 0, f = 1;
    if (normalize) {
      const float total = slots_sum<32>(w, slots), dot = slots_sum<32>(g * w, slots);
      f = total == 0 ? 0.0f : __fdividef(1.0f, total);
      mean = dot * f;
    }
    const float c = e < 0 ? 0.0f : w * f * (g - mean) * rest;
    const unsigned same = __match_any_sync(~0u, e < 0 ? -1 - lane : e * 32 + which);
    const bool twice = __any_sync(~0u, (same & (same - 1)) != 0);  // which zc_moe_route does not choose
    for (int s = 0; s < together && first + s < tokens; ++s) {
      float d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = 0;
      if (Dense) {
        const R r = ahead;
        const size_t t = s + 1 < together ? first + s + 1 : first + step;
        ahead.load(logits + t * pitch, t < tokens ? experts : 0);
        float largest, factor;
        whole_row(r, a, softmax, [](float) { return 0.0f; }, d, largest, factor);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) mine[R::column(i)] = d[i];
      __syncwarp();
      if (!twice) {
        if (which == s && e >= 0) mine[e] += c;
      } else {
        for (int q = 0; q < k; ++q) {  // one after the other
          if (which == s && j == q && e >= 0) mine[e] += c;
          __syncwarp();
        }
      }
      __syncwarp();
      R out;
#pragma unroll
      for (int i = 0; i < N; ++i) out.v[i] = from_float<typename R::T>(mine[R::column(i)]);
      __syncwarp();
      out.store(d_logits + (first + s) * d_pitch, experts);
    }
  }
}

}  // namespace

cudaError_t launch_route_grad(const RouterShape& s, const float* d_weights, const int* ids, const float* d_loss,
                              const float* slope, const void* logits, size_t pitch, void* d_logits, size_t d_pitch,
                              const DeviceInfo& dev, cudaStream_t stream) {
  const bool dense = slope != nullptr || (s.score == ZC_SCORE_SOFTMAX && !s.normalize);
  const bool narrow = d_weights == nullptr || s.k <= lanes_of(s.experts);
  const bool whole = s.score == ZC_SCORE_SOFTMAX && !s.normalize;
  if (d_weights != nullptr && !whole && s.k <= kMostShared && !(narrow && lanes_of(s.experts) < 32) &&
      s.tokens >= 20 * static_cast<size_t>(dev.sm_count))
    return by_row(s.type, s.experts, false, {logits, d_logits}, {pitch, d_pitch}, [&](auto row) {
      using R = decltype(row);
      using T = typename R::T;
      const auto go = [&](auto all) {
        if constexpr (R::W < 32) {
          return cudaErrorInvalidValue;  // (rows share no warp here)
        } else {
          constexpr bool kDense = decltype(all)::value;
          const int log_slots = s.k <= 4 ? 2 : s.k <= 8 ? 3 : 4;
          const size_t each = static_cast<size_t>(32 >> log_slots) * kWarps, needed = (s.tokens + each - 1) / each;
          const size_t most = static_cast<size_t>(dev.sm_count) * shared_ctas<R, kDense>();
          return launch(ZC_KERNEL_MOE_ROUTE_GRAD, shared_grad_kernel<R, kDense>,
                        static_cast<unsigned>(needed < most ? needed : most), 32 * kWarps, 0, stream, d_weights, ids, d_loss, slope,
                        static_cast<const T*>(logits), pitch, s.tokens, s.experts, s.k, log_slots, s.score, s.normalize, s.scale,
                        static_cast<T*>(d_logits), d_pitch);
        }
      };
      return dense ? go(std::true_type()) : go(std::false_type());
    });
  return by_row(s.type, s.experts, narrow, {logits, d_logits}, {pitch, d_pitch}, [&](auto row) {
    using R = decltype(row);
    using T = typename R::T;
    const auto go = [&](auto all, auto chosen) {
      constexpr bool kDense = decltype(all)::value;
      const size_t each = 32 / R::W * kWarps, needed = (s.tokens + each - 1) / each;
      const size_t most = static_cast<size_t>(dev.sm_count) * ctas<R, kDense>();
      return launch(ZC_KERNEL_MOE_ROUTE_GRAD, route_grad_kernel<R, kDense, decltype(chosen)::value>,
                    static_cast<unsigned>(needed < most ? needed : most), 32 * kWarps, 0, stream, d_weights, ids, d_loss, slope,
                    static_cast<const T*>(logits), pitch, s.tokens, s.experts, s.k, s.score, s.normalize, s.scale,
                    static_cast<T*>(d_logits), d_pitch);
    };
    if (!d_weights) return go(std::true_type(), std::false_type());
    return dense ? go(std::true_type(), std::true_type()) : go(std::false_type(), std::true_type());
  });
}

}  // namespace ex
}  // namespace zc
