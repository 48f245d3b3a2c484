// ex_route_grad.cu -- the gradient of a router's weights and of its balance loss with respect to the logits.
//
// With g the gradients of a token's weights, times scale:
//   softmax of the chosen   d_j = w_j (g_j - sum g w)
//   sigmoids over their sum d_j = w_j (1 - s_j) (g_j - sum g w)
//   sigmoids                d_j = s_j (1 - s_j) g_j
//   softmax of the row      d_i = p_i (g_i - sum g p), g_i the sum over the slots of expert i
// and of the balance loss  d_i = d_loss p_i (slope_i - sum slope p), times 1 - s_i for sigmoids.
// What belongs to chosen experts goes through a row in shared memory, so that a row is written once and whole.  Bound by
// instructions and the exchanges' latency: 16384 x 256, eight chosen, the weights' alone 7.8 us (fp32: 17 MB written, 2.6 us
// at the copy rate), with the balance loss 11.6, 32768 x 64 5.0 and 7.1.
#include "ex_router.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kWarps = 8;

// Dense: the balance loss or a softmax over the row takes part, so that all of a row is read; else only the chosen logits.
template <typename R, bool Dense>
constexpr int ctas() { return R::N > 8 ? 1 : Dense ? 4 : 8; }  // on an SM at a time

template <typename R, bool Dense>
__global__ void __launch_bounds__(32 * kWarps, (ctas<R, Dense>()))
    route_grad_kernel(const float* d_weights, const int* ids, const float* d_loss, const float* slope, const typename R::T* logits,
                      size_t pitch, size_t tokens, int experts, int k, int score, int normalize, float scale, typename R::T* d_logits,
                      size_t d_pitch) {
  using T = typename R::T;
  constexpr int N = R::N, W = R::W;
  __shared__ __align__(16) float rows[32 * kWarps][N];  // of each lane
  wait_for_previous();
  let_next_start();
  const int lane = R::lane();
  float* own = rows[threadIdx.x];
  float* mine = rows[threadIdx.x - lane];  // of the token's lanes
  const bool softmax = score == ZC_SCORE_SOFTMAX, whole = Dense && softmax && !normalize && d_weights != nullptr, many = W == 32 && k > 32;
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
  constexpr int kTokens = 32 / W * kWarps;  // of a CTA at a time
  const size_t step = static_cast<size_t>(gridDim.x) * kTokens;
  size_t t = static_cast<size_t>(blockIdx.x) * kTokens + threadIdx.x / W;
  ask(t);
  // (A warp goes on while it has a token: its first is the one that ends last.)
  for (; t - threadIdx.x % 32 / W < tokens; t += step) {
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
    if (Dense) {
      float v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = to_float(r.v[i]);
        top = larger(top, v[i]);
      }
      top = row_max<W>(top);
      {
        const float m = top == -kInf ? 0.0f : softmax ? top : fminf(top, 0.0f);  // (a row of padding: scores of 0)
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
      for (int i = 0; i < N; ++i) own[i] = d[i];
      __syncwarp();
      const auto add = [&](int to, float v) { mine[R::lane_of(to) * N + R::place_of(to)] += v; };
      // (A lane without a slot has a number of its own, and so has each token of a warp.)
      const int token = threadIdx.x % 32 / W;
      const unsigned same = __match_any_sync(~0u, e[0] < 0 ? -1 - lane - token * W : e[0] * (32 / W) + token);
      if (!many && __all_sync(~0u, (same & (same - 1)) == 0)) {
        if (e[0] >= 0) add(e[0], c[0]);
      } else {  // the same expert twice, which zc_moe_route does not choose, or many slots: one after the other
        for (int j = 0; j < k; ++j) {
          if (lane == (j & (W - 1))) {
            const bool second = W == 32 && j >= 32;
            const int to = second ? e[1] : e[0];
            if (to >= 0) add(to, second ? c[1] : c[0]);
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
    out.store(d_logits + t * d_pitch, t < tokens ? experts : 0);
  }
}

}  // namespace

cudaError_t launch_route_grad(const RouterShape& s, const float* d_weights, const int* ids, const float* d_loss,
                              const float* slope, const void* logits, size_t pitch, void* d_logits, size_t d_pitch,
                              const DeviceInfo& dev, cudaStream_t stream) {
  const bool dense = slope != nullptr || (s.score == ZC_SCORE_SOFTMAX && !s.normalize);
  const bool narrow = d_weights == nullptr || s.k <= lanes_of(s.experts);
  return by_row(s.type, s.experts, narrow, {logits, d_logits}, {pitch, d_pitch}, [&](auto row) {
    using R = decltype(row);
    using T = typename R::T;
    const auto go = [&](auto all) {
      constexpr bool kDense = decltype(all)::value;
      const size_t each = 32 / R::W * kWarps, needed = (s.tokens + each - 1) / each;
      const size_t most = static_cast<size_t>(dev.sm_count) * ctas<R, kDense>();
      return launch(ZC_KERNEL_MOE_ROUTE_GRAD, route_grad_kernel<R, kDense>,
                    static_cast<unsigned>(needed < most ? needed : most), 32 * kWarps, 0, stream, d_weights, ids, d_loss, slope,
                    static_cast<const T*>(logits), pitch, s.tokens, s.experts, s.k, s.score, s.normalize, s.scale,
                    static_cast<T*>(d_logits), d_pitch);
    };
    return dense ? go(std::true_type()) : go(std::false_type());
  });
}

}  // namespace ex
}  // namespace zc
