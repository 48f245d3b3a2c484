// ex_rows.cu -- rows to their places in the order by expert and back, with weights, and the
// gradients.  The order is a permutation known from the sort, so every kernel here is driven by
// tokens: a token's row is read (or written) once and its k sorted rows once each, which is all
// the traffic there is, and every sum over j runs inside one thread in slot order (no atomics).
// Bound by HBM when there are many tokens, by two dependent loads (position, then row) when there
// are few; so a thread asks for the rows of eight slots before it uses the first.  16384 tokens x 8 x
// 7168, bf16: dispatch 321 us (6.6 TB/s; with the sort), combine 298 (7.1), combine's gradient 578 (6.9, part of
// it from the L2); one token, calls from Python back to back: 5.5, 3.8 and 6.6 us.
#include <initializer_list>

#include "ex_common.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kMaxThreads = 256;
// Smaller CTAs keep an SM's loads further apart: combine of 16384 x 8 x 7168 with 256 threads 365
// us, with 128 336 us; of 4999 x 6 x 2050 53 and 41 us.
constexpr int kCombineThreads = 128;

// A position that may be used as an address; reported otherwise.
__device__ __forceinline__ bool in_range(int p, size_t slots, int* status) {
  if (p >= 0 && static_cast<size_t>(p) < slots) return true;
  set_error(status, ZC_ERR_CORRUPT);
  return false;
}

// How a row's vectors are shared out: to `parts` CTAs of `threads`, one vector a thread.
struct Cut {
  unsigned parts, threads;
};
Cut cut_row(size_t vecs, unsigned most) {
  const unsigned parts = static_cast<unsigned>((vecs + most - 1) / most);
  const unsigned each = static_cast<unsigned>((vecs + parts - 1) / parts);
  return {parts, (each + 31) / 32 * 32};
}
// Vectors of a row; one more where a row may start inside a vector.
size_t row_vectors(size_t bytes, bool aligned) { return (bytes + 15) / 16 + (aligned ? 0 : 1); }

// 16 bytes of a token's row, vector c of it, as a thread holds them to store them in rows that start
// elsewhere: a vector of such a row holds bytes of this vector and of the one before.
template <bool Aligned, int E, bool Select = false>
struct Held {
  uint4 before, here;
  __device__ __forceinline__ void load(const uint8_t* row, int c, int bytes) {
    if (Aligned) {
      here = load_if(row + 16 * c, 16 * c < bytes);
      return;
    }
    const unsigned s = low4(row);
    uint4 v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int at = 16 * (c + i - 1) - static_cast<int>(s);
      v[i] = load_if(row + at, at > -16 && at < bytes && (i < 2 || s));
    }
    before = shift_bytes<Select>(v[0], v[1], s);
    here = shift_bytes<Select>(v[1], v[2], s);
  }
  // The bytes that lie in vector c of a row at `row`, and where they start in the row.
  __device__ __forceinline__ uint4 for_row(const uint8_t* row, int c, int* from) const {
    const unsigned s = Aligned ? 0 : low4(row);
    *from = 16 * c - static_cast<int>(s);
    return s ? shift_bytes<Select>(before, here, 16 - s) : here;
  }
  __device__ __forceinline__ void store(uint8_t* row, int c, int bytes, bool zeros) const {
    int from;
    const uint4 v = for_row(row, c, &from);
    put16<Aligned, E>(row, from, bytes, zeros ? make_uint4(0, 0, 0, 0) : v);
  }
};

// rows[position[t, j]] = x[t].  Short rows share a CTA, one token for each threadIdx.y: it only stores,
// so what bounds them is how fast CTAs start (16384 x 2 x 1024: 28 -> 22 us; the other kernels
// lose more by giving up uniform registers for a token's positions and addresses, the combine
// gradient at that size 53 -> 84 us).
template <bool Aligned, int E>
__global__ void __launch_bounds__(kMaxThreads) dispatch_kernel(const uint8_t* x, size_t x_pitch, uint8_t* rows,
                                                               size_t rows_pitch, int bytes, unsigned parts,
                                                               size_t tokens, int k, const int* position,
                                                               const int* total, int* status) {
  let_next_start();
  const size_t t = static_cast<size_t>(blockIdx.x / parts) * blockDim.y + threadIdx.y, slots = tokens * k;
  const int c = static_cast<int>(blockIdx.x % parts * blockDim.x + threadIdx.x);
  if (t >= tokens) return;
  Held<Aligned, E> held;
  held.load(x + t * x_pitch, c, bytes);  // x does not come from the sort
  wait_for_previous();
  const int kept = *total;
  int next = position[t * k];  // (asked for a slot ahead of the stores)
  for (int j = 0; j < k; ++j) {
    const int p = next;
    if (j + 1 < k) next = position[t * k + j + 1];
    if (in_range(p, slots, status)) held.store(rows + p * rows_pitch, c, bytes, p >= kept);
  }
}

// Sort and dispatch of few slots in one launch: every CTA counts, for the slots of its token, the
// slots that come before them -- slots x k comparisons, shared by its threads -- so no CTA waits
// for another.  At 64 tokens x 8 that is 16 comparisons a thread.
constexpr size_t kSmallSlots = 1024;

template <typename Id, bool Aligned, int E>
__global__ void __launch_bounds__(kMaxThreads) small_dispatch_kernel(
    const Id* ids, int slots, int experts, const uint8_t* x, size_t x_pitch, uint8_t* rows, size_t rows_pitch,
    int bytes, unsigned parts, int k, int* position, int* offsets) {
  __shared__ short keys[kSmallSlots];
  __shared__ int place[ZC_MOE_MAX_K];
  __shared__ int bins[ZC_MOE_MAX_EXPERTS + 1];
  __shared__ int kept;
  let_next_start();
  wait_for_previous();
  const int t = static_cast<int>(blockIdx.x / parts), part = static_cast<int>(blockIdx.x % parts);
  const int c = part * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x), lane = threadIdx.x % 32;
  Held<Aligned, E> held;
  held.load(x + t * x_pitch, c, bytes);
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
    held.store(rows + p * rows_pitch, c, bytes, p >= kept);
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

// A warp's lanes on unaligned rows: each loads one aligned vector and takes the next one from the
// lane above it, so that as many rows are in flight as on aligned ones (without weights 4999 x 6 x 2050, fp16:
// 33 us, by two loads a lane 39; 16384 x 8 x 7167 351 and 445).  The last lane only loads.
constexpr int kTaking = 31;
__device__ __forceinline__ uint4 from_next_lane(const uint4& v) {
  return make_uint4(__shfl_down_sync(~0u, v.x, 1), __shfl_down_sync(~0u, v.y, 1), __shfl_down_sync(~0u, v.z, 1),
                    __shfl_down_sync(~0u, v.w, 1));
}
// The aligned vector that holds byte `from` of a row.
__device__ __forceinline__ uint4 vector_at(const uint8_t* row, int from, int bytes, bool on) {
  const int at = from - static_cast<int>(low4(row + from));
  return load_if(row + at, on && at > -16 && at < bytes);
}

// out[t] = sum over j of weights[t, j] rows[position[t, j]].  A thread takes Tokens tokens that follow
// one another, with a share of each one's slots at a time: as many rows in flight however few slots a
// token has.
// (Nine CTAs to an SM, with weights spilling 32 to 48 bytes: 16384 x 8 x 7167 with weights 374 us; measured before
// the positions were checked ahead of the loads: nine 381, without the bound on registers 394, ten 423.)
template <typename T, bool Aligned, int Tokens, bool Weighted>
__global__ void __launch_bounds__(kCombineThreads, !Aligned && Tokens == 1 ? 9 : 0)
    combine_kernel(const uint8_t* rows, size_t rows_pitch, const float* weights, uint8_t* out, size_t out_pitch,
                   int bytes, unsigned parts, size_t tokens, int k, const int* position, const int* total,
                   int* status) {
  // (four tokens of one slot on unaligned rows: 80 us for 16384 x 1 x 5851 by four, 108 by eight)
  constexpr int N = 16 / sizeof(T), kBatch = !Aligned && Tokens == 4 ? 4 : 8, S = kBatch / Tokens;
  let_next_start();
  wait_for_previous();
  const size_t t0 = static_cast<size_t>(blockIdx.x / parts) * Tokens, slots = tokens * k;
  const int thread = static_cast<int>(blockIdx.x % parts * blockDim.x + threadIdx.x), lane = threadIdx.x % 32;
  const int c = Aligned ? thread : thread / 32 * kTaking + lane;
  // (on unaligned rows only whole warps leave)
  if (t0 >= tokens || (Aligned ? 16 * c >= bytes : 16 * (c - lane) >= bytes + 16)) return;
  const int kept = *total;
  // vector c of each token's row of out: its first byte in the row
  int from[Tokens];
#pragma unroll
  for (int i = 0; i < Tokens; ++i)
    from[i] = 16 * c - (Aligned ? 0 : static_cast<int>(low4(out + (t0 + i) * out_pitch)));
  float acc[Tokens][N] = {};
  for (int j0 = 0; j0 < k; j0 += S) {
    uint4 l[kBatch];
    float w[kBatch];
    int at[kBatch];
    bool here[kBatch];  // (the same for all of a warp)
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const size_t t = min(t0 + i / S, tokens - 1), s = t * k + min(j0 + i % S, k - 1);
      at[i] = position[s];
      w[i] = Weighted ? weights[s] : 1.f;
    }
    // (all reported before the first load, since none crosses an atomic: 16384 x 8 x 7168 298 us, one by one 311)
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      here[i] = j0 + i % S < k && t0 + i / S < tokens && in_range(at[i], slots, status) && at[i] < kept;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) l[i] = vector_at(rows + at[i] * rows_pitch, from[i / S], bytes, here[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!here[i]) continue;
      Pack<T, 16> v;
      v.raw = Aligned ? l[i] : shift_bytes(l[i], from_next_lane(l[i]), low4(rows + at[i] * rows_pitch + from[i / S]));
#pragma unroll
      for (int e = 0; e < N; ++e) acc[i / S][e] = fmaf(w[i], to_float(v.v[e]), acc[i / S][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < Tokens; ++i) {
    Pack<T, 16> o;
#pragma unroll
    for (int e = 0; e < N; ++e) o.v[e] = from_float<T>(acc[i][e]);
    if (t0 + i < tokens && (Aligned || lane < kTaking))
      put16<Aligned, sizeof(T)>(out + (t0 + i) * out_pitch, from[i], bytes, o.raw);
  }
}

// What holds bytes from .. from + 15 of a row of `bytes` bytes (from may lie outside it).
struct Loaded {
  uint4 a, b;
};
template <bool Aligned>
__device__ __forceinline__ Loaded fetch16(const uint8_t* row, int from, int bytes, bool on) {
  Loaded l;
  if (Aligned) {
    l.a = load_if(row + from, on && from < bytes);
  } else {
    const unsigned s = low4(row + from);
    const int at = from - static_cast<int>(s);  // of the first vector, from the row's start
    l.a = load_if(row + at, on && at > -16 && at < bytes);
    l.b = load_if(row + at + 16, on && s && at > -32 && at + 16 < bytes);
  }
  return l;
}
template <bool Aligned>
__device__ __forceinline__ uint4 settle(const Loaded& l, const uint8_t* row, int from) {
  return Aligned ? l.a : shift_bytes<true>(l.a, l.b, low4(row + from));
}

// d_rows[position[t, j]] = weights[t, j] d_out[t], d_weights[t, j] = <d_out[t], rows[...]>.  One
// CTA a token: each thread sums its vectors' products, then lanes, then warps, in a fixed order.
template <typename T, bool Aligned, int Batch>
__global__ void __launch_bounds__(kMaxThreads) combine_grad_kernel(
    const uint8_t* d_out, size_t d_out_pitch, const uint8_t* rows, size_t rows_pitch, const float* weights,
    uint8_t* d_rows, size_t d_rows_pitch, float* d_weights, int bytes, size_t tokens, int k, const int* position,
    const int* total, int* status) {
  constexpr int N = 16 / sizeof(T);
  __shared__ float sums[Batch][kMaxThreads / 32];
  let_next_start();
  wait_for_previous();
  const size_t t = blockIdx.x, slots = tokens * k;
  const int vecs = (bytes + 15) / 16 + (Aligned ? 0 : 1);
  const int kept = *total, warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int j0 = 0; j0 < k; j0 += Batch) {
    int at[Batch];
    float w[Batch], dot[Batch];
    bool ok[Batch], here[Batch];
#pragma unroll
    for (int i = 0; i < Batch; ++i) {
      const size_t s = t * k + j0 + i;
      at[i] = j0 + i < k ? position[s] : 0;
      ok[i] = j0 + i < k && in_range(at[i], slots, status);
      here[i] = ok[i] && at[i] < kept;
      w[i] = here[i] ? weights[s] : 0.f;
      dot[i] = 0.f;
    }
    for (int c = threadIdx.x; c < vecs; c += blockDim.x) {
      Held<Aligned, sizeof(T), true> held;
      held.load(d_out + t * d_out_pitch, c, bytes);
      Loaded l[Batch];
#pragma unroll
      for (int i = 0; i < Batch; ++i) l[i] = fetch16<Aligned>(rows + at[i] * rows_pitch, 16 * c, bytes, here[i]);
      const int real = (bytes - 16 * c) / static_cast<int>(sizeof(T));  // values of this vector in the row
      Pack<T, 16> d;
      d.raw = held.here;
#pragma unroll
      for (int i = 0; i < Batch; ++i) {
        if (!ok[i]) continue;
        uint8_t* to = d_rows + at[i] * d_rows_pitch;
        int from;
        Pack<T, 16> o, r;
        o.raw = held.for_row(to, c, &from);
        r.raw = settle<Aligned>(l[i], rows + at[i] * rows_pitch, 16 * c);
        if (here[i]) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            o.v[e] = from_float<T>(w[i] * to_float(o.v[e]));
            if (Aligned || e < real) dot[i] = fmaf(to_float(d.v[e]), to_float(r.v[e]), dot[i]);
          }
        } else {
          o.raw = make_uint4(0, 0, 0, 0);
        }
        put16<Aligned, sizeof(T)>(to, from, bytes, o.raw);
      }
    }
#pragma unroll
    for (int i = 0; i < Batch; ++i) {
      for (int m = 16; m; m /= 2) dot[i] += __shfl_xor_sync(~0u, dot[i], m);
      if (lane == 0) sums[i][warp] = dot[i];
    }
    __syncthreads();
    if (threadIdx.x < Batch && j0 + static_cast<int>(threadIdx.x) < k) {
      float s = 0.f;
      for (int i = 0; i < warps; ++i) s += sums[threadIdx.x][i];
      d_weights[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

template <typename F>
cudaError_t by_alignment(bool aligned, F&& f) {
  return aligned ? f(std::true_type{}) : f(std::false_type{});
}
template <typename F>
cudaError_t by_size(int type, bool aligned, F&& f) {
  return by_alignment(aligned, [&](auto a) {
    return type_bytes(type) == 4 ? f(a, std::integral_constant<int, 4>{}) : f(a, std::integral_constant<int, 2>{});
  });
}
template <typename F>
cudaError_t by_type(int type, bool aligned, F&& f) {
  return by_alignment(aligned, [&](auto a) {
    return type == ZC_TYPE_FP32 ? f(float{}, a) : type == ZC_TYPE_FP16 ? f(__half{}, a) : f(__nv_bfloat16{}, a);
  });
}

}  // namespace

cudaError_t launch_dispatch(const RowShape& s, const void* x, size_t x_pitch, void* rows, size_t rows_pitch,
                            const int* position, const int* offsets, int* status, cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const bool aligned = whole_vectors(b, s.hidden, {x, rows}, {x_pitch, rows_pitch});
  const Cut cut = cut_row(row_vectors(s.hidden * b, aligned), kMaxThreads);
  return by_size(s.type, aligned, [&](auto a, auto e) {
    const unsigned together = kMaxThreads / cut.threads;  // tokens of a CTA
    return launch(ZC_KERNEL_MOE_DISPATCH, dispatch_kernel<a(), e()>,
                  static_cast<unsigned>((s.tokens + together - 1) / together) * cut.parts,
                  dim3(cut.threads, together), 0, stream, static_cast<const uint8_t*>(x), x_pitch * b,
                  static_cast<uint8_t*>(rows), rows_pitch * b, static_cast<int>(s.hidden * b), cut.parts, s.tokens,
                  s.k, position, offsets + s.experts, status);
  });
}

bool small_dispatch(size_t slots) { return slots > 0 && slots <= kSmallSlots; }

cudaError_t launch_small_dispatch(const RowShape& s, const void* ids, int id_bytes, const void* x, size_t x_pitch,
                                  void* rows, size_t rows_pitch, int* position, int* offsets, cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const bool aligned = whole_vectors(b, s.hidden, {x, rows}, {x_pitch, rows_pitch});
  const Cut cut = cut_row(row_vectors(s.hidden * b, aligned), kMaxThreads);
  const unsigned threads = cut.threads < 64 ? 64 : cut.threads;  // at least ZC_MOE_MAX_K
  return by_size(s.type, aligned, [&](auto a, auto e) {
    const auto go = [&](auto* p) {
      using Id = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
      return launch(ZC_KERNEL_MOE_DISPATCH, small_dispatch_kernel<Id, a(), e()>,
                    static_cast<unsigned>(s.tokens) * cut.parts, threads, 0, stream, p,
                    static_cast<int>(s.tokens * s.k), s.experts, static_cast<const uint8_t*>(x), x_pitch * b,
                    static_cast<uint8_t*>(rows), rows_pitch * b, static_cast<int>(s.hidden * b), cut.parts, s.k,
                    position, offsets);
    };
    return id_bytes == 8 ? go(static_cast<const long long*>(ids)) : go(static_cast<const int*>(ids));
  });
}

cudaError_t launch_combine(const RowShape& s, const void* rows, size_t rows_pitch, const float* weights,
                           const int* position, const int* offsets, void* out, size_t out_pitch, int* status,
                           cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const bool aligned = whole_vectors(b, s.hidden, {rows, out}, {rows_pitch, out_pitch});
  const size_t vecs = row_vectors(s.hidden * b, aligned);
  const Cut cut = cut_row(aligned ? vecs : (vecs + kTaking - 1) / kTaking * 32, kCombineThreads);
  const auto go = [&](auto type, auto a, auto tokens) {
    return launch(ZC_KERNEL_MOE_COMBINE,
                  weights ? combine_kernel<decltype(type), a(), tokens(), true>
                          : combine_kernel<decltype(type), a(), tokens(), false>,
                  static_cast<unsigned>((s.tokens + tokens() - 1) / tokens()) * cut.parts, cut.threads, 0, stream,
                  static_cast<const uint8_t*>(rows), rows_pitch * b, weights, static_cast<uint8_t*>(out),
                  out_pitch * b, static_cast<int>(s.hidden * b), cut.parts, s.tokens, s.k, position,
                  offsets + s.experts, status);
  };
  return by_type(s.type, aligned, [&](auto type, auto a) {
    // few tokens: one a thread, so that they spread over the SMs
    const bool many = s.tokens * cut.parts >= 2048;
    return many && s.k <= 2   ? go(type, a, std::integral_constant<int, 4>{})
           : many && s.k <= 4 ? go(type, a, std::integral_constant<int, 2>{})
                              : go(type, a, std::integral_constant<int, 1>{});
  });
}

cudaError_t launch_combine_grad(const RowShape& s, const void* d_out, size_t d_out_pitch, const void* rows,
                                size_t rows_pitch, const float* weights, const int* position, const int* offsets,
                                void* d_rows, size_t d_rows_pitch, float* d_weights, int* status,
                                cudaStream_t stream) {
  const size_t b = type_bytes(s.type);
  const bool aligned = whole_vectors(b, s.hidden, {d_out, rows, d_rows}, {d_out_pitch, rows_pitch, d_rows_pitch});
  const size_t vecs = row_vectors(s.hidden * b, aligned);
  // A token's sums need all of its row, which the CTA's threads walk: with few tokens more threads
  // finish a row sooner (1 token x 8 x 7168: 12 us with 256, 16 with 128, 25 with 64), with many
  // fewer leave more CTAs to an SM (16384 x 2 x 1024: 41 us with 64, 53 with 128, 16384 x 8 x
  // 7168: 582 and 576).
  const unsigned most = s.tokens < 2048 ? 256 : vecs <= 256 ? 64 : 128;
  const auto go = [&](auto type, auto a, auto batch) {
    return launch(ZC_KERNEL_MOE_COMBINE_GRAD, combine_grad_kernel<decltype(type), a(), batch()>,
                  static_cast<unsigned>(s.tokens),
                  cut_row(vecs, most).threads, 0, stream, static_cast<const uint8_t*>(d_out), d_out_pitch * b,
                  static_cast<const uint8_t*>(rows), rows_pitch * b, weights, static_cast<uint8_t*>(d_rows),
                  d_rows_pitch * b, d_weights, static_cast<int>(s.hidden * b), s.tokens, s.k, position,
                  offsets + s.experts, status);
  };
  // Slots taken together: no more than there are, which leaves room for more CTAs, and two where
  // every row's vector takes two registers' worth of loads and a shift (4999 x 6 x 2050: 70 us by
  // twos, 84 by fours, 88 by eights).
  return by_type(s.type, aligned, [&](auto type, auto a) {
    if (s.k == 1) return go(type, a, std::integral_constant<int, 1>{});
    if (s.k == 2 || !a()) return go(type, a, std::integral_constant<int, 2>{});
    return s.k <= 4 ? go(type, std::true_type{}, std::integral_constant<int, 4>{})
                    : go(type, std::true_type{}, std::integral_constant<int, 8>{});
  });
}

}  // namespace ex
}  // namespace zc
