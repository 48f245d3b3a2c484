// ex_int4.cu -- weights in 4 bits: rounding them, and the values that they stand for.
//
// A warp takes one record, 16 rows x 128 columns: lane 4 g + t holds columns 8 (t + 4 c), c = 0 .. 3, of rows g and
// g + 8, so that four lanes read 64 neighbouring values and the lanes of a row share its group's scale by two
// exchanges.  The record wants the columns 32 t .. 32 t + 31 in lane 4 g + t: the four words of a row's lanes are
// turned over by exchanges, and a lane writes 16 bytes.
#include "ex_int4.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kRecordWarps = 8;

// Word w of lane t (of four neighbouring lanes) becomes word t of lane w.
__device__ __forceinline__ void turn(uint32_t (&w)[4]) {
  const int t = threadIdx.x % 4;
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    const bool up = t & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
      const uint32_t give = up ? w[i] : w[i + d];
      const uint32_t got = __shfl_xor_sync(~0u, give, d);
      if (up) w[i] = got;
      else w[i + d] = got;
    }
  }
}

// The bits of q + 8 of weight j in its word.
__host__ __device__ constexpr int place(int j) { return 4 * (j / 2 + 4 * (j % 2)); }

// Eight neighbouring values of a row, as fp32; zeros past its end.
template <typename T, bool Aligned>
__device__ __forceinline__ void read8(const T* row, size_t col, size_t cols, float (&v)[8]) {
  if (Aligned) {
    constexpr int kVectors = 8 * sizeof(T) / 16;
    Pack<T, 16> p[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
      p[i].raw = load_if(row + col + i * (16 / sizeof(T)), col + i * (16 / sizeof(T)) < cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_float(p[j / (16 / sizeof(T))].v[j % (16 / sizeof(T))]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + j < cols ? to_float(row[col + j]) : 0.0f;
  }
}

// The smallest bfloat16 value s >= a / 7 (7 s is exact in fp32, so the comparison decides it); 1 for a = 0.
__device__ __forceinline__ float scale_of(float a) {
  if (a == 0) return 1.0f;
  uint32_t b = __float_as_uint(__fdiv_rn(a, 7.0f)) & 0xFFFF0000u;
  if (7.0f * __uint_as_float(b) < a) b += 0x10000u;
  return __uint_as_float(b);
}

// x / s rounded to nearest, ties to even, exactly: x - q s is exact next to a tie, and says which side it is on.
__device__ __forceinline__ int round_quotient(float x, float s, float inverse) {
  float q = rintf(x * inverse);
  const float rest = fmaf(-q, s, x), twice = fabsf(rest) + fabsf(rest);
  if (twice > s || (twice == s && (static_cast<int>(q) & 1))) q += copysignf(1.0f, rest);
  return static_cast<int>(q);
}

template <typename T, bool Aligned>
__global__ void __launch_bounds__(32 * kRecordWarps)
    int4_quantize_kernel(const T* w, size_t count, Int4Shape s, uint8_t* values, __nv_bfloat16* scales) {
  wait_for_previous();
  let_next_start();
  const size_t record = static_cast<size_t>(blockIdx.x) * kRecordWarps + threadIdx.x / 32;
  if (record >= count) return;
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const size_t blocks = s.blocks(), tiles = s.tiles();
  const size_t block = record % blocks, tile = record / blocks % tiles, group = record / blocks / tiles;
  uint8_t* to = values + record * kInt4Record;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t r = tile * kInt4Rows + 8 * h + g;
    const size_t cols = r < s.n ? s.k : 0;
    const T* row = w + (group * s.n + (r < s.n ? r : 0)) * s.k;
    float v[4][8], amax = 0;
    bool odd = false;  // an infinity or a NaN
#pragma unroll
    for (int c = 0; c < 4; ++c) read8<T, Aligned>(row, block * kInt4Group + 8 * (t + 4 * c), cols, v[c]);
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        odd |= !(fabsf(v[c][j]) < __builtin_inff());
        amax = fmaxf(amax, fabsf(v[c][j]));
      }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
      amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
      odd |= __shfl_xor_sync(~0u, odd, d);
    }
    uint32_t words[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
    float scale = __uint_as_float(0x7FC00000u);
    if (!odd) {
      scale = scale_of(amax);
      // (The reciprocal of a very small scale would overflow: both are lifted, which is exact.)
      const float lift = scale < 0x1p-100f ? 0x1p64f : 1.0f, up = scale * lift, inverse = 1.0f / up;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        words[c] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          words[c] |= static_cast<uint32_t>(round_quotient(v[c][j] * lift, up, inverse) + 8) << place(j);
      }
    }
    turn(words);
    reinterpret_cast<uint4*>(to)[32 * h + lane] = make_uint4(words[0], words[1], words[2], words[3]);
    if (t == 0) scales[record * kInt4Rows + 8 * h + g] = __float2bfloat16_rn(scale);
  }
}

template <typename T, bool Aligned>
__global__ void __launch_bounds__(32 * kRecordWarps)
    int4_values_kernel(const uint8_t* values, const __nv_bfloat16* scales, size_t count, Int4Shape s, T* out) {
  wait_for_previous();
  let_next_start();
  const size_t record = static_cast<size_t>(blockIdx.x) * kRecordWarps + threadIdx.x / 32;
  if (record >= count) return;
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const size_t blocks = s.blocks(), tiles = s.tiles();
  const size_t block = record % blocks, tile = record / blocks % tiles, group = record / blocks / tiles;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t r = tile * kInt4Rows + 8 * h + g;
    const uint4 q = reinterpret_cast<const uint4*>(values + record * kInt4Record)[32 * h + lane];
    const float scale = __bfloat162float(scales[record * kInt4Rows + 8 * h + g]);
    uint32_t words[4] = {q.x, q.y, q.z, q.w};
    turn(words);
    if (r < s.n) {
      T* row = out + (group * s.n + r) * s.k;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const size_t col = block * kInt4Group + 8 * (t + 4 * c);
        Pack<T, 16> p[8 * sizeof(T) / 16];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          p[j / (16 / sizeof(T))].v[j % (16 / sizeof(T))] =
              from_float<T>(scale * static_cast<float>(static_cast<int>(words[c] >> place(j) & 15) - 8));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          constexpr int kEach = 16 / sizeof(T);
          if (Aligned) {
            if (j % kEach == 0 && col + j < s.k) *reinterpret_cast<uint4*>(row + col + j) = p[j / kEach].raw;
          } else if (col + j < s.k) {
            row[col + j] = p[j / kEach].v[j % kEach];
          }
        }
      }
    }
  }
}

template <typename F>
cudaError_t by_type(int type, bool aligned, F f) {
  const auto go = [&](auto t) {
    return aligned ? f(t, std::integral_constant<bool, true>()) : f(t, std::integral_constant<bool, false>());
  };
  if (type == ZC_TYPE_BF16) return go(__nv_bfloat16());
  if (type == ZC_TYPE_FP16) return go(__half());
  return go(float());
}

unsigned ctas_of(size_t records) { return static_cast<unsigned>((records + kRecordWarps - 1) / kRecordWarps); }

}  // namespace

cudaError_t launch_int4_quantize(const void* w, int type, size_t groups, const Int4Shape& s, uint8_t* values,
                                 __nv_bfloat16* scales, cudaStream_t stream) {
  const size_t count = groups * s.records();
  return by_type(type, whole_vectors(type_bytes(type), s.k, {w}, {}), [&](auto t, auto aligned) {
    using T = decltype(t);
    return launch(ZC_KERNEL_INT4_WEIGHT, int4_quantize_kernel<T, decltype(aligned)::value>, ctas_of(count),
                  32 * kRecordWarps, 0, stream, static_cast<const T*>(w), count, s, values, scales);
  });
}

cudaError_t launch_int4_values(const uint8_t* values, const __nv_bfloat16* scales, size_t groups, const Int4Shape& s,
                               int type, void* out, cudaStream_t stream) {
  const size_t count = groups * s.records();
  return by_type(type, whole_vectors(type_bytes(type), s.k, {out}, {}), [&](auto t, auto aligned) {
    using T = decltype(t);
    return launch(ZC_KERNEL_INT4_VALUES, int4_values_kernel<T, decltype(aligned)::value>, ctas_of(count),
                  32 * kRecordWarps, 0, stream, values, scales, count, s, static_cast<T*>(out));
  });
}

}  // namespace ex
}  // namespace zc
