// ex_int4.cu -- weights in 4 bits: rounding them, and the values that they stand for.
//
// Bound by DRAM where rows are whole 16-byte vectors (16 x 2048 x 7168: bfloat16 98 us, 6.0 TB/s, fp32 181, 5.9; values in
// bfloat16 87, 6.8, in fp32 158, 6.7).  Unaligned rows: 4 x 2047 x 7167 in bfloat16 47 us, in fp32 72.
//
// A warp takes one record, 16 rows x 128 columns: lane 4 g + t holds columns 8 (t + 4 c), c = 0 .. 3, of rows g and
// g + 8, so that four lanes read 64 neighbouring values and the lanes of a row share its group's scale by two
// exchanges.  The record wants the columns 32 t .. 32 t + 31 in lane 4 g + t: the four words of a row's lanes are
// turned over by exchanges, and a lane writes 16 bytes.
#include "ex_int4.cuh"

#include <type_traits>

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

// Eight neighbouring values of a row as they lie in memory; zeros past its end.
template <typename T>
struct Eight {
  static constexpr int kVectors = 8 * sizeof(T) / 16, kEach = 16 / sizeof(T);
  uint4 v[kVectors];

  template <bool Aligned>
  __device__ __forceinline__ void load(const T* row, size_t col, size_t cols) {
    if (Aligned) {
#pragma unroll
      for (int i = 0; i < kVectors; ++i) v[i] = load_if(row + col + i * kEach, col + i * kEach < cols);
    } else if constexpr (sizeof(T) == 2) {
      // Put together from the two aligned vectors that hold it.  (4 x 2047 x 7167 47 us, and 63 value by value; fp32, which
      // has three for two, 82 and 72.)
      const unsigned shift = low4(row + col);
      const uint8_t *at = reinterpret_cast<const uint8_t*>(row + col) - shift, *end = reinterpret_cast<const uint8_t*>(row + cols);
      const uint4 a = load_if(at, at < end), b = load_if(at + 16, at + 16 < end && shift != 0);
      Pack<T, 16> p;
      p.raw = shift_bytes<true>(a, b, shift);
      if (col + 8 > cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j >= cols) p.v[j] = from_float<T>(0.0f);
      }
      v[0] = p.raw;
    } else {
      Pack<T, 16> p[kVectors];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j / kEach].v[j % kEach] = col + j < cols ? row[col + j] : from_float<T>(0.0f);
#pragma unroll
      for (int i = 0; i < kVectors; ++i) v[i] = p[i].raw;
    }
  }
  __device__ __forceinline__ float value(int j) const {
    Pack<T, 16> p;
    p.raw = v[j / kEach];
    return to_float(p.v[j % kEach]);
  }
  // The largest magnitude so far, as bits: a whole word, or two halves next to each other.
  __device__ __forceinline__ uint32_t largest(uint32_t so_far) const {
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        so_far = sizeof(T) == 2 ? __vmaxu2(so_far, w[j] & 0x7FFF7FFFu) : max(so_far, w[j] & 0x7FFFFFFFu);
    }
    return so_far;
  }
};

// The smallest bfloat16 value s >= a / 7 (7 s is exact in fp32, so the comparison decides it); 1 for a = 0.
__device__ __forceinline__ float scale_of(float a) {
  if (a == 0) return 1.0f;
  uint32_t b = __float_as_uint(__fdiv_rn(a, 7.0f)) & 0xFFFF0000u;
  if (7.0f * __uint_as_float(b) < a) b += 0x10000u;
  return __uint_as_float(b);
}

// x / s rounded to nearest, ties to even, plus 8, in the last bits of an fp32 number above 2^23.
constexpr float kRound = 12582912.0f + 8.0f;
constexpr uint32_t kRoundBits = 0x4B400000u;
// Values of at most 11 bits: x / s is a half (on its way to 7 / 2) exactly or by 2^-13 at least not (with x = X 2^a and s = S 2^b,
// S < 256, the difference is a multiple of 2^-4 / 2 S where x is not small), so x times the rounded reciprocal, whose
// error is below 2^-21, is first rounded to a multiple of 2^-15, which is the half then.
__device__ __forceinline__ uint32_t quotient_bits(float x, float inverse) {
  return __float_as_uint(fmaf(x, inverse, 384.0f) - 384.0f + kRound);
}
// Any x: x - q s is exact next to a tie, and says which side it is on.
__device__ __forceinline__ uint32_t quotient_bits(float x, float s, float inverse) {
  float q = rintf(x * inverse);
  const float rest = fmaf(-q, s, x), twice = fabsf(rest) + fabsf(rest);
  if (twice > s || (twice == s && (static_cast<int>(q) & 1))) q += copysignf(1.0f, rest);
  return __float_as_uint(q + kRound);
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
  Eight<T> x[2][4];  // all of the lane's loads in flight together
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t r = tile * kInt4Rows + 8 * h + g;
    const T* row = w + (group * s.n + (r < s.n ? r : 0)) * s.k;
#pragma unroll
    for (int c = 0; c < 4; ++c) x[h][c].template load<Aligned>(row, block * kInt4Group + 8 * (t + 4 * c), r < s.n ? s.k : 0);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t bits = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) bits = x[h][c].largest(bits);
    if (sizeof(T) == 2) bits = max(bits & 0xFFFFu, bits >> 16);
#pragma unroll
    for (int d = 1; d < 4; d *= 2) bits = max(bits, __shfl_xor_sync(~0u, bits, d));
    const float amax = std::is_same_v<T, __half> ? __half2float(__ushort_as_half(static_cast<unsigned short>(bits)))
                                                 : __uint_as_float(sizeof(T) == 2 ? bits << 16 : bits);
    uint32_t words[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
    float scale = __uint_as_float(0x7FC00000u);
    if (amax < __builtin_inff()) {  // else a group with an infinity or a NaN
      scale = scale_of(amax);
      // (The reciprocal of a very small scale would overflow: both are lifted, which is exact.)
      const float lift = scale < 0x1p-100f ? 0x1p64f : 1.0f, up = scale * lift, inverse = 1.0f / up;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // (What the numbers' upper bits add up to is taken off at the end.)
        uint32_t word = 0u - kRoundBits * 0x11111111u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = x[h][c].value(j);
          if (!std::is_same_v<T, __half>) v *= lift;
          word += (sizeof(T) == 2 ? quotient_bits(v, inverse) : quotient_bits(v, up, inverse)) << place(j);
        }
        words[c] = word;
      }
    }
    turn(words);
    reinterpret_cast<uint4*>(to)[32 * h + lane] = make_uint4(words[0], words[1], words[2], words[3]);
    if (t == 0) scales[record * kInt4Rows + 8 * h + g] = __float2bfloat16_rn(scale);
  }
}

// How a row of the result may be written: by 32 bytes, a whole sector of the L2 (by halves fp32 values of
// 16 x 2048 x 7168 took 236 us where they take 158); by 16; or value by value, neighbouring values by neighbouring
// lanes, after a turn through shared memory (4 x 2047 x 7167 in bfloat16: 221 us without it, 29 with it).
enum Width { kByValue, kBy16, kBy32 };

template <typename T, int By>
__global__ void __launch_bounds__(32 * kRecordWarps)
    int4_values_kernel(const uint8_t* values, const __nv_bfloat16* scales, size_t count, Int4Shape s, T* out) {
  // (A row's values and 16 bytes, so that rows start in different banks.)
  __shared__ __align__(16) T turned[By == kByValue ? kRecordWarps : 1][8][kInt4Group + 16 / sizeof(T)];
  const int warp = threadIdx.x / 32;
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
    constexpr int kEach = 16 / sizeof(T), kVectors = 8 / kEach;
    T* row = out + (group * s.n + r) * s.k;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const size_t col = block * kInt4Group + 8 * (t + 4 * c);
      Pack<T, 16> p[kVectors];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p[j / kEach].v[j % kEach] = from_float<T>(scale * static_cast<float>(static_cast<int>(words[c] >> place(j) & 15) - 8));
      if constexpr (By == kByValue) {
#pragma unroll
        for (int i = 0; i < kVectors; ++i) *reinterpret_cast<uint4*>(&turned[warp][g][8 * (t + 4 * c) + i * kEach]) = p[i].raw;
      } else if constexpr (By == kBy32) {
        const uint4 &a = p[0].raw, &b = p[1].raw;
        if (r < s.n && col < s.k)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + col), "r"(a.x), "r"(a.y), "r"(a.z),
                       "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                       : "memory");
      } else {
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
          if (r < s.n && col + i * kEach < s.k) *reinterpret_cast<uint4*>(row + col + i * kEach) = p[i].raw;
      }
    }
    if constexpr (By == kByValue) {
      __syncwarp();
      for (int i = 0; i < 8; ++i) {
        const size_t at = tile * kInt4Rows + 8 * h + i;
        if (at >= s.n) break;
        T* to = out + (group * s.n + at) * s.k + block * kInt4Group;
#pragma unroll
        for (int j = lane; j < kInt4Group; j += 32)
          if (block * kInt4Group + j < s.k) to[j] = turned[warp][i][j];
      }
      __syncwarp();
    }
  }
}

template <typename F>
cudaError_t by_type(int type, F f) {
  if (type == ZC_TYPE_BF16) return f(__nv_bfloat16());
  if (type == ZC_TYPE_FP16) return f(__half());
  return f(0.0f);
}

unsigned ctas_of(size_t records) { return static_cast<unsigned>((records + kRecordWarps - 1) / kRecordWarps); }

}  // namespace

cudaError_t launch_int4_quantize(const void* w, int type, size_t groups, const Int4Shape& s, uint8_t* values,
                                 __nv_bfloat16* scales, cudaStream_t stream) {
  const size_t count = groups * s.records();
  const bool whole = whole_vectors(type_bytes(type), s.k, {w}, {});
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    return launch(ZC_KERNEL_INT4_WEIGHT, whole ? int4_quantize_kernel<T, true> : int4_quantize_kernel<T, false>, ctas_of(count),
                  32 * kRecordWarps, 0, stream, static_cast<const T*>(w), count, s, values, scales);
  });
}

cudaError_t launch_int4_values(const uint8_t* values, const __nv_bfloat16* scales, size_t groups, const Int4Shape& s,
                               int type, void* out, cudaStream_t stream) {
  const size_t count = groups * s.records();
  const bool whole = whole_vectors(type_bytes(type), s.k, {out}, {});
  const bool sectors = (reinterpret_cast<uintptr_t>(out) | s.k * type_bytes(type)) % 32 == 0;
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    auto* kernel = int4_values_kernel<T, kByValue>;
    if (whole) kernel = int4_values_kernel<T, kBy16>;
    if constexpr (sizeof(T) == 4)
      if (sectors) kernel = int4_values_kernel<T, kBy32>;
    return launch(ZC_KERNEL_INT4_VALUES, kernel, ctas_of(count), 32 * kRecordWarps, 0, stream, values, scales, count, s,
                  static_cast<T*>(out));
  });
}

}  // namespace ex
}  // namespace zc
