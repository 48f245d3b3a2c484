// ex_quantize.cu -- rows, columns of row groups, and weights rounded to 8 bits in blocks of 128.
// Bound by HBM: each input value is read once, into registers, where its block's largest
// magnitude is found and the values are rounded, and each 8-bit value is written once.
#include <initializer_list>

#include "ex_fp8.cuh"

namespace zc {
namespace ex {
namespace {

// Eight consecutive values of a row as they lie in memory.
template <typename T>
union Raw8 {
  uint4 q[sizeof(T) / 2];
  uint32_t w[2 * sizeof(T)];
  typename Bytes<sizeof(T)>::type bits[8];
  T v[8];
  __device__ Raw8() {}
};
// The loads of eight values, `left` of them in the row (none where left <= 0), and the values, zeros
// past them.  Vec: rows start on 16-byte boundaries; otherwise the values lie in one aligned vector
// more.  All of a thread's loads are issued before the first value is made.
template <typename T, bool Vec, bool Select = false>
struct Fetch8 {
  static constexpr int kVectors = sizeof(T) / 2 + (Vec ? 0 : 1);
  uint4 q[kVectors];
  __device__ __forceinline__ void load(const T* at, int left) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(at);
    const unsigned s = Vec ? 0 : low4(p);
    const int bytes = min(left, 8) * static_cast<int>(sizeof(T)) + static_cast<int>(s);
#pragma unroll
    for (int i = 0; i < kVectors; ++i) q[i] = load_if(p - s + 16 * i, left > 0 && 16 * i < bytes);
  }
  __device__ __forceinline__ void values(const T* at, int left, Raw8<T>& r) const {
    if constexpr (Vec) {
#pragma unroll
      for (int i = 0; i < kVectors; ++i) r.q[i] = q[i];
    } else {
      const unsigned s = low4(at);
#pragma unroll
      for (int i = 0; i + 1 < kVectors; ++i) r.q[i] = shift_bytes<Select>(q[i], q[i + 1], s);
    }
    if (left < 8)
#pragma unroll
      for (int i = 0; i < 8; ++i) r.bits[i] = i < left ? r.bits[i] : 0;
  }
};

// Magnitudes are compared as the type's own bits without the sign, which order like the values;
// Inf and NaN are the bits from kInf on.  16-bit values go two at a time.
template <typename T>
struct Bits;
template <>
struct Bits<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7F80;
  static __device__ uint32_t fp32(uint32_t m) { return m << 16; }
};
template <>
struct Bits<__half> {
  static constexpr uint32_t kInf = 0x7C00;
  static __device__ uint32_t fp32(uint32_t m) {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
  }
};
template <>
struct Bits<float> {
  static constexpr uint32_t kInf = 0x7F800000u;
  static __device__ uint32_t fp32(uint32_t m) { return m; }
};

// The largest magnitude of N vectors, value by value: word w of `m` holds that of words w (two
// values each for 16-bit types).  odd: there is an Inf or NaN among them; they are then left out.
template <typename T, int N>
__device__ __forceinline__ void magnitudes(const Raw8<T>* r, uint32_t (&m)[2 * sizeof(T)], bool& odd) {
  constexpr bool wide = sizeof(T) == 4;
  constexpr uint32_t mask = wide ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  constexpr int words = 2 * sizeof(T);
  uint32_t most = 0;
#pragma unroll
  for (int w = 0; w < words; ++w) {
    m[w] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m[w] = wide ? max(m[w], r[i].w[w] & mask) : max_u16x2(m[w], r[i].w[w] & mask);
    most = wide ? max(most, m[w]) : max_u16x2(most, m[w]);
  }
  odd = wide ? most >= Bits<T>::kInf : (most & 0xFFFFu) >= Bits<T>::kInf || most >> 16 >= Bits<T>::kInf;
  if (odd) {
#pragma unroll
    for (int w = 0; w < words; ++w) {
      m[w] = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t v = r[i].w[w] & mask;
        if (wide) {
          m[w] = max(m[w], v < Bits<T>::kInf ? v : 0u);
        } else {
          const uint32_t lo = v & 0xFFFFu, hi = v >> 16;
          m[w] = max_u16x2(m[w], (lo < Bits<T>::kInf ? lo : 0u) | (hi < Bits<T>::kInf ? hi : 0u) << 16);
        }
      }
    }
  }
}
// The largest of the words' values.
template <typename T>
__device__ __forceinline__ uint32_t largest(const uint32_t (&m)[2 * sizeof(T)]) {
  uint32_t most = m[0];
#pragma unroll
  for (int w = 1; w < static_cast<int>(2 * sizeof(T)); ++w) most = sizeof(T) == 4 ? max(most, m[w]) : max_u16x2(most, m[w]);
  return sizeof(T) == 4 ? most : max(most & 0xFFFFu, most >> 16);
}

// Four values times f rounded, the first in the low byte.  odd: there may be an Inf or NaN, which
// does not go through the saturating conversion.
template <int Fmt>
__device__ __forceinline__ uint32_t round8x4(float a, float b, float c, float d, float f, bool odd) {
  uint32_t r = round8x2(a * f, b * f, Fmt) | static_cast<uint32_t>(round8x2(c * f, d * f, Fmt)) << 16;
  if (odd) {
    const auto fix = [&](float v, int i) {
      if (!isfinite(v)) r = (r & ~(0xFFu << (8 * i))) | nonfinite8(v, Fmt) << (8 * i);
    };
    fix(a, 0);
    fix(b, 1);
    fix(c, 2);
    fix(d, 3);
  }
  return r;
}
// Eight values of a row.
template <int Fmt, typename T>
__device__ __forceinline__ uint2 round_row(const Raw8<T>& r, float f, bool odd) {
  return make_uint2(round8x4<Fmt>(to_float(r.v[0]), to_float(r.v[1]), to_float(r.v[2]), to_float(r.v[3]), f, odd),
                    round8x4<Fmt>(to_float(r.v[4]), to_float(r.v[5]), to_float(r.v[6]), to_float(r.v[7]), f, odd));
}
// Value j of eight rows.
template <int Fmt, typename T>
__device__ __forceinline__ uint2 round_column(const Raw8<T> (&r)[8], int j, float f, bool odd) {
  return make_uint2(
      round8x4<Fmt>(to_float(r[0].v[j]), to_float(r[1].v[j]), to_float(r[2].v[j]), to_float(r[3].v[j]), f, odd),
      round8x4<Fmt>(to_float(r[4].v[j]), to_float(r[5].v[j]), to_float(r[6].v[j]), to_float(r[7].v[j]), f, odd));
}

// A warp takes four blocks (one scale word) of each of R rows: lane l holds values 8l .. 8l + 7
// of the first two blocks and of the last two, so 16 lanes share a block.  A CTA's 4 R rows have
// their scale words next to each other.  With R = 4 a lane has 128 bytes of 16-bit input in flight
// (R = 8, with the registers that takes: 138 us for 102 below).
constexpr int kRowWarps = 4;  // (32768 x 7168, bf16: 102 us, 6.9 TB/s; 8 warps 108, 16 warps 117)
template <typename T, bool Vec, int Fmt, int R>
__global__ void __launch_bounds__(32 * kRowWarps) quantize_kernel(const T* x, size_t pitch, size_t rows, int cols,
                                                                  unsigned words, uint8_t* values, uint32_t* scales) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x % 32;
  const unsigned word = blockIdx.x % words;
  const size_t r0 = (static_cast<size_t>(blockIdx.x / words) * kRowWarps + threadIdx.x / 32) * R;
  const int blocks = (cols + kBlock - 1) / kBlock, wide = blocks * kBlock;
  const int c0 = static_cast<int>(word) * 4 * kBlock + lane * 8;
  Fetch8<T, Vec> in[R][2];
  const auto place = [&](int i, int h) { return x + (r0 + i) * pitch + c0 + h * 2 * kBlock; };
  const auto left = [&](int i, int h) { return r0 + i < rows ? cols - (c0 + h * 2 * kBlock) : 0; };
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) in[i][h].load(place(i, h), left(i, h));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const size_t r = r0 + i;
    if (r >= rows) break;  // the whole warp
    int s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Raw8<T> raw;
      in[i][h].values(place(i, h), left(i, h), raw);
      uint32_t words[2 * sizeof(T)];
      bool odd;
      magnitudes<T, 1>(&raw, words, odd);
      uint32_t m = largest<T>(words);
#pragma unroll
      for (int d = 8; d; d /= 2) m = max(m, __shfl_xor_sync(~0u, m, d));
      s[h] = block_exponent(Bits<T>::fp32(m), Fmt);
      const uint2 q = round_row<Fmt>(raw, inverse_scale(s[h]), odd);
      const int c = c0 + h * 2 * kBlock;
      if (c < wide) *reinterpret_cast<uint2*>(values + r * wide + c) = q;
    }
    // lanes 0 and 16 hold the exponents of blocks 0, 2 and 1, 3 (0 for a block past the last)
    const uint32_t even = (s[0] + 127) | (s[1] + 127) << 16;
    const uint32_t odd = __shfl_sync(~0u, even, 16);
    if (lane == 0) scales[word * rows + r] = even | odd << 8;
  }
}

// The scales as fp32: 2^(byte - 127), by the bits; byte 0 is the subnormal 2^-127, 255 a NaN.
__global__ void __launch_bounds__(256) scale_values_kernel(const uint32_t* scales, size_t words, float4* out) {
  let_next_start();
  wait_for_previous();
  const size_t i = blockIdx.x * size_t(256) + threadIdx.x;
  if (i >= words) return;
  const uint32_t w = scales[i];
  const auto value = [](uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
  };
  out[i] = make_float4(value(w & 255), value(w >> 8 & 255), value(w >> 16 & 255), value(w >> 24));
}

// Blocks of group g (none, and reported, where its rows are not in range).
__device__ __forceinline__ int group_blocks(const int* offsets, int g, int rows, int* status) {
  const int a = offsets ? offsets[g] : 0, z = offsets ? offsets[g + 1] : rows;
  if (a < 0 || z < a || z > rows || (g == 0 && a != 0)) {
    set_error(status, ZC_ERR_CORRUPT);
    return 0;
  }
  return (z - a + kBlock - 1) / kBlock;
}
// The sum of the values of the threads before this one (up to 32 warps, all of which call it).
__device__ __forceinline__ int sum_before(int n, int* sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int incl = n;
  for (int d = 1; d < 32; d *= 2) {
    const int u = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = incl - n;
  for (int w = 0; w < warp; ++w) before += sums[w];
  return before;
}

// block_offsets[g] = blocks of the groups before g, by one CTA of 1024 threads.
__global__ void __launch_bounds__(1024) block_offsets_kernel(const int* offsets, int rows, int groups,
                                                             int* block_offsets, int* status) {
  __shared__ int sums[32];
  let_next_start();
  wait_for_previous();
  const int g = threadIdx.x;
  const int n = g < groups ? group_blocks(offsets, g, rows, status) : 0;
  const int before = sum_before(n, sums);
  if (g < groups) block_offsets[g] = before;
  if (g == groups - 1) block_offsets[groups] = before + n;
}

// ------------------------------------------------------------------ 128 x 128 tiles
//
// 256 threads; thread (row group rg = tid / 16, column group cg = tid % 16) holds rows 8 rg .. 8 rg + 7 of
// columns 8 cg .. 8 cg + 7: a row of the tile is read as 16 neighbouring vectors.

struct TileShared {
  alignas(16) uint2 turned[kBlock * 16];  // [column][unit of 8 rows], the unit at place unit ^ (column / 8)
  uint32_t amax[8];                       // of each warp's values
};

// Eight values of each of eight rows (`rows` of them real), `left` of a row's in it.
template <typename T, bool Vec>
__device__ __forceinline__ void load_tile(const T* at, size_t pitch, int rows, int left, Raw8<T> (&raw)[8]) {
  Fetch8<T, Vec, true> in[8];  // (a warp's lanes are in two rows, which start differently)
#pragma unroll
  for (int i = 0; i < 8; ++i) in[i].load(at + i * pitch, i < rows ? left : 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) in[i].values(at + i * pitch, i < rows ? left : 0, raw[i]);
}

// The tile's transpose by way of shared memory: column c's bytes of rows 8 rg .. as one unit.  The
// places are chosen so that the 16 column groups of a store, and the 8 lanes of a load, hit
// different banks.
__device__ __forceinline__ void put_column(TileShared& s, int c, int rg, uint2 v) { s.turned[c * 16 + (rg ^ (c / 8))] = v; }
// Rows 16 i .. 16 i + 15 of column c.
__device__ __forceinline__ uint4 get_column(const TileShared& s, int c, int i) {
  const int x = c / 8;
  const uint4 v = reinterpret_cast<const uint4*>(s.turned)[c * 8 + (i ^ (x / 2))];
  return x % 2 ? make_uint4(v.z, v.w, v.x, v.y) : v;
}

// 128 rows x 64 columns a CTA, thread (row group tid / 8, column group tid % 8) with 8 x 8 values.  Bound by HBM as
// long as enough loads are in flight while other CTAs turn their tiles: 32768 x 7168, bf16, takes 113 us (6.3
// TB/s) with nine CTAs to an SM, 119 with eight, 123 with seven, 121 with ten, which spill, and 123 with CTAs of 128
// columns; rows that start anywhere, with a vector more to load for each, 88 us for 16384 x 7167 with
// six (aligned 63; six spill 8 to 16 bytes, and five CTAs of fp32 12 to 28).
//
// Inline: every CTA counts the blocks before its own, one group a thread, and the first writes
// block_offsets, which saves a launch; otherwise they come from block_offsets_kernel.  With many
// CTAs the counting costs more than the launch (8192 x 4096, 4608 CTAs: 26.6 us with the launch,
// 24.6 without; 32768 x 7168, 30,464 CTAs: 119.5 and 123).
constexpr int kColumns = 64;  // of a CTA's tile
constexpr int kColumnThreads = 128;
constexpr int kInlineGroups = kColumnThreads;
constexpr size_t kInlineCtas = 8192;

// The tile's transpose by way of shared memory, as for TileShared.
struct ColumnShared {
  alignas(16) uint2 turned[kColumns * 16];   // [column][unit of 8 rows], the unit at place unit ^ 2 (column / 8)
  alignas(16) uint32_t amax[16][kColumns];   // 16-bit types: two columns a word
  float inverse[kColumns];
};
template <typename T, bool Vec, int Fmt, bool Inline>
__global__ void __launch_bounds__(kColumnThreads, sizeof(T) == 4 ? (Vec ? 5 : 4) : Vec ? 9 : 6)
    quantize_columns_kernel(const T* x, size_t pitch, int rows, int cols, int groups, const int* offsets, int capacity,
                            uint8_t* values, uint8_t* scales, int* block_offsets, int* status) {
  __shared__ ColumnShared s;
  __shared__ int first, last;  // this block's rows
  __shared__ int sums[kColumnThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x, cg = tid % 8, rg = tid / 8;
  const int c = blockIdx.y * kColumns + cg * 8;
  if (tid == 0) first = last = 0;
  let_next_start();
  wait_for_previous();
  const auto take = [&](int g, int b0) {  // this block is the group's, whose first one is b0
    const long long a = (offsets ? offsets[g] : 0) + static_cast<long long>(b - b0) * kBlock;
    const int z = offsets ? offsets[g + 1] : rows;
    first = static_cast<int>(a);
    last = static_cast<int>(min(static_cast<long long>(z), a + kBlock));
  };
  if (Inline) {
    const int n = tid < groups ? group_blocks(offsets, tid, rows, status) : 0;
    const int b0 = sum_before(n, sums);
    if (b0 <= b && b < b0 + n) take(tid, b0);
    if (b == 0 && blockIdx.y == 0) {
      if (tid < groups) block_offsets[tid] = b0;
      if (tid == groups - 1) block_offsets[groups] = b0 + n;
    }
  } else {
    __syncthreads();
    for (int g = tid; g < groups; g += kColumnThreads) {
      const int b0 = block_offsets[g];
      if (b0 <= b && b < block_offsets[g + 1]) take(g, b0);  // (a group with bad starts has no blocks)
    }
  }
  __syncthreads();
  const long long r0 = static_cast<long long>(first) + rg * 8;
  Raw8<T> raw[8];
  load_tile<T, Vec>(x + r0 * pitch + c, pitch, static_cast<int>(min(8ll, last - r0)), cols - c, raw);
  constexpr int words = 2 * sizeof(T);  // of eight columns
  uint32_t most[words];
  bool odd;
  magnitudes<T, 8>(raw, most, odd);
#pragma unroll
  for (int w = 0; w < words; w += 4)
    *reinterpret_cast<uint4*>(&s.amax[rg][cg * words + w]) = make_uint4(most[w], most[w + 1], most[w + 2], most[w + 3]);
  __syncthreads();
  if (tid < kColumns) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      m = max(m, sizeof(T) == 4 ? s.amax[i][tid] : reinterpret_cast<const unsigned short*>(s.amax[i])[tid]);
    const int e = block_exponent(Bits<T>::fp32(m), Fmt);
    s.inverse[tid] = inverse_scale(e);
    const size_t row = static_cast<size_t>(blockIdx.y) * kColumns + tid;
    if (row < static_cast<size_t>(cols)) {
      scales[scale_at(row, b, cols)] = static_cast<uint8_t>(e + 127);
      if (b == capacity - 1)
        for (int q = capacity; q % 4; ++q) scales[scale_at(row, q, cols)] = 127;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    s.turned[(cg * 8 + j) * 16 + (rg ^ 2 * cg)] = round_column<Fmt>(raw, j, s.inverse[cg * 8 + j], odd);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int column = i * 16 + tid / 8, part = tid % 8;
    const size_t row = static_cast<size_t>(blockIdx.y) * kColumns + column;
    if (row < static_cast<size_t>(cols))
      reinterpret_cast<uint4*>(values + (row * capacity + b) * kBlock)[part] =
          reinterpret_cast<const uint4*>(s.turned)[column * 8 + (part ^ (column / 8))];
  }
}

// One scale for the tile; its rows are written from registers, its transpose through shared memory
// (16 matrices of 4096 x 7168, bf16, both written: 297 us, 6.3 TB/s).  Of the tile's 64 values a thread, aligned
// 16-bit ones spill 8 bytes at four CTAs to an SM, unaligned ones 88 to 116 at three, unaligned fp32 16 to 20 at two.
template <typename T, bool Vec, int Fmt>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : Vec ? 4 : 3)
    quantize_weight_kernel(const T* w, int rows, int cols, uint8_t* values, uint8_t* scales, uint8_t* values_t,
                           uint8_t* scales_t) {
  __shared__ TileShared s;
  let_next_start();
  wait_for_previous();
  const int rb = (rows + kBlock - 1) / kBlock, cb = (cols + kBlock - 1) / kBlock;
  const int bc = blockIdx.x, br = blockIdx.y, tid = threadIdx.x, cg = tid % 16, rg = tid / 16;
  const size_t g = blockIdx.z;
  const int c = bc * kBlock + cg * 8;
  w += g * rows * cols;
  const int r0 = br * kBlock + rg * 8;
  Raw8<T> raw[8];
  load_tile<T, Vec>(w + static_cast<size_t>(r0) * cols + c, cols, min(8, rows - r0), cols - c, raw);
  uint32_t words[2 * sizeof(T)];
  bool odd;
  magnitudes<T, 8>(raw, words, odd);
  uint32_t m = __reduce_max_sync(~0u, largest<T>(words));
  if (tid % 32 == 0) s.amax[tid / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s.amax[i]);
  const int e = block_exponent(Bits<T>::fp32(m), Fmt);
  const float f = inverse_scale(e);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < rows)
      *reinterpret_cast<uint2*>(values + ((g * rows + r0 + i) * cb + bc) * kBlock + cg * 8) = round_row<Fmt>(raw[i], f, odd);
  // the block's scale for each of its rows (and, behind the last block, the word's empty bytes)
  const auto put_scales = [&](uint8_t* to, int n, int block_row, int b, int blocks) {
    to += g * ((blocks + 3) / 4) * 4 * n;
    const int row = block_row * kBlock + tid;
    if (tid < kBlock && row < n) {
      to[scale_at(row, b, n)] = static_cast<uint8_t>(e + 127);
      if (b == blocks - 1)
        for (int q = blocks; q % 4; ++q) to[scale_at(row, q, n)] = 127;
    }
  };
  put_scales(scales, rows, br, bc, cb);
  if (values_t == nullptr) return;
  put_scales(scales_t, cols, bc, br, rb);
#pragma unroll
  for (int j = 0; j < 8; ++j) put_column(s, cg * 8 + j, rg, round_column<Fmt>(raw, j, f, odd));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int column = i * 32 + tid / 8, part = tid % 8;
    const int row = bc * kBlock + column;
    if (row < cols)
      reinterpret_cast<uint4*>(values_t + ((g * cols + row) * rb + br) * kBlock)[part] = get_column(s, column, part);
  }
}

// The type, whether 16-byte loads reach every row, and the format, as template arguments.
template <typename F>
cudaError_t variant(int type, bool vec, int fmt, F&& f) {
  using std::integral_constant;
  const auto with_fmt = [&](auto t, auto v) {
    return fmt == ZC_FP8_E4M3 ? f(t, v, integral_constant<int, ZC_FP8_E4M3>{})
                              : f(t, v, integral_constant<int, ZC_FP8_E5M2>{});
  };
  const auto with_vec = [&](auto t) {
    return vec ? with_fmt(t, std::true_type{}) : with_fmt(t, std::false_type{});
  };
  return type == ZC_TYPE_FP32 ? with_vec(float{}) : type == ZC_TYPE_FP16 ? with_vec(__half{}) : with_vec(__nv_bfloat16{});
}

bool vector_rows(const void* x, size_t pitch, int type) {
  return (reinterpret_cast<uintptr_t>(x) | pitch * type_bytes(type)) % 16 == 0;
}

}  // namespace

size_t column_blocks(size_t rows, int groups) {
  return rows / kBlock + (rows < static_cast<size_t>(groups) ? rows : static_cast<size_t>(groups));
}

cudaError_t launch_quantize(const void* x, size_t pitch, int type, size_t rows, size_t cols, int fmt, uint8_t* values,
                            uint8_t* scales, cudaStream_t stream) {
  const size_t words = ceil_div(cols, 4 * kBlock);
  return variant(type, vector_rows(x, pitch, type), fmt, [&](auto t, auto vec, auto f) {
    using T = decltype(t);
    const auto go = [&](auto per_warp) {
      constexpr int R = per_warp();
      return launch(ZC_KERNEL_FP8_ROWS, quantize_kernel<T, vec(), f(), R>,
                    static_cast<unsigned>(ceil_div(rows, kRowWarps * R) * words), 32 * kRowWarps, 0, stream,
                    static_cast<const T*>(x), pitch, rows, static_cast<int>(cols), static_cast<unsigned>(words), values,
                    reinterpret_cast<uint32_t*>(scales));
    };
    // four rows a warp once that still gives every SM a few CTAs; one row a warp below
    return ceil_div(rows, kRowWarps * 4) * words >= 2048 ? go(std::integral_constant<int, vec() ? 4 : 2>{})
                                                         : go(std::integral_constant<int, 1>{});
  });
}

cudaError_t launch_scale_values(const void* scales, size_t words, float* out, cudaStream_t stream) {
  return launch(ZC_KERNEL_FP8_SCALES, scale_values_kernel, static_cast<unsigned>(ceil_div(words, 256)), 256, 0, stream,
                static_cast<const uint32_t*>(scales), words, reinterpret_cast<float4*>(out));
}

cudaError_t launch_quantize_columns(const void* x, size_t pitch, int type, size_t rows, size_t cols, int groups,
                                    const int* offsets, int fmt, uint8_t* values, uint8_t* scales, int* block_offsets,
                                    int* status, cudaStream_t stream) {
  const size_t capacity = column_blocks(rows, groups);
  const bool inline_groups =
      capacity > 0 && groups <= kInlineGroups && capacity * ceil_div(cols, kColumns) <= kInlineCtas;
  if (!inline_groups) {
    const cudaError_t err = launch(ZC_KERNEL_FP8_COLUMNS, block_offsets_kernel, 1, 1024, 0, stream, offsets,
                                   static_cast<int>(rows), groups, block_offsets, status);
    if (err != cudaSuccess || capacity == 0) return err;
  }
  const dim3 grid(static_cast<unsigned>(capacity), static_cast<unsigned>(ceil_div(cols, kColumns)));
  return variant(type, vector_rows(x, pitch, type), fmt, [&](auto t, auto vec, auto f) {
    using T = decltype(t);
    return launch(ZC_KERNEL_FP8_COLUMNS,
                  inline_groups ? quantize_columns_kernel<T, vec(), f(), true>
                                : quantize_columns_kernel<T, vec(), f(), false>,
                  grid, kColumnThreads, 0, stream, static_cast<const T*>(x), pitch, static_cast<int>(rows),
                  static_cast<int>(cols), groups, offsets, static_cast<int>(capacity), values, scales, block_offsets,
                  status);
  });
}

cudaError_t launch_quantize_weight(const void* w, int type, int groups, size_t rows, size_t cols, int fmt,
                                   uint8_t* values, uint8_t* scales, uint8_t* values_t, uint8_t* scales_t,
                                   cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(ceil_div(cols, kBlock)), static_cast<unsigned>(ceil_div(rows, kBlock)),
                  static_cast<unsigned>(groups));
  return variant(type, vector_rows(w, cols, type), fmt, [&](auto t, auto vec, auto f) {
    using T = decltype(t);
    return launch(ZC_KERNEL_FP8_WEIGHT, quantize_weight_kernel<T, vec(), f()>, grid, 256, 0, stream,
                  static_cast<const T*>(w), static_cast<int>(rows), static_cast<int>(cols), values, scales, values_t,
                  scales_t);
  });
}

}  // namespace ex
}  // namespace zc
