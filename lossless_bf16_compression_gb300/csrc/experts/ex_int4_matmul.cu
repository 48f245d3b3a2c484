// ex_int4_matmul.cu -- the experts' products on 4-bit weights, for few rows.
//
// out[r, i] = sum over b of s[i, b] * (sum over j in b of x[r, j] q[i, j]).  Bound by the weights' bytes, or by what it
// takes to unpack them.  A warp takes 2 x 16 weight rows (a record of 1 KB for each 128 columns) and multiplies them by
// eight or sixteen columns, the rows of x, on the warp-level matrix instructions: with so few rows the tensor cores
// have time to spare (1024 products a cycle and SM by this way; the tensor-memory instructions want 128 weight rows at a
// time, too coarse for one token's experts, and the unpacked weights written to tensor or shared memory first; for many rows
// of an expert, where they would serve more columns at a time, they were not tried).  The group's scale multiplies the group's
// sum, once for 128 products.
//
// fp32 rows of x are split into three bfloat16 values that add up to them exactly, the second held 2^8 times its size and the
// third 2^16 times; they are columns of their own, added at the end.  Measured (2048 x 7168, graph replays): eight experts of 64, a row each, 15.7 to 17.8 us (59 MB, 8.7 us at the
// copy rate; 2 us of launch, 3 of finding the work and bringing x, the rest not accounted for); 64 experts, one to eight rows
// each, 96 to 100 us (485 MB: 4.9 TB/s; without the loads about 80, without unpacking and products too 24), nine to sixteen 128 to
// 132; fp32 rows, one, five and eight each, 97, 144 and 254.  A scheduler's two cycles
// for each logic operation and eight for a product make 40 us of unpacking and 25 of products (sixteen columns: 50); four
// warps, which is what the registers hold, overlap these in part.
#include <type_traits>

#include "ex_int4.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kColumnPitch = 20;  // of 16 partial sums (in fp32), free of bank conflicts
constexpr size_t kShared = 226 * 1024;

// The 16-bit type that x and the weights are multiplied in: x's own, or bfloat16 for the parts of fp32.
template <typename T>
using Form = std::conditional_t<std::is_same_v<T, __half>, __half, __nv_bfloat16>;

// d (+)= a b for 16 weight rows and eight columns, 16 values of k.
template <typename F, bool First>
__device__ __forceinline__ void multiply(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (First && std::is_same_v<F, __half>)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else if constexpr (First)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else if constexpr (std::is_same_v<F, __half>)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two times 16 bytes, 512 apart, where `on` is set; else they are as they were, and not used.
__device__ __forceinline__ void fetch_record(uint4& a, uint4& b, const void* p, int on) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %9, 0;\n\t"
               "@q ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%8];\n\t"
               "@q ld.global.L1::no_allocate.v4.u32 {%4, %5, %6, %7}, [%8 + 512];\n\t}"
               : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w), "+r"(b.x), "+r"(b.y), "+r"(b.z), "+r"(b.w)
               : "l"(p), "r"(on));
}
// 16 bits where `on` is set; else `v` is as it was.
__device__ __forceinline__ void fetch_scale(uint32_t& v, const void* p, int on) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
               : "+r"(v)
               : "l"(p), "r"(on));
}


// The eight weights of a word as pairs of 16-bit numbers, weights 2 p and 2 p + 1 in the p-th, each q / weight_unit (128 for fp32
// rows, whose second and third parts are held up to twice as large as the first).  The bits of a nibble alone, in the low
// eight bits of such a number, are one too small to be normal, u or 16 u times the smallest (2^-133 or 2^-24), and one fused
// multiply-add makes (u - 8) / weight_unit of either, exactly: five logic operations and four multiply-adds for eight weights.
// (Or'ed into the low bits of 128, with a subtraction, they took seven and four: 153 us where these take 147, 512 rows over 64
// experts at the time.)
template <typename T>
constexpr float weight_unit() { return std::is_same_v<T, __half> ? 512.0f : std::is_same_v<T, float> ? 128.0f : 64.0f; }
template <typename F>
__device__ __forceinline__ uint32_t fma_pair(uint32_t v, uint32_t times, uint32_t plus) {
  uint32_t r;
  if constexpr (std::is_same_v<F, __half>) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(times), "r"(plus));
  else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(times), "r"(plus));
  return r;
}
struct Four {
  uint32_t v[4];
};
template <typename T>
__device__ __forceinline__ Four four(uint32_t word) {
  using F = Form<T>;
  constexpr bool kHalf = std::is_same_v<T, __half>, kFloat = std::is_same_v<T, float>;
  constexpr uint32_t kLow = kHalf ? 0x78007800u : kFloat ? 0x7E807E80u : 0x7F007F00u;    // 2^15, 2^126, 2^127
  constexpr uint32_t kHigh = kHalf ? 0x68006800u : kFloat ? 0x7C807C80u : 0x7D007D00u;   // 2^11, 2^122, 2^123
  constexpr uint32_t kMinus = kHalf ? 0xA400A400u : kFloat ? 0xBD80BD80u : 0xBE00BE00u;  // -8 / 512, -8 / 128, -8 / 64
  const uint32_t up = word >> 8;
  return {fma_pair<F>(word & 0x000F000Fu, kLow, kMinus), fma_pair<F>(word & 0x00F000F0u, kHigh, kMinus),
          fma_pair<F>(up & 0x000F000Fu, kLow, kMinus), fma_pair<F>(up & 0x00F000F0u, kHigh, kMinus)};
}

// a / b of whole numbers, 0 <= a < 2^20, without the long division: the quotient's error is below a / b 2^-21, the distance
// of (a + 1/2) / b from a whole number at least 1 / 2b.
__device__ __forceinline__ int divide(int a, int b) { return static_cast<int>((a + 0.5f) * __fdividef(1.0f, b)); }

// ------------------------------------------------------------------ rows of x as columns

template <typename T>
struct Parts;
template <>
struct Parts<__nv_bfloat16> { static constexpr int n = 1; };
template <>
struct Parts<__half> { static constexpr int n = 1; };
template <>
struct Parts<float> { static constexpr int n = 3; };

// v's leading 8 significant bits, and the rest, which is exact.  An infinity or NaN has no rest.
__device__ __forceinline__ uint32_t lead(float& v) {
  const uint32_t b = __float_as_uint(v);
  const bool finite = (b & 0x7F800000u) != 0x7F800000u;
  const uint32_t top = finite ? b & 0xFFFF0000u : b & 0x007FFFFFu ? 0x7FC00000u : b;
  v = finite ? v - __uint_as_float(top) : 0.0f;
  return top >> 16;
}

// Eight neighbouring values as `Parts` vectors of eight bfloat16, each part kPartUnit^-1 times its size: so lifted a part is at
// most twice as large as the first, which fp32's largest value and the weights' unit allow, and its last bit is not below
// bfloat16's smallest number where x's is not below fp32's.  (Unlifted, x below 2^-110 lost its last bits, and large scales
// showed it.)
constexpr float kPartUnit = 0x1p-8f;
template <typename T>
__device__ __forceinline__ void split(const T (&v)[8], uint4 (&out)[Parts<T>::n]) {
  if constexpr (Parts<T>::n == 1) {
    out[0] = *reinterpret_cast<const uint4*>(v);
  } else {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_float(v[j]);
#pragma unroll
    for (int p = 0; p < Parts<T>::n; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = lead(f[2 * j]);
        w[j] = lo | lead(f[2 * j + 1]) << 16;
        f[2 * j] *= 1 / kPartUnit;
        f[2 * j + 1] *= 1 / kPartUnit;
      }
      out[p] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Puts `count` blocks of `rows` rows of x, from block `first` on, where the products read them: for each block and
// eight columns 4 x 512 bytes, in the c-th of which lane 4 g + t finds values 32 t + 8 c .. + 7 of column g (in the place of
// lane 4 (g ^ 1) + t for odd c, so that the rows that come in meet in half as many banks).  By loads and stores, four
// vectors at a time: asynchronous copies to such scattered places take longer even where there is something to do meanwhile
// (one row of 4096 x 7168 8.5 us instead of 6.9, eight rows 15.4 and 9.3, 256 rows over 16 experts 69 and 60), eight at
// a time a little longer.
constexpr int kBatch = 4;
template <typename T>
__device__ __forceinline__ void stage(const T* x, size_t pitch, int rows, int first, int count, size_t k, bool aligned,
                                      int tiles, uint4* to) {
  // A thread takes a vector of eight values of one row, or of each.
  const int vectors = count * (kInt4Group / 8);
  const int side = vectors < kThreads ? divide(kThreads, vectors) : 1;  // rows side by side
  const int row0 = side > 1 ? divide(threadIdx.x, vectors) : 0;
  for (int v = threadIdx.x - row0 * vectors; v < vectors && row0 < side; v += kThreads) {
    const size_t col = static_cast<size_t>(first) * kInt4Group + 8 * v;
    const int block = v / 16, t = v % 16 / 4, c = v % 4;
    const auto place = [&](int column) {
      return to + ((block * tiles + column / 8) * 4 + c) * 32 + ((column % 8 * 4 + t) ^ (c & 1) * 4);
    };
    constexpr int kVectors = 8 * sizeof(T) / 16, kEach = 16 / sizeof(T), kRows = kBatch / kVectors;
    const auto put_row = [&](int row, const T(&values)[8]) {
      uint4 out[Parts<T>::n];
      split<T>(values, out);
#pragma unroll
      for (int p = 0; p < Parts<T>::n; ++p) *place(row * Parts<T>::n + p) = out[p];
    };
    if (aligned) {
      for (int r = row0; r < rows; r += kRows * side) {
        alignas(16) T in[kRows][8];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int j = 0; j < kVectors; ++j)  // (past the end of the row: zeros)
            reinterpret_cast<uint4*>(in[i])[j] =
                load_if(x + (r + i * side) * pitch + col + j * kEach, col + j * kEach < k && r + i * side < rows);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (r + i * side < rows) put_row(r + i * side, in[i]);
      }
      continue;
    }
    for (int r = row0; r < rows; r += side) {
      // Each vector put together from the two aligned ones that hold it; zeros past the row's end.
      const T* from = x + r * pitch + col;
      alignas(16) T in[8];
      uint4* whole = reinterpret_cast<uint4*>(in);
      const unsigned shift = low4(from);
      const uint8_t *at = reinterpret_cast<const uint8_t*>(from) - shift, *end = reinterpret_cast<const uint8_t*>(x + r * pitch + k);
      uint4 w[kVectors + 1];
#pragma unroll
      for (int j = 0; j <= kVectors; ++j) w[j] = load_if(at + 16 * j, at + 16 * j < end && (j < kVectors || shift != 0));
#pragma unroll
      for (int j = 0; j < kVectors; ++j) whole[j] = shift_bytes<true>(w[j], w[j + 1], shift);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j >= k) in[j] = from_float<T>(0.0f);
      put_row(r, in);
    }
  }
}

struct Job {
  const void* x;
  size_t x_pitch;
  const uint8_t* values;
  const __nv_bfloat16* scales;
  const int* offsets;
  void* out;
  size_t out_pitch;
  int* status;
  Int4Shape w;
  int rows, groups, out_type;
  int room;  // for x in shared memory: blocks of eight columns
  bool aligned;
  unsigned parts_inverse, lines_inverse;  // of the CTAs, and of a pass's lines
};

__device__ __forceinline__ void put(const Job& p, size_t row, size_t col, float v) {
  const size_t at = row * p.out_pitch + col;
  if (p.out_type == ZC_TYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else if (p.out_type == ZC_TYPE_FP16) static_cast<__half*>(p.out)[at] = __float2half_rn(v);
  else static_cast<float*>(p.out)[at] = v;
}

// ------------------------------------------------------------------ passes
//
// A pass is up to `each` rows of one group, the columns that the products take at once.  A pass of more columns takes
// longer on the same weights (measured: by a third for sixteen instead of eight), so CTAs share the work by cost: 2 and
// 1 for each eight columns begun.

constexpr int cost_of(int columns) { return 2 + (columns + 7) / 8; }

struct Pass {
  int group, row, rows;
};
// In shared memory, of each group and past the last: its first row and first pass.
struct Passes {
  int *start, *first;
};
// A CTA's part of the list, in lines of all passes, one pass's after the other's; and where it begins.
struct Part {
  size_t begin, end;
  Pass pass;
  int index, line;
};

template <int kEach, int kParts>
__device__ __forceinline__ int cost_of_rows(int rows) {
  const int rest = rows % kEach;
  return rows / kEach * cost_of(kEach * kParts) + (rest ? cost_of(rest * kParts) : 0);
}
// a / b, with inverse = floor((2^32 - 1) / b): the product's upper half is the quotient or one less.
__device__ __forceinline__ unsigned quotient(unsigned a, unsigned b, unsigned inverse) {
  const unsigned q = __umulhi(a, inverse);
  return q + (a - q * b >= b);
}
__device__ __forceinline__ size_t quotient(size_t a, unsigned b, unsigned) { return a / b; }
// Of a group with `rows` rows, its first passes and cost and those of all groups: whether this CTA's part begins or ends
// in it.  U holds the cost of all lines: in 32 bits where it fits them, as long divisions take a microsecond.
template <int kEach, int kParts, typename U>
__device__ __forceinline__ void find_part(const Job& p, Part& part, int group, int row, int rows, int2 before, int2 all, int lines,
                                          bool last) {
  constexpr int kFull = cost_of(kEach * kParts);
  const U total = static_cast<U>(all.y) * lines, lower = static_cast<U>(before.y) * lines,
          upper = lower + static_cast<U>(cost_of_rows<kEach, kParts>(rows)) * lines;
  const U each = quotient(total, gridDim.x, p.parts_inverse), more = total - each * gridDim.x;  // shared out evenly
  const U begin = each * blockIdx.x + min(static_cast<U>(blockIdx.x), more), end = begin + each + (blockIdx.x < more);
  const int full = rows / kEach;
  const auto line_at = [&](U point) {  // of the group's
    const U in = point - lower, whole = static_cast<U>(full) * kFull * lines, rest = in - whole;
    if (in < whole) return in / kFull;
    const int cost = cost_of(rows % kEach * kParts);
    return static_cast<U>(full) * lines + (cost == 3 ? rest / 3 : rest / 4);
  };
  static_assert(cost_of(1) == 3 && cost_of(16) == 4);
  const size_t first = static_cast<size_t>(before.x) * lines;
  if (begin >= lower && begin < upper) {
    const U line = line_at(begin);
    const int pass = static_cast<int>(quotient(line, lines, p.lines_inverse));
    part.begin = first + line;
    part.index = before.x + pass;
    part.line = static_cast<int>(line - static_cast<U>(pass) * lines);
    part.pass = {group, row + pass * kEach, min(kEach, rows - pass * kEach)};
  }
  if (end >= lower && end < upper) part.end = first + line_at(end);
  if (last) {
    if (begin >= total) part.begin = static_cast<size_t>(all.x) * lines;
    if (end >= total) part.end = static_cast<size_t>(all.x) * lines;
  }
}
// The passes, and this CTA's part of them.  Only the warps that have groups work (of all sixteen, each instruction costs
// a scheduler eight cycles).
template <int kEach, int kParts>
__device__ __forceinline__ void find_passes(const Job& p, const Passes& s, int lines, Part& part) {
  const auto put_part = [&](int g, int row, int rows, int2 before, int2 all) {
    const bool last = g == p.groups - 1;
    s.start[g] = row;
    s.first[g] = before.x;
    if (last) s.first[g + 1] = all.x;
    if (static_cast<size_t>(all.y) * lines < (size_t(1) << 31)) find_part<kEach, kParts, unsigned>(p, part, g, row, rows, before, all, lines, last);
    else find_part<kEach, kParts, size_t>(p, part, g, row, rows, before, all, lines, last);
  };
  if (p.offsets == nullptr) {  // one group
    if (threadIdx.x == 0) {
      s.start[1] = p.rows;
      put_part(0, 0, p.rows, make_int2(0, 0), make_int2((p.rows + kEach - 1) / kEach, cost_of_rows<kEach, kParts>(p.rows)));
    }
    __syncthreads();
    return;
  }
  __shared__ int2 sums[kWarps];  // of each warp's groups: passes and cost (below 0: an offset is wrong)
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  constexpr int kGroups = (ZC_MOE_MAX_EXPERTS + kThreads - 1) / kThreads;  // of a thread, the most
  const int each = p.groups <= kThreads ? 1 : kGroups, warps = (p.groups + 32 * each - 1) / (32 * each);
  int begin[kGroups], rows[kGroups];
  int2 upto = make_int2(0, 0), mine = upto, own[kGroups];
  if (warp < warps) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = threadIdx.x * each + i;
      begin[i] = rows[i] = 0;
      if (i < each && g < p.groups) {
        const int a = p.offsets[g], z = p.offsets[g + 1];
        bad |= a < 0 || z < a || z > p.rows || (g == 0 && a != 0);
        begin[i] = a;
        rows[i] = z - a;
      }
    }
    if (bad) set_error(p.status, ZC_ERR_CORRUPT);
    bad = __any_sync(~0u, bad);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      own[i] = bad ? make_int2(0, 0) : make_int2((rows[i] + kEach - 1) / kEach, cost_of_rows<kEach, kParts>(rows[i]));
      upto.x += own[i].x;
      upto.y += own[i].y;
    }
    mine = upto;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(~0u, upto.x, d), y = __shfl_up_sync(~0u, upto.y, d);
      if (lane >= d) upto.x += x, upto.y += y;
    }
    if (lane == 31) sums[warp] = bad ? make_int2(0, -1) : upto;
    if (warps == 1) __syncwarp();
  }
  if (warps > 1) __syncthreads();
  if (warp < warps) {
    upto.x -= mine.x;
    upto.y -= mine.y;
    const int2 of = lane < warps ? sums[lane] : make_int2(0, 0);
    const bool bad = __any_sync(~0u, of.y < 0);
    int2 all = of;
    if (warps > 1) {
      all = make_int2(__reduce_add_sync(~0u, of.x), __reduce_add_sync(~0u, of.y));
      upto.x += __reduce_add_sync(~0u, lane < warp ? of.x : 0);
      upto.y += __reduce_add_sync(~0u, lane < warp ? of.y : 0);
    } else {
      all = make_int2(__shfl_sync(~0u, of.x, 0), __shfl_sync(~0u, of.y, 0));
    }
    if (bad) all = upto = make_int2(0, 0);  // (then there are no passes: their rows could be anywhere)
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int g = threadIdx.x * each + i;
      if (i < each && g < p.groups) {
        if (bad) begin[i] = rows[i] = 0, own[i] = make_int2(0, 0);
        if (g == p.groups - 1) s.start[g + 1] = bad ? p.rows : begin[i] + rows[i];
        put_part(g, begin[i], rows[i], upto, all);
        upto.x += own[i].x;
        upto.y += own[i].y;
      }
    }
  }
  __syncthreads();
}
// The last group whose entry is at most `value` (a group without passes has the next one's entry).
__device__ __forceinline__ int group_of(const int* table, int groups, int value) {
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (table[mid] <= value) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ Pass pass_at(const Passes& s, int groups, int each, int index) {
  const int g = group_of(s.first, groups, index), row = s.start[g] + (index - s.first[g]) * each;
  return {g, row, min(each, s.start[g + 1] - row)};
}

// ------------------------------------------------------------------ the product
//
// The work is a list of record rows, pass after pass, of which each CTA takes a run of equal cost.  It goes through
// them in rounds of up to a record row for each warp, of one pass; where fewer are left the warps share the blocks of
// each, and their sums are added in their order.  The pass's x lies in shared memory, all of it where it fits, else
// in chunks of k, two at a time: the next one is brought before this one is read, so that warps that are done with this one
// wait for the others alone.  A warp asks for the first blocks of its next record row (or chunk) while it works on the last
// ones of this.

struct Phase {  // what a warp reads next: `count` records from this one on, and as many `apart` further on
  uint32_t record, apart;
  int count;
};
constexpr int kTiles = 2;            // record rows side by side that a warp takes: each fragment of x serves twice
constexpr int kAhead = 4 / kTiles;  // blocks in flight for each warp: 4 KB
template <int NT>
struct Sums {
  float of[kWarps][kTiles][8 * NT][kColumnPitch];
};

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 1) int4_product_kernel(const __grid_constant__ Job p) {
  extern __shared__ __align__(16) uint8_t shared[];
  using F = Form<T>;
  constexpr int kParts = Parts<T>::n, kEach = 8 * NT / kParts;
  Sums<NT>& sums = *reinterpret_cast<Sums<NT>*>(shared);
  uint4* xs = reinterpret_cast<uint4*>(shared + sizeof(Sums<NT>));
  int* tables = reinterpret_cast<int*>(xs + p.room * 128);
  const Passes passes{tables, tables + p.groups + 1};
  __shared__ Part part_of_list;
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;

  // A line: kTiles record rows.
  const int record_rows = static_cast<int>(p.w.tiles()), blocks = static_cast<int>(p.w.blocks());
  const int lines_each = (record_rows + kTiles - 1) / kTiles;  // of a pass
  find_passes<kEach, kParts>(p, passes, lines_each, part_of_list);
  // The rows behind the last group.
  if (const int end = passes.start[p.groups]; end < p.rows) {
    const size_t step = static_cast<size_t>(gridDim.x) * kThreads, last = static_cast<size_t>(p.rows - end) * p.w.n;
    for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < last; i += step)
      put(p, end + i / p.w.n, i % p.w.n, 0.0f);
  }
  int left = static_cast<int>(part_of_list.end - part_of_list.begin), index = part_of_list.index, line = part_of_list.line;
  if (left == 0) return;
  Pass pass = part_of_list.pass;

  // What is in flight, and the scales, in the lanes: lane 4 g + t holds those of rows g and g + 8 of record
  // t % kTiles of block t / kTiles.
  uint4 a[kAhead][kTiles], b[kAhead][kTiles];
  uint32_t scale_a = 0, scale_b = 0;
  const auto fetch = [&](int i, const Phase& f) {
#pragma unroll
    for (int h = 0; h < kTiles; ++h)
      fetch_record(a[i][h], b[i][h],
                   p.values + static_cast<size_t>(f.record + h * f.apart) * kInt4Record + i * kInt4Record + 16 * lane, i < f.count);
  };
  const auto fetch_scales = [&](const Phase& f) {  // (as they come: a warp would wait here for anything done with them)
    const __nv_bfloat16* s = p.scales + static_cast<size_t>(f.record + t % kTiles * f.apart + t / kTiles) * kInt4Rows + g;
    fetch_scale(scale_a, s, t / kTiles < f.count);
    fetch_scale(scale_b, s + 8, t / kTiles < f.count);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int h = 0; h < kTiles; ++h) a[i][h] = b[i][h] = make_uint4(0, 0, 0, 0);

  // How a pass's x lies in shared memory: eight columns to a tile, and as many blocks at a time as there is room for.
  const auto tiles_of = [&](const Pass& of) { return (of.rows * kParts + 7) / 8; };
  const auto chunk_of = [&](const Pass& of) {
    const int room = NT == 1 ? p.room : divide(p.room, tiles_of(of));
    return blocks <= room ? blocks : room / 2;
  };
  const auto length = [&](int chunk, int c) { return min(chunk, blocks - c * chunk); };
  const auto lines_of = [&](int at) {  // of a round: a few are left over where that keeps more warps at work
    const int most = min(kWarps, min(left, lines_each - at));
    return most > kWarps / 2 && most < kWarps * 3 / 4 ? kWarps / 2 : most;
  };
  const auto phase = [&](const Pass& of, int first, int lines, int c) {
    const int chunk = chunk_of(of), sharing = divide(kWarps, lines), part = divide(warp, lines), len = length(chunk, c);
    const int sub = divide(len + sharing - 1, sharing), at = part * sub, row = (first + warp - part * lines) * kTiles;
    // (A record row past the last one: the first of the warp again, for sums that no one reads.)
    return Phase{static_cast<uint32_t>((static_cast<size_t>(of.group) * record_rows + row) * blocks + c * chunk + at),
                 row + 1 < record_rows ? static_cast<uint32_t>(blocks) : 0u, part < sharing ? max(0, min(sub, len - at)) : 0};
  };
  int half = 0;  // of the x in shared memory, where it is read in chunks
  const auto bring = [&](const Pass& of, int c, int into) {
    const int chunk = chunk_of(of), tiles = tiles_of(of);
    stage<T>(static_cast<const T*>(p.x) + static_cast<size_t>(of.row) * p.x_pitch, p.x_pitch, of.rows, c * chunk,
             length(chunk, c), p.w.k, p.aligned, tiles, xs + into * (p.room / 2 * 128));
  };

  int lines = lines_of(line);
  bring(pass, 0, 0);  // (before the weights, behind which it would wait)
  Phase now = phase(pass, line, lines, 0);
  fetch_scales(now);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i, now);
  __syncthreads();

  for (;;) {
    // The round after this one.
    Pass next_pass = pass;
    int next_line = line + lines, next_lines = 0;
    left -= lines;
    if (next_line == lines_each) {
      next_line = 0;
      if (left > 0) next_pass = pass_at(passes, p.groups, kEach, ++index);
    }
    if (left > 0) next_lines = lines_of(next_line);
    const int sharing = divide(kWarps, lines), part = divide(warp, lines), tiles = tiles_of(pass), chunk = chunk_of(pass);
    const int chunks = blocks <= chunk ? 1 : (blocks + chunk - 1) / chunk;
    const bool resident = chunks == 1;

    float sum[kTiles][NT][4];
#pragma unroll
    for (int h = 0; h < kTiles; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[h][n][i] = 0;
    for (int c = 0; c < chunks; ++c) {
      const bool last = c + 1 == chunks;
      Phase next{0, 0, 0};
      if (!last) next = phase(pass, line, lines, c + 1);
      else if (next_lines > 0) next = phase(next_pass, next_line, next_lines, 0);
      // The chunk after this one, into the other half: of this pass, for the same lines or the next ones.
      if (!resident && (!last || (next_lines > 0 && next_line > 0))) bring(pass, last ? 0 : c + 1, half ^ 1);
      // (Columns past the pass's hold whatever was there: they only reach sums that no one reads.)
      const auto blocks_of = [&](auto column_tiles) {
        constexpr int N = decltype(column_tiles)::value;
        const int odd = (lane ^ 4) - lane;
        const uint4* x = xs + half * (p.room / 2 * 128) + part * divide(length(chunk, c) + sharing - 1, sharing) * (N * 128) + lane;
        for (bool more = true; more;) {
          more = now.count > kAhead;
          const Phase then = more ? Phase{now.record + kAhead, now.apart, now.count - kAhead} : next;
          const uint32_t scales = scale_a | scale_b << 16;
          fetch_scales(then);
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            if (i < now.count) {
              float block_sum[kTiles][N][4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint4 v[N];
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] = x[i * (N * 128) + (n * 4 + q) * 32 + (q % 2 ? odd : 0)];
#pragma unroll
                for (int h = 0; h < kTiles; ++h) {
                  const uint32_t wa = q == 0 ? a[i][h].x : q == 1 ? a[i][h].y : q == 2 ? a[i][h].z : a[i][h].w;
                  const uint32_t wb = q == 0 ? b[i][h].x : q == 1 ? b[i][h].y : q == 2 ? b[i][h].z : b[i][h].w;
                  const Four fa = four<T>(wa), fb = four<T>(wb);
#pragma unroll
                  for (int n = 0; n < N; ++n) {
                    if (q == 0) multiply<F, true>(block_sum[h][n], fa.v[0], fb.v[0], fa.v[1], fb.v[1], v[n].x, v[n].y);
                    else multiply<F, false>(block_sum[h][n], fa.v[0], fb.v[0], fa.v[1], fb.v[1], v[n].x, v[n].y);
                  }
#pragma unroll
                  for (int n = 0; n < N; ++n)
                    multiply<F, false>(block_sum[h][n], fa.v[2], fb.v[2], fa.v[3], fb.v[3], v[n].z, v[n].w);
                }
              }
#pragma unroll
              for (int h = 0; h < kTiles; ++h) {
                const uint32_t both = __shfl_sync(~0u, scales, (lane & 28) + i * kTiles + h);
                const float fa = __uint_as_float(both << 16), fb = __uint_as_float(both & 0xFFFF0000u);
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                  for (int j = 0; j < 4; ++j) sum[h][n][j] = fmaf(j < 2 ? fa : fb, block_sum[h][n][j], sum[h][n][j]);
              }
            }
            fetch(i, then);
          }
          x += kAhead * N * 128;
          now = then;
        }
      };
      if (NT == 1 || tiles == 1) blocks_of(std::integral_constant<int, 1>());
      else blocks_of(std::integral_constant<int, NT>());
      if (!last) {
        __syncthreads();
        half ^= 1;
      }
    }

#pragma unroll
    for (int h = 0; h < kTiles; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums.of[warp][h][8 * n + 2 * t + i % 2][g + i / 2 * 8] = sum[h][n][i];
    const auto result = [&](int at, int r, int c) {  // row r of the pass, weight row c of the at-th line
      float v = 0;
      const auto add = [&](auto most) {  // of up to `most` warps, all asked for together
        float part[decltype(most)::value][kParts];
#pragma unroll
        for (int h = 0; h < decltype(most)::value; ++h)
#pragma unroll
          for (int q = 0; q < kParts; ++q)
            part[h][q] = h < sharing ? sums.of[h * lines + at][c / kInt4Rows][r * kParts + q][c % kInt4Rows] : 0.0f;
#pragma unroll
        for (int h = 0; h < decltype(most)::value; ++h)
#pragma unroll
          for (int q = 0; q < kParts; ++q) v = fmaf(part[h][q], q == 0 ? 1.0f : q == 1 ? kPartUnit : kPartUnit * kPartUnit, v);
      };
      if (sharing == 1) add(std::integral_constant<int, 1>());
      else if (sharing <= 4) add(std::integral_constant<int, 4>());
      else add(std::integral_constant<int, kWarps>());
      const size_t column = static_cast<size_t>(line + at) * (kTiles * kInt4Rows) + c;
      if (column < p.w.n) put(p, pass.row + r, column, weight_unit<T>() * v);
    };
    constexpr int kWide = kTiles * kInt4Rows;
    if (sharing == 1) {  // a warp's own
      __syncwarp();
      if (warp < lines)
        for (int i = lane; i < pass.rows * kWide; i += 32) result(warp, i / kWide, i % kWide);
      __syncwarp();
    } else {
      __syncthreads();
      for (int i = threadIdx.x; i < pass.rows * lines * kWide; i += kThreads) {
        const int r = divide(i / kWide, lines);
        result(i / kWide - r * lines, r, i % kWide);
      }
    }
    if (next_lines == 0) return;
    if (next_line == 0) {  // another pass's x
      __syncthreads();
      half = 0;
      bring(next_pass, 0, 0);
      __syncthreads();
    } else if (!resident) {  // on its way
      __syncthreads();
      half ^= 1;
    } else if (sharing > 1) {
      __syncthreads();
    }
    pass = next_pass;
    line = next_line;
    lines = next_lines;
  }
}

// ------------------------------------------------------------------ the launch

template <typename T, int NT>
cudaError_t run(Job p, const DeviceInfo& dev, cudaStream_t stream) {
  const size_t tables = 2 * sizeof(int) * (p.groups + 1);
  const int most_room = static_cast<int>((kShared - sizeof(Sums<NT>) - tables) / 2048) / (2 * NT) * (2 * NT);
  const cudaError_t err = allow_shared_memory<int4_product_kernel<T, NT>>(kShared);
  if (err != cudaSuccess) return err;
  const int wanted = static_cast<int>(p.w.blocks()) * NT;
  p.room = wanted < most_room ? wanted : most_room;
  const size_t passes = (static_cast<size_t>(p.rows) * Parts<T>::n + 8 * NT - 1) / (8 * NT) + (p.groups < p.rows ? p.groups : p.rows);
  const size_t most = passes * p.w.tiles(), sms = static_cast<size_t>(dev.sm_count);
  const unsigned ctas = static_cast<unsigned>(most < sms ? most : sms);
  p.parts_inverse = ~0u / ctas;
  p.lines_inverse = ~0u / static_cast<unsigned>((p.w.tiles() + kTiles - 1) / kTiles);
  return launch(ZC_KERNEL_INT4_PRODUCT, int4_product_kernel<T, NT>, ctas, kThreads,
                sizeof(Sums<NT>) + static_cast<size_t>(p.room) * 2048 + tables, stream, p);
}

// Sixteen columns at a time, or eight where there are no more.  (Thirty-two leave the tensor cores, at 1024 products a
// cycle and SM, no room to hide in: 256 rows over 16 experts of 2048 x 7168 took 83 us with it and 70 without, while x
// came by asynchronous copies.)
template <typename T>
cudaError_t by_rows(const Job& p, const DeviceInfo& dev, cudaStream_t stream) {
  return static_cast<size_t>(p.rows) * Parts<T>::n <= 8 ? run<T, 1>(p, dev, stream) : run<T, 2>(p, dev, stream);
}

}  // namespace

cudaError_t launch_int4_matmul(const Int4Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  const Job q{p.x, p.x_pitch, p.values, p.scales, p.offsets, p.out, p.out_pitch, dev.status, p.w,
              static_cast<int>(p.rows), p.groups, p.out_type, 0, whole_vectors(type_bytes(p.type), p.w.k, {p.x}, {p.x_pitch})};
  if (p.type == ZC_TYPE_BF16) return by_rows<__nv_bfloat16>(q, dev, stream);
  if (p.type == ZC_TYPE_FP16) return by_rows<__half>(q, dev, stream);
  return by_rows<float>(q, dev, stream);
}

}  // namespace ex
}  // namespace zc
