// ex_int4_matmul.cu -- the experts' products on 4-bit weights, for few rows.
//
// out[r, i] = sum over b of s[i, b] * (sum over j in b of x[r, j] q[i, j]).  Bound by the weights' bytes.  A warp
// takes 16 weight rows (one record for each 128 columns, read as 2 x 512 neighbouring bytes) and multiplies them by
// up to 8 NT columns, the rows of x, on the warp-level matrix instructions: with so few rows the tensor cores are far
// from busy, and what counts is the unpacking.  A 4-bit value u = q + 8 becomes 128 + u by one logic operation (the
// low bits of a bfloat16 128) and q by a subtraction, both for two values at a time and exact.  The group's scale
// multiplies the group's sum, once for 128 products.
//
// x of 16 or 32 bits that bfloat16 does not hold is split into two or three bfloat16 values that add up to it exactly;
// they are columns of their own, added at the end.
#include "ex_int4.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTile = kWarps * kInt4Rows;  // weight rows of a CTA
constexpr int kChunk = 8;                  // blocks of x in shared memory at a time
constexpr int kAhead = 4;                  // blocks of weights in flight for each warp
constexpr int kPitch = kTile + 4;          // of a column of partial sums (in fp32), free of bank conflicts

__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A value in the same place of another CTA's shared memory.
__device__ __forceinline__ float peer_value(uint32_t address, int rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(address), "r"(rank)
               : "memory");
  return v;
}

__device__ __forceinline__ void multiply(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights 2 p and 2 p + 1 of a word as two bfloat16 values.
template <int P>
__device__ __forceinline__ uint32_t pair(uint32_t word) {
  const uint32_t v = (word >> 4 * P & 0x000F000Fu) | 0x43004300u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __float2bfloat162_rn(136.0f));
  return *reinterpret_cast<uint32_t*>(&r);
}

// ------------------------------------------------------------------ rows of x as columns of bfloat16

template <typename T>
struct Parts;
template <>
struct Parts<__nv_bfloat16> { static constexpr int n = 1; };
template <>
struct Parts<__half> { static constexpr int n = 2; };
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

// Eight neighbouring values as `Parts` vectors of eight bfloat16.
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
      }
      out[p] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Puts blocks first .. first + count - 1 of `rows` rows of x where the products read them: for each block and eight
// columns 4 x 512 bytes, in the c-th of which lane 4 g + t finds values 32 t + 8 c .. + 7 of column g.
template <typename T, int NT>
__device__ __forceinline__ void stage(const T* x, size_t pitch, int rows, size_t first, int count, size_t k, bool aligned,
                                      uint8_t* to) {
  const int vectors = count * (kInt4Group / 8);
  for (int i = threadIdx.x; i < rows * vectors; i += kThreads) {
    const int r = i / vectors, v = i % vectors;
    const size_t col = first * kInt4Group + 8 * static_cast<size_t>(v);
    const T* from = x + r * pitch + col;
    alignas(16) T in[8];
    if (aligned) {
#pragma unroll
      for (int j = 0; j < 8; j += 16 / sizeof(T))
        *reinterpret_cast<uint4*>(in + j) = load_if(from + j, col + j < k);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) in[j] = col + j < k ? from[j] : from_float<T>(0.0f);
    }
    uint4 out[Parts<T>::n];
    split<T>(in, out);
    const int block = v / 16, t = v % 16 / 4, c = v % 4;
#pragma unroll
    for (int p = 0; p < Parts<T>::n; ++p) {
      const int column = r * Parts<T>::n + p;
      reinterpret_cast<uint4*>(to)[((block * NT + column / 8) * 4 + c) * 32 + column % 8 * 4 + t] = out[p];
    }
  }
}

// ------------------------------------------------------------------ groups

struct Span {
  int group, begin, end;
};

// The index-th group that has rows (group -1: there are not so many), found by the whole CTA.
__device__ __forceinline__ Span find_group(const int* offsets, int groups, int rows, int index, int* status) {
  __shared__ Span found;
  __shared__ int counts[kWarps];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int each = (groups + kThreads - 1) / kThreads, first = threadIdx.x * each;
  int mine = 0;
  bool bad = false;
  for (int i = 0; i < each; ++i) {
    const int g = first + i;
    if (g >= groups) break;
    const int a = offsets[g], z = offsets[g + 1];
    bad |= a < 0 || z < a || z > rows || (g == 0 && a != 0);
    mine += min(max(z, 0), rows) > min(max(a, 0), rows);
  }
  if (bad) set_error(status, ZC_ERR_CORRUPT);
  int before = mine;
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(~0u, before, d);
    if (lane >= d) before += v;
  }
  if (lane == 31) counts[warp] = before;
  if (threadIdx.x == 0) found.group = -1;
  __syncthreads();
  before -= mine;
  for (int w = 0; w < warp; ++w) before += counts[w];
  if (index >= before && index < before + mine) {
    for (int i = 0; i < each; ++i) {
      const int g = first + i;
      const int a = min(max(offsets[g], 0), rows), z = min(max(offsets[g + 1], 0), rows);
      if (z > a && before++ == index) found = {g, a, z};
    }
  }
  __syncthreads();
  return found;
}

// ------------------------------------------------------------------ the product

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
  int rows, groups, out_type, slices;
  bool aligned;
};

__device__ __forceinline__ void put(const Job& p, size_t row, size_t col, float v) {
  const size_t at = row * p.out_pitch + col;
  if (p.out_type == ZC_TYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  else if (p.out_type == ZC_TYPE_FP16) static_cast<__half*>(p.out)[at] = __float2half_rn(v);
  else static_cast<float*>(p.out)[at] = v;
}

template <int NT>
constexpr size_t shared_bytes() {
  const size_t x = static_cast<size_t>(kChunk) * NT * 2048, sums = sizeof(float) * 8 * NT * kPitch;
  return x > sums ? x : sums;
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads) int4_product_kernel(const __grid_constant__ Job p) {
  extern __shared__ __align__(16) uint8_t shared[];
  constexpr int kParts = Parts<T>::n, kRowsAtOnce = 8 * NT / kParts;
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int rank = blockIdx.x % p.slices;
  const size_t column0 = static_cast<size_t>(blockIdx.x / p.slices) * kTile;
  Span span{0, 0, p.rows};
  if (p.offsets != nullptr) {
    if (blockIdx.y == gridDim.y - 1) {  // the rows behind the last group
      const int end = min(max(p.offsets[p.groups], 0), p.rows);
      if (rank == 0)
        for (size_t i = threadIdx.x; i < static_cast<size_t>(p.rows - end) * kTile; i += kThreads)
          if (column0 + i % kTile < p.w.n) put(p, end + i / kTile, column0 + i % kTile, 0.0f);
      return;
    }
    span = find_group(p.offsets, p.groups, p.rows, blockIdx.y, p.status);
    if (span.group < 0) return;
  }
  const size_t tiles = p.w.tiles(), blocks = p.w.blocks(), tile = column0 / kInt4Rows + warp;
  const int per = static_cast<int>((blocks + p.slices - 1) / p.slices);
  const size_t begin = min(blocks, static_cast<size_t>(rank) * per);
  const int count = tile < tiles ? static_cast<int>(min(blocks, begin + per) - begin) : 0;  // of this warp
  const int staged = static_cast<int>(min(blocks, begin + per) - begin);
  const size_t record0 = (span.group * tiles + tile) * blocks + begin;
  const uint8_t* values = p.values + record0 * kInt4Record + 16 * lane;
  const __nv_bfloat16* scales = p.scales + record0 * kInt4Rows + g;

  for (int row = span.begin; row < span.end; row += kRowsAtOnce) {
    const int rows = min(kRowsAtOnce, span.end - row), columns = rows * kParts;
    uint4 a[kAhead], b[kAhead];
    float sa[kAhead], sb[kAhead];
    const auto fetch = [&](int i, int block) {
      const bool on = block < count;
      a[i] = load_if(values + static_cast<size_t>(block) * kInt4Record, on);
      b[i] = load_if(values + static_cast<size_t>(block) * kInt4Record + 512, on);
      sa[i] = on ? __bfloat162float(scales[static_cast<size_t>(block) * kInt4Rows]) : 0.0f;
      sb[i] = on ? __bfloat162float(scales[static_cast<size_t>(block) * kInt4Rows + 8]) : 0.0f;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(i, i);
    float sum[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] = 0;
    const T* x = static_cast<const T*>(p.x) + static_cast<size_t>(row) * p.x_pitch;
    for (int base = 0; base < staged; base += kAhead) {
      if (base % kChunk == 0) {
        __syncthreads();
        stage<T, NT>(x, p.x_pitch, rows, begin + base, min(kChunk, staged - base), p.w.k, p.aligned, shared);
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (base + i < count) {
          const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
          const uint4* at = reinterpret_cast<const uint4*>(shared) + (base + i) % kChunk * (NT * 128) + lane;
          float part[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[n][j] = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t a0 = pair<0>(wa[c]), a1 = pair<1>(wa[c]), a2 = pair<2>(wa[c]), a3 = pair<3>(wa[c]);
            const uint32_t b0 = pair<0>(wb[c]), b1 = pair<1>(wb[c]), b2 = pair<2>(wb[c]), b3 = pair<3>(wb[c]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (8 * n + g < columns) v = at[(n * 4 + c) * 32];
              multiply(part[n], a0, b0, a1, b1, v.x, v.y);
              multiply(part[n], a2, b2, a3, b3, v.z, v.w);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            sum[n][0] = fmaf(sa[i], part[n][0], sum[n][0]);
            sum[n][1] = fmaf(sa[i], part[n][1], sum[n][1]);
            sum[n][2] = fmaf(sb[i], part[n][2], sum[n][2]);
            sum[n][3] = fmaf(sb[i], part[n][3], sum[n][3]);
          }
        }
        fetch(i, base + i + kAhead);
      }
    }
    // The CTA's sums, column after column, then those of the slices of k added in their order.
    __syncthreads();
    float* sums = reinterpret_cast<float*>(shared);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sums[(8 * n + 2 * t + i % 2) * kPitch + warp * kInt4Rows + g + i / 2 * 8] = sum[n][i];
    cluster_sync();
    const uint32_t at = shared_address(sums);
    for (int i = rank * kThreads + threadIdx.x; i < rows * kTile; i += p.slices * kThreads) {
      const int r = i / kTile, c = i % kTile;
      if (column0 + c >= p.w.n) continue;
      float v = 0;
      for (int s = 0; s < p.slices; ++s)
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          v += peer_value(at + sizeof(float) * ((r * kParts + q) * kPitch + c), s);
      put(p, row + r, column0 + c, v);
    }
    cluster_sync();
  }
}

template <typename T, int NT>
cudaError_t run(const Job& p, int jobs, cudaStream_t stream) {
  cudaError_t err = cudaSuccess;
  if (shared_bytes<NT>() > 48 * 1024) err = allow_shared_memory<int4_product_kernel<T, NT>>(shared_bytes<NT>());
  if (err != cudaSuccess) return err;
  const auto tiles = static_cast<unsigned>((p.w.n + kTile - 1) / kTile);
  return launch_clusters(ZC_KERNEL_INT4_PRODUCT, p.slices, int4_product_kernel<T, NT>,
                         dim3(tiles * p.slices, static_cast<unsigned>(jobs)), kThreads, shared_bytes<NT>(), stream, p);
}

template <typename T>
cudaError_t by_rows(const Job& p, int jobs, cudaStream_t stream) {
  // Columns at a time: what an average group has, and some more.
  const int groups = p.groups < p.rows ? p.groups : p.rows;
  const int columns = (p.rows + groups - 1) / groups * Parts<T>::n;
  if (columns <= 8) return run<T, 1>(p, jobs, stream);
  if (columns <= 16) return run<T, 2>(p, jobs, stream);
  return run<T, 4>(p, jobs, stream);
}

}  // namespace

cudaError_t launch_int4_matmul(const Int4Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  Job q{p.x, p.x_pitch, p.values, p.scales, p.offsets, p.out, p.out_pitch, dev.status, p.w,
            static_cast<int>(p.rows), p.groups, p.out_type, 1, whole_vectors(type_bytes(p.type), p.w.k, {p.x}, {p.x_pitch})};
  while (q.slices < 8 && q.slices * kChunk < static_cast<int>(p.w.blocks())) q.slices *= 2;
  const int jobs = p.offsets == nullptr ? 1 : (q.groups < q.rows ? q.groups : q.rows) + 1;
  if (p.type == ZC_TYPE_BF16) return by_rows<__nv_bfloat16>(q, jobs, stream);
  if (p.type == ZC_TYPE_FP16) return by_rows<__half>(q, jobs, stream);
  return by_rows<float>(q, jobs, stream);
}

}  // namespace ex
}  // namespace zc
