// ex_quantize.cu -- rows, columns of row groups, and weights rounded to 8 bits in blocks of 128.
// Bound by HBM: each input value is read once and each 8-bit value written once.
#include "ex_fp8.cuh"

namespace zc {
namespace ex {
namespace {

// One warp a block of 128 values of a row; lane l takes values l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ x, size_t pitch, size_t rows, size_t cols,
                                                       int fmt, uint8_t* __restrict__ values,
                                                       uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x % 32;
  const size_t blocks = ceil_div(cols, kBlock), words = ceil_div(blocks, 4);
  const size_t item = static_cast<size_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  if (item >= rows * words * 4) return;
  const size_t r = item / (words * 4), b = item % (words * 4);
  if (b >= blocks) {
    if (lane == 0) scales[scale_at(r, b, rows)] = 127;
    return;
  }
  float v[4];
  uint32_t m = 0;
  for (int i = 0; i < 4; ++i) {
    const size_t c = b * kBlock + i * 32 + lane;
    v[i] = c < cols ? to_float(x[r * pitch + c]) : 0.f;
    m = max(m, finite_magnitude(v[i]));
  }
  m = __reduce_max_sync(~0u, m);
  const int s = block_exponent(m, fmt);
  for (int i = 0; i < 4; ++i)
    values[(r * blocks + b) * kBlock + i * 32 + lane] = round8(v[i], inverse_scale(s), fmt);
  if (lane == 0) scales[scale_at(r, b, rows)] = s + 127;
}

// block_offsets[g] = blocks of the groups before g.
__global__ void block_offsets_kernel(const int* __restrict__ offsets, int rows, int groups, int capacity,
                                     int* __restrict__ block_offsets, int* status) {
  int at = 0;
  if (offsets && offsets[0] != 0) set_error(status, ZC_ERR_CORRUPT);
  for (int g = 0; g < groups; ++g) {
    block_offsets[g] = at;
    const int a = offsets ? offsets[g] : 0, z = offsets ? offsets[g + 1] : rows;
    if (a < 0 || z < a || z > rows) set_error(status, ZC_ERR_CORRUPT);
    else at = min(capacity, at + (z - a + kBlock - 1) / kBlock);
  }
  block_offsets[groups] = at;
}

// One CTA of 128 threads a block of 128 rows and 32 columns.
template <typename T>
__global__ void __launch_bounds__(128) quantize_columns_kernel(const T* __restrict__ x, size_t pitch, size_t rows,
                                                               size_t cols, int groups,
                                                               const int* __restrict__ offsets, int fmt,
                                                               size_t capacity, uint8_t* __restrict__ values,
                                                               uint8_t* __restrict__ scales,
                                                               const int* __restrict__ block_offsets) {
  __shared__ uint32_t amax[4][32];
  __shared__ uint8_t tile[32][kBlock + 4];
  wait_for_previous();
  const int b = blockIdx.x;
  int g = 0;
  while (g < groups && b >= block_offsets[g + 1]) ++g;
  long long begin = 0, end = 0;
  if (g < groups) {
    begin = offsets ? offsets[g] : 0;
    end = offsets ? offsets[g + 1] : rows;
    begin += static_cast<long long>(b - block_offsets[g]) * kBlock;
    end = min(end, static_cast<long long>(rows));
    if (begin < 0) end = begin;
  }
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const size_t c = static_cast<size_t>(blockIdx.y) * 32 + lane;
  float v[32];
  uint32_t m = 0;
  for (int i = 0; i < 32; ++i) {
    const long long r = begin + warp * 32 + i;
    v[i] = c < cols && r < end ? to_float(x[r * pitch + c]) : 0.f;
    m = max(m, finite_magnitude(v[i]));
  }
  amax[warp][lane] = m;
  __syncthreads();
  for (int w = 0; w < 4; ++w) m = max(m, amax[w][lane]);
  const int s = block_exponent(m, fmt);
  for (int i = 0; i < 32; ++i) tile[lane][warp * 32 + i] = round8(v[i], inverse_scale(s), fmt);
  if (warp == 0 && c < cols) scales[scale_at(c, b, cols)] = s + 127;
  if (blockIdx.x == capacity - 1 && warp == 0 && c < cols)
    for (size_t q = capacity; q % 4; ++q) scales[scale_at(c, q, cols)] = 127;
  __syncthreads();
  for (int i = warp; i < 32; i += 4) {
    const size_t row = static_cast<size_t>(blockIdx.y) * 32 + i;
    if (row < cols)
      reinterpret_cast<uint32_t*>(values + (row * capacity + b) * kBlock)[lane] =
          *reinterpret_cast<const uint32_t*>(&tile[i][lane * 4]);
  }
}

// One CTA a 128 x 128 block of a weight; the transpose goes through shared memory.
template <typename T>
__global__ void __launch_bounds__(256) quantize_weight_kernel(const T* __restrict__ w, size_t rows, size_t cols,
                                                              int fmt, uint8_t* __restrict__ values,
                                                              uint8_t* __restrict__ scales,
                                                              uint8_t* __restrict__ values_t,
                                                              uint8_t* __restrict__ scales_t) {
  __shared__ uint8_t tile[kBlock][kBlock + 4];
  __shared__ uint32_t amax[8];
  const size_t rb = ceil_div(rows, kBlock), cb = ceil_div(cols, kBlock);
  const size_t br = blockIdx.y, bc = blockIdx.x, g = blockIdx.z;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  w += g * rows * cols;
  const auto load = [&](int i, int q) {
    const size_t r = br * kBlock + i, c = bc * kBlock + q * 32 + lane;
    return r < rows && c < cols ? to_float(w[r * cols + c]) : 0.f;
  };
  uint32_t m = 0;
  for (int i = warp; i < kBlock; i += 8)
    for (int q = 0; q < 4; ++q) m = max(m, finite_magnitude(load(i, q)));
  m = __reduce_max_sync(~0u, m);
  if (lane == 0) amax[warp] = m;
  __syncthreads();
  for (int i = 0; i < 8; ++i) m = max(m, amax[i]);
  const int s = block_exponent(m, fmt);
  uint8_t* v = values + g * rows * cb * kBlock;
  for (int i = warp; i < kBlock; i += 8)
    for (int q = 0; q < 4; ++q) {
      const uint8_t byte = round8(load(i, q), inverse_scale(s), fmt);
      tile[i][q * 32 + lane] = byte;
      const size_t r = br * kBlock + i;
      if (r < rows) v[(r * cb + bc) * kBlock + q * 32 + lane] = byte;
    }
  // the block's scale for each of its rows (and, behind the last block, the word's empty bytes)
  const auto put_scales = [&](uint8_t* to, size_t n, size_t first, size_t b, size_t blocks) {
    to += g * ceil_div(blocks, 4) * 4 * n;
    for (int i = threadIdx.x; i < kBlock; i += 256)
      if (first + i < n) {
        to[scale_at(first + i, b, n)] = s + 127;
        if (b == blocks - 1)
          for (size_t q = blocks; q % 4; ++q) to[scale_at(first + i, q, n)] = 127;
      }
  };
  put_scales(scales, rows, br * kBlock, bc, cb);
  if (values_t == nullptr) return;
  put_scales(scales_t, cols, bc * kBlock, br, rb);
  __syncthreads();
  uint8_t* vt = values_t + g * cols * rb * kBlock;
  for (int i = warp; i < kBlock; i += 8)
    for (int q = 0; q < 4; ++q) {
      const size_t c = bc * kBlock + i;
      if (c < cols) vt[(c * rb + br) * kBlock + q * 32 + lane] = tile[q * 32 + lane][i];
    }
}

template <typename F>
cudaError_t by_type(int type, F&& f) {
  return type == ZC_TYPE_FP32 ? f(float{}) : type == ZC_TYPE_FP16 ? f(__half{}) : f(__nv_bfloat16{});
}

}  // namespace

size_t column_blocks(size_t rows, int groups) {
  return rows / kBlock + (rows < static_cast<size_t>(groups) ? rows : static_cast<size_t>(groups));
}

cudaError_t launch_quantize(const void* x, size_t pitch, int type, size_t rows, size_t cols, int fmt, uint8_t* values,
                            uint8_t* scales, cudaStream_t stream) {
  const size_t items = rows * ceil_div(ceil_div(cols, kBlock), 4) * 4;
  if (items == 0) return cudaSuccess;
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    return launch(quantize_kernel<T>, static_cast<unsigned>(ceil_div(items, 8)), 256, 0, stream, false,
                  static_cast<const T*>(x), pitch, rows, cols, fmt, values, scales);
  });
}

cudaError_t launch_quantize_columns(const void* x, size_t pitch, int type, size_t rows, size_t cols, int groups,
                                    const int* offsets, int fmt, uint8_t* values, uint8_t* scales, int* block_offsets,
                                    int* status, cudaStream_t stream) {
  const size_t capacity = column_blocks(rows, groups);
  cudaError_t err = launch(block_offsets_kernel, 1, 1, 0, stream, false, offsets, static_cast<int>(rows), groups,
                           static_cast<int>(capacity), block_offsets, status);
  if (err != cudaSuccess || capacity == 0) return err;
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    return launch(quantize_columns_kernel<T>,
                  dim3(static_cast<unsigned>(capacity), static_cast<unsigned>(ceil_div(cols, 32))), 128, 0, stream,
                  true, static_cast<const T*>(x), pitch, rows, cols, groups, offsets, fmt, capacity, values, scales,
                  block_offsets);
  });
}

cudaError_t launch_quantize_weight(const void* w, int type, int groups, size_t rows, size_t cols, int fmt,
                                   uint8_t* values, uint8_t* scales, uint8_t* values_t, uint8_t* scales_t,
                                   cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(ceil_div(cols, kBlock)), static_cast<unsigned>(ceil_div(rows, kBlock)),
                  static_cast<unsigned>(groups));
  return by_type(type, [&](auto t) {
    using T = decltype(t);
    return launch(quantize_weight_kernel<T>, grid, 256, 0, stream, false, static_cast<const T*>(w), rows, cols, fmt,
                  values, scales, values_t, scales_t);
  });
}

}  // namespace ex
}  // namespace zc
