// ex_int4.cuh -- the layout of 4-bit weights, and the launchers of ex_int4.cu and ex_int4_matmul.cu.
#pragma once

#include "ex_common.cuh"
#include "zc_int4.h"

namespace zc {
namespace ex {

constexpr int kInt4Group = ZC_INT4_GROUP, kInt4Rows = ZC_INT4_ROWS;
constexpr int kInt4Record = kInt4Group * kInt4Rows / 2;  // bytes

struct Int4Shape {
  size_t n, k;
  __host__ __device__ size_t tiles() const { return (n + kInt4Rows - 1) / kInt4Rows; }
  __host__ __device__ size_t blocks() const { return (k + kInt4Group - 1) / kInt4Group; }
  __host__ __device__ size_t records() const { return tiles() * blocks(); }
};

cudaError_t launch_int4_quantize(const void* w, int type, size_t groups, const Int4Shape& s, uint8_t* values,
                                 __nv_bfloat16* scales, cudaStream_t stream);
cudaError_t launch_int4_values(const uint8_t* values, const __nv_bfloat16* scales, size_t groups, const Int4Shape& s,
                               int type, void* out, cudaStream_t stream);

struct Int4Product {
  const void* x;
  size_t x_pitch;
  int type;
  size_t rows;
  const uint8_t* values;
  const __nv_bfloat16* scales;
  int groups;
  Int4Shape w;
  const int* offsets;
  void* out;
  size_t out_pitch;
  int out_type;
};
cudaError_t launch_int4_matmul(const Int4Product& p, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace ex
}  // namespace zc
