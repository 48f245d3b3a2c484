// ex_matmul.cu -- the experts' products on 8-bit blocks, the weights' gradient among them.
#include "ex_fp8.cuh"

namespace zc {
namespace ex {
namespace {

constexpr int kTile = 64;  // rows and columns of a CTA's tile; 256 threads, 4 x 4 outputs each

struct SimpleParams {
  const uint8_t *a, *a_scales, *b, *b_scales;
  int a_fmt, b_fmt, groups, out_type;
  size_t rows, n, pitch, a_scale_rows, out_pitch;
  const int* offsets;  // row groups, or block groups when by_blocks
  void* out;
  bool by_blocks;
  int* status;
};

// Tile q of the rows (each group's tiles, then the tiles of the rows behind the last group):
// its group and rows.  False when there are fewer.
__device__ bool row_tile(const SimpleParams& p, int q, int* group, long long* r0, long long* r1) {
  long long a = 0;
  if (p.offsets && p.offsets[0] != 0) set_error(p.status, ZC_ERR_CORRUPT);
  for (int g = 0; g <= p.groups; ++g) {
    long long z = g == p.groups ? static_cast<long long>(p.rows) : p.offsets ? p.offsets[g + 1] : static_cast<long long>(p.rows);
    if (z > static_cast<long long>(p.rows) || z < a) {
      set_error(p.status, ZC_ERR_CORRUPT);
      z = z < a ? a : static_cast<long long>(p.rows);
    }
    const int tiles = static_cast<int>((z - a + kTile - 1) / kTile);
    if (q < tiles) {
      *group = g;
      *r0 = a + static_cast<long long>(q) * kTile;
      *r1 = z;
      return true;
    }
    q -= tiles;
    a = z;
  }
  return false;
}

__global__ void __launch_bounds__(256) simple_matmul_kernel(SimpleParams p) {
  __shared__ float sa[32][kTile + 1], sb[32][kTile + 1];
  const size_t i0 = static_cast<size_t>(blockIdx.y) * kTile;
  int g = blockIdx.z;
  long long r0 = static_cast<long long>(blockIdx.x) * kTile, r1 = p.rows;
  size_t k0 = 0, k1 = p.pitch;
  const uint8_t *b = p.b, *b_scales = p.b_scales;
  if (p.by_blocks) {
    k0 = static_cast<size_t>(max(0, p.offsets[g])) * kBlock;
    k1 = min(p.pitch, static_cast<size_t>(max(0, p.offsets[g + 1])) * kBlock);
  } else {
    if (!row_tile(p, blockIdx.x, &g, &r0, &r1)) return;
    if (g == p.groups) {
      k1 = 0;  // rows without a group: zeros
    } else {
      b += g * p.n * p.pitch;
      b_scales += g * ceil_div(p.pitch / kBlock, 4) * 4 * p.n;
    }
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (size_t k = k0; k < k1; k += 32) {
    for (int i = threadIdx.x; i < kTile * 32; i += 256) {
      const int row = i / 32, c = i % 32;
      const size_t blk = (k + c) / kBlock;
      const size_t r = r0 + row, n = i0 + row;
      sa[c][row] = static_cast<long long>(r) < r1 ? value8(p.a[r * p.pitch + k + c], p.a_fmt) *
                                                        scale_value(p.a_scales[scale_at(r, blk, p.a_scale_rows)])
                                                  : 0.f;
      sb[c][row] = n < p.n ? value8(b[n * p.pitch + k + c], p.b_fmt) * scale_value(b_scales[scale_at(n, blk, p.n)]) : 0.f;
    }
    __syncthreads();
    for (int c = 0; c < 32; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[c][ty * 4 + i], sb[c][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const size_t r = r0 + ty * 4 + i, n = i0 + tx * 4 + j;
      if (static_cast<long long>(r) >= r1 || n >= p.n) continue;
      const size_t at = (p.by_blocks ? g * p.rows * p.out_pitch : 0) + r * p.out_pitch + n;
      if (p.out_type == ZC_TYPE_FP32) static_cast<float*>(p.out)[at] = acc[i][j];
      else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[i][j]);
    }
}

}  // namespace

cudaError_t launch_matmul(const Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  SimpleParams s{p.a, p.a_scales, p.b, p.b_scales, p.a_fmt, p.b_fmt, p.groups, p.out_type, p.rows, p.n,
                 ceil_div(p.k, kBlock) * kBlock, p.rows, p.out_pitch, p.offsets, p.out, false, dev.status};
  const dim3 grid(static_cast<unsigned>(ceil_div(p.rows, kTile)) + p.groups + 1, static_cast<unsigned>(ceil_div(p.n, kTile)));
  return launch(simple_matmul_kernel, grid, 256, 0, stream, false, s);
}

cudaError_t launch_weight_grad(const Product& p, const DeviceInfo& dev, cudaStream_t stream) {
  SimpleParams s{p.a, p.a_scales, p.b, p.b_scales, p.a_fmt, p.b_fmt, p.groups, p.out_type, p.n, p.k,
                 p.rows * kBlock, p.n, p.k, p.offsets, p.out, true, dev.status};
  const dim3 grid(static_cast<unsigned>(ceil_div(p.n, kTile)), static_cast<unsigned>(ceil_div(p.k, kTile)), p.groups);
  return launch(simple_matmul_kernel, grid, 256, 0, stream, false, s);
}

}  // namespace ex
}  // namespace zc
