// ex_common.cuh -- what the exchange and expert kernels share: row vectors, types, launch helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <initializer_list>

#include "zc_common.cuh"
#include "zc_moe.h"

namespace zc {
namespace ex {

// B bytes of a row moved at once.
template <int B>
struct Bytes;
template <>
struct Bytes<16> { using type = uint4; };
template <>
struct Bytes<4> { using type = uint32_t; };
template <>
struct Bytes<2> { using type = unsigned short; };

// The values of a vector as fp32, and back (rounded to nearest even).
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float(float v) { return v; }

template <typename T, int B>
union Pack {
  typename Bytes<B>::type raw;
  T v[B / sizeof(T)];
  __device__ Pack() {}
};

// A load that happens only where `on` is set, zeros elsewhere: a predicated instruction, not a
// branch, so that a thread's loads go out together.  Volatile, so that it stays behind
// wait_for_previous, and not by the read-only path, which is for memory that no one writes while the
// kernel is there: a kernel that starts early is there while the one before it writes.
__device__ __forceinline__ uint4 load_if(const void* p, bool on) {
  uint4 v = make_uint4(0, 0, 0, 0);
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
               : "l"(p), "r"(static_cast<int>(on)));
  return v;
}

// ------------------------------------------------------------------ rows as 16-byte vectors
//
// Aligned: every row starts on a 16-byte boundary.  Otherwise 16 bytes of a row are put together from
// the two aligned vectors that hold them (the second is the neighbouring lane's first one, so it
// comes from the L1): loads stay as wide as on aligned rows.  An aligned vector is only touched
// when it holds a byte of the row.

// Bytes s .. s + 15 of a and b, 0 <= s < 16, a multiple of two.  s is the same for a row's lanes, so a
// branch on the word costs less than selecting among them, except where a kernel has many of them and
// their code no longer fits the caches, or where lanes of a warp are in several rows.  (Dispatch of
// 16384 x 8 x 7167: 328 us by branches, 374 by selection, quantized rows of 16384 x 7167 72 and 76; combine's
// gradient, which shifts twice for each slot: 864 and 797, quantized columns 106 and 94.)
__device__ __forceinline__ uint4 shift_words(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t w4,
                                             unsigned s) {
  const unsigned bits = (s & 2) * 8;
  return make_uint4(__funnelshift_r(w0, w1, bits), __funnelshift_r(w1, w2, bits), __funnelshift_r(w2, w3, bits),
                    __funnelshift_r(w3, w4, bits));
}
template <bool Select = false>
__device__ __forceinline__ uint4 shift_bytes(const uint4& a, const uint4& b, unsigned s) {
  if (Select) {
    const bool h = s & 8, q = s & 4;
    const uint32_t w0 = h ? a.z : a.x, w1 = h ? a.w : a.y, w2 = h ? b.x : a.z, w3 = h ? b.y : a.w,
                   w4 = h ? b.z : b.x, w5 = h ? b.w : b.y;
    return shift_words(q ? w1 : w0, q ? w2 : w1, q ? w3 : w2, q ? w4 : w3, q ? w5 : w4, s);
  }
  if (s < 8) return s < 4 ? shift_words(a.x, a.y, a.z, a.w, b.x, s) : shift_words(a.y, a.z, a.w, b.x, b.y, s);
  return s < 12 ? shift_words(a.z, a.w, b.x, b.y, b.z, s) : shift_words(a.w, b.x, b.y, b.z, b.w, s);
}

__device__ __forceinline__ unsigned low4(const void* p) {
  return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)) & 15u;
}

// Stores bytes from .. from + 15 of a row, an aligned vector, as far as they lie in it; E: bytes of a value.
template <bool Aligned, int E>
__device__ __forceinline__ void put16(uint8_t* row, int from, int bytes, const uint4& v) {
  if (from >= 0 && from + 16 <= bytes) {
    *reinterpret_cast<uint4*>(row + from) = v;
  } else if (!Aligned) {
    using V = typename Bytes<E>::type;
    union {
      uint4 q;
      V v[16 / E];
    } u;
    u.q = v;
#pragma unroll
    for (int i = 0; i < 16 / E; ++i)
      if (from + i * E >= 0 && from + i * E < bytes) *reinterpret_cast<V*>(row + from + i * E) = u.v[i];
  }
}

// Whether all of these rows of `row_values` values are whole aligned vectors.
inline bool whole_vectors(size_t element, size_t row_values, std::initializer_list<const void*> bases,
                          std::initializer_list<size_t> pitches) {
  uintptr_t all = row_values * element;
  for (const void* b : bases) all |= reinterpret_cast<uintptr_t>(b);
  for (size_t p : pitches) all |= p * element;
  return all % 16 == 0;
}

inline size_t type_bytes(int type) { return type == ZC_TYPE_FP32 ? 4 : 2; }

// Lets a kernel's launches have up to `most` bytes of dynamic shared memory: asked once for each device
// and never lowered, since another thread may be between asking and launching.
template <auto Kernel>
cudaError_t allow_shared_memory(size_t most) {
  static std::atomic<unsigned long long> done{0};
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = 1ull << (device % 64);
  if (done.load() & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  if (err == cudaSuccess) done.fetch_or(bit);
  return err;
}

// A launch, with CUDA events around it under the kernel's id while timing is enabled (zc_timing_enable).
// It may start while the kernel before it in the stream still runs (whoever launched that one), so the
// kernel calls wait_for_previous before it touches memory.  Two kernels
// read before their wait what the kernel before them does not write: place_kernel the ids and
// dispatch_kernel x.  They are only launched behind count_kernel and place_kernel, which let the next
// kernel start after their own wait, when all that came earlier in the stream is done.
//
// Pointers to global memory are not __restrict__ in kernels that start early: the compiler may take
// it that nothing but the kernel's own accesses touches such memory, the wait included, and load
// before it.
template <typename... P, typename... A>
cudaError_t launch_clusters(int id, int cluster, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  TimingRecord t = timing_begin(id, stream);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  timing_end(t, stream);
  return err;
}
template <typename... P, typename... A>
cudaError_t launch(int id, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
  return launch_clusters(id, 1, kernel, grid, block, smem, stream, args...);
}

// (Clobbers memory: no access that the compiler knows of crosses it.)
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// ------------------------------------------------------------------ launchers

struct RowShape {
  size_t tokens, hidden;
  int k, experts, type;
};

size_t sort_workspace(size_t slots, int experts);
cudaError_t launch_sort(const void* ids, int id_bytes, size_t slots, int experts, int* position, int* offsets,
                        void* workspace, cudaStream_t stream);
cudaError_t launch_dispatch(const RowShape& s, const void* x, size_t x_pitch, void* rows, size_t rows_pitch,
                            const int* position, const int* offsets, int* status, cudaStream_t stream);
// Few slots: the sort and the dispatch in one launch, without a workspace.
bool small_dispatch(size_t slots);
cudaError_t launch_small_dispatch(const RowShape& s, const void* ids, int id_bytes, const void* x, size_t x_pitch,
                                  void* rows, size_t rows_pitch, int* position, int* offsets, cudaStream_t stream);
cudaError_t launch_combine(const RowShape& s, const void* rows, size_t rows_pitch, const float* weights,
                           const int* position, const int* offsets, void* out, size_t out_pitch, int* status,
                           cudaStream_t stream);
cudaError_t launch_combine_grad(const RowShape& s, const void* d_out, size_t d_out_pitch, const void* rows,
                                size_t rows_pitch, const float* weights, const int* position, const int* offsets,
                                void* d_rows, size_t d_rows_pitch, float* d_weights, int* status, cudaStream_t stream);

size_t column_blocks(size_t rows, int groups);
cudaError_t launch_quantize(const void* x, size_t pitch, int type, size_t rows, size_t cols, int fmt, uint8_t* values,
                            uint8_t* scales, cudaStream_t stream);
cudaError_t launch_scale_values(const void* scales, size_t words, float* out, cudaStream_t stream);
cudaError_t launch_quantize_columns(const void* x, size_t pitch, int type, size_t rows, size_t cols, int groups,
                                    const int* offsets, int fmt, uint8_t* values, uint8_t* scales, int* block_offsets,
                                    int* status, cudaStream_t stream);
cudaError_t launch_quantize_weight(const void* w, int type, int groups, size_t rows, size_t cols, int fmt,
                                   uint8_t* values, uint8_t* scales, uint8_t* values_t, uint8_t* scales_t,
                                   cudaStream_t stream);

// A product's waits: how long one may take, and (for their test) the CTA that loads nothing; -1: none.
struct Waits {
  unsigned long long limit_ns;
  int stalled;
};
constexpr Waits kWaits = {4000000000ull, -1};
struct Product {
  const uint8_t *a, *a_scales, *b, *b_scales;
  int a_fmt, b_fmt, groups, out_type;
  size_t rows, n, k, out_pitch;
  const int* offsets;
  void *out, *workspace;
  Waits waits;
};
// rows: the capacity in blocks for weight_grad.
size_t matmul_workspace(size_t rows, int groups, size_t n, size_t k);
cudaError_t launch_matmul(const Product& p, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_weight_grad(const Product& p, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace ex
}  // namespace zc
