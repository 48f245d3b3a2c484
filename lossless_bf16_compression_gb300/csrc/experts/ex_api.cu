// ex_api.cu -- the entry points of zc_moe.h: argument checks and launches.
#include <initializer_list>

#include "ex_common.cuh"

using namespace zc;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// Whether an output overlaps another output or an input.
bool clash(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    for (auto q = o + 1; q != outputs.end(); ++q)
      if (overlap(*o, *q)) return true;
    for (const Span& i : inputs)
      if (overlap(*o, i)) return true;
  }
  return false;
}

bool type_ok(int type) { return type == ZC_TYPE_BF16 || type == ZC_TYPE_FP16 || type == ZC_TYPE_FP32; }
bool fmt_ok(int fmt) { return fmt == ZC_FP8_E4M3 || fmt == ZC_FP8_E5M2; }
bool groups_ok(int groups) { return groups >= 1 && groups <= ZC_MOE_MAX_EXPERTS; }

constexpr size_t kMaxRows = 0x7FFFFFFF - 131072;  // rows and row tiles fit in 32 bits with room to spare
constexpr size_t kMaxBlocks = 0x7FFFFFFF / ZC_FP8_BLOCK;  // of kMaxRows rows in ZC_MOE_MAX_EXPERTS groups
constexpr size_t kMaxCols = size_t(1) << 20;
bool matrix_ok(size_t rows, size_t cols) { return rows <= kMaxRows && cols >= 1 && cols <= kMaxCols; }

size_t rows_bytes(size_t rows, size_t pitch, size_t values, int type) {
  return rows ? ((rows - 1) * pitch + values) * ex::type_bytes(type) : 0;
}
size_t blocks_of(size_t cols) { return (cols + ZC_FP8_BLOCK - 1) / ZC_FP8_BLOCK; }
size_t values_bytes(size_t rows, size_t cols) { return rows * blocks_of(cols) * ZC_FP8_BLOCK; }
size_t scales_bytes(size_t rows, size_t cols) { return rows * ((blocks_of(cols) + 3) / 4) * 4; }

bool slots_ok(size_t tokens, int k, int experts) {
  return k >= 1 && k <= ZC_MOE_MAX_K && groups_ok(experts) && tokens <= ZC_MOE_MAX_SLOTS / static_cast<size_t>(k);
}

int check_sort(const void* ids, int id_bytes, size_t tokens, int k, int experts, const int* position,
               const int* offsets, const void* workspace) {
  if (!slots_ok(tokens, k, experts) || (id_bytes != 4 && id_bytes != 8)) return ZC_ERR_INVALID_ARG;
  const size_t slots = tokens * k, scratch = ex::sort_workspace(slots, experts);
  if (!offsets || (scratch && !workspace) || (slots && (!ids || !position))) return ZC_ERR_INVALID_ARG;
  if (!aligned(ids, id_bytes) || !aligned(position, 4) || !aligned(offsets, 4) || !aligned(workspace, 16))
    return ZC_ERR_MISALIGNED;
  if (clash({{position, 4 * slots}, {offsets, 4 * size_t(experts + 1)}, {workspace, scratch}},
            {{ids, id_bytes * slots}}))
    return ZC_ERR_INVALID_ARG;
  return ZC_OK;
}

int finish(cudaError_t err) {
  if (err == cudaSuccess) return ZC_OK;
  cudaGetLastError();  // the error is the call's: it does not stay behind
  return ZC_ERR_CUDA;
}

int matmul(const void* a, const void* a_scales, int a_fmt, size_t rows, const void* b, const void* b_scales,
           int b_fmt, int groups, size_t n, size_t k, const int* offsets, void* out, size_t out_pitch,
           int out_type, void* workspace, cudaStream_t stream,
           const ex::Waits& waits) {
  if (!fmt_ok(a_fmt) || !fmt_ok(b_fmt) || !groups_ok(groups) || !matrix_ok(rows, k) || n < 1 || n > kMaxCols ||
      out_pitch < n || (out_type != ZC_TYPE_BF16 && out_type != ZC_TYPE_FP32) || (!offsets && groups != 1))
    return ZC_ERR_INVALID_ARG;
  if (rows == 0) return ZC_OK;
  const size_t scratch = ex::matmul_workspace(rows, groups, n, k);
  if (!a || !a_scales || !b || !b_scales || !out || (scratch && !workspace)) return ZC_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return ZC_ERR_MISALIGNED;
  if (!aligned(a, 128) || !aligned(b, 128) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(offsets, 4) || !aligned(out, ex::type_bytes(out_type)))
    return ZC_ERR_MISALIGNED;
  const size_t g = groups;
  if (clash({{out, rows_bytes(rows, out_pitch, n, out_type)}, {workspace, scratch}},
            {{a, values_bytes(rows, k)},
             {a_scales, scales_bytes(rows, k)},
             {b, g * values_bytes(n, k)},
             {b_scales, g * scales_bytes(n, k)},
             {offsets, offsets ? 4 * (g + 1) : 0}}))
    return ZC_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (const cudaError_t err = device_info(&dev); err != cudaSuccess) return finish(err);
  const ex::Product p{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales),
                      static_cast<const uint8_t*>(b), static_cast<const uint8_t*>(b_scales),
                      a_fmt, b_fmt, groups, out_type, rows, n, k, out_pitch, offsets, out, workspace,
                      waits};
  return finish(ex::launch_matmul(p, dev, stream));
}

int weight_grad(const void* a, const void* a_scales, int a_fmt, const void* b, const void* b_scales, int b_fmt,
                size_t capacity, int groups, size_t n, size_t k, const int* block_offsets, void* out,
                int out_type, cudaStream_t stream, const ex::Waits& waits) {
  if (!fmt_ok(a_fmt) || !fmt_ok(b_fmt) || !groups_ok(groups) || capacity > kMaxBlocks || n < 1 ||
      n > kMaxCols || k < 1 || k > kMaxCols || (out_type != ZC_TYPE_BF16 && out_type != ZC_TYPE_FP32) || !out ||
      !block_offsets || (capacity && (!a || !a_scales || !b || !b_scales)))
    return ZC_ERR_INVALID_ARG;
  if (!aligned(a, 128) || !aligned(b, 128) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(block_offsets, 4) || !aligned(out, ex::type_bytes(out_type)))
    return ZC_ERR_MISALIGNED;
  const size_t g = groups, wide = capacity * ZC_FP8_BLOCK;
  if (clash({{out, g * n * k * ex::type_bytes(out_type)}},
            {{a, values_bytes(n, wide)},
             {a_scales, scales_bytes(n, wide)},
             {b, values_bytes(k, wide)},
             {b_scales, scales_bytes(k, wide)},
             {block_offsets, 4 * (g + 1)}}))
    return ZC_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (const cudaError_t err = device_info(&dev); err != cudaSuccess) return finish(err);
  const ex::Product p{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(a_scales),
                      static_cast<const uint8_t*>(b), static_cast<const uint8_t*>(b_scales),
                      a_fmt, b_fmt, groups, out_type, capacity, n, k, k, block_offsets, out, nullptr,
                      waits};
  return finish(ex::launch_weight_grad(p, dev, stream));
}

}  // namespace

extern "C" {

size_t zc_moe_sort_workspace(size_t slots, int experts) {
  if (slots > ZC_MOE_MAX_SLOTS || !groups_ok(experts)) return 0;
  return ex::sort_workspace(slots, experts);
}

int zc_moe_sort(const void* ids, int id_bytes, size_t tokens, int k, int experts, int* position, int* offsets,
                void* workspace, cudaStream_t stream) {
  const int rc = check_sort(ids, id_bytes, tokens, k, experts, position, offsets, workspace);
  if (rc != ZC_OK) return rc;
  const size_t slots = tokens * k;
  return finish(ex::launch_sort(ids, id_bytes, slots, experts, position, offsets, workspace, stream));
}

int zc_moe_dispatch(const void* x, size_t x_pitch, int type, const void* ids, int id_bytes, size_t tokens, int k,
                    int experts, size_t hidden, void* rows, size_t rows_pitch, int* position, int* offsets,
                    void* workspace, cudaStream_t stream) {
  if (!slots_ok(tokens, k, experts) || !type_ok(type) || !matrix_ok(tokens * k, hidden) || x_pitch < hidden ||
      rows_pitch < hidden || (tokens && (!x || !rows)))
    return ZC_ERR_INVALID_ARG;
  const size_t b = ex::type_bytes(type), slots = tokens * k;
  if (!aligned(x, b) || !aligned(rows, b)) return ZC_ERR_MISALIGNED;
  if (clash({{rows, rows_bytes(slots, rows_pitch, hidden, type)}},
            {{x, rows_bytes(tokens, x_pitch, hidden, type)},
             {ids, id_bytes * slots},
             {position, 4 * slots},
             {offsets, 4 * size_t(experts + 1)},
             {workspace, ex::sort_workspace(slots, experts)}}))
    return ZC_ERR_INVALID_ARG;
  int rc = check_sort(ids, id_bytes, tokens, k, experts, position, offsets, workspace);
  if (rc != ZC_OK) return rc;
  if (ex::small_dispatch(slots))
    return finish(ex::launch_small_dispatch({tokens, hidden, k, experts, type}, ids, id_bytes, x, x_pitch, rows,
                                            rows_pitch, position, offsets, stream));
  rc = finish(ex::launch_sort(ids, id_bytes, slots, experts, position, offsets, workspace, stream));
  if (rc != ZC_OK || tokens == 0) return rc;
  DeviceInfo dev;
  if (const cudaError_t err = device_info(&dev); err != cudaSuccess) return finish(err);
  return finish(ex::launch_dispatch({tokens, hidden, k, experts, type}, x, x_pitch, rows, rows_pitch, position,
                                    offsets, dev.status, stream));
}

int zc_moe_combine(const void* rows, size_t rows_pitch, int type, const float* weights, const int* position,
                   const int* offsets, size_t tokens, int k, int experts, size_t hidden, void* out, size_t out_pitch,
                   cudaStream_t stream) {
  if (!slots_ok(tokens, k, experts) || !type_ok(type) || !matrix_ok(tokens * k, hidden) || rows_pitch < hidden ||
      out_pitch < hidden)
    return ZC_ERR_INVALID_ARG;
  if (tokens == 0) return ZC_OK;
  if (!rows || !position || !offsets || !out) return ZC_ERR_INVALID_ARG;
  const size_t b = ex::type_bytes(type), slots = tokens * k;
  if (!aligned(rows, b) || !aligned(out, b) || !aligned(weights, 4) || !aligned(position, 4) || !aligned(offsets, 4))
    return ZC_ERR_MISALIGNED;
  if (clash({{out, rows_bytes(tokens, out_pitch, hidden, type)}},
            {{rows, rows_bytes(slots, rows_pitch, hidden, type)},
             {weights, weights ? 4 * slots : 0},
             {position, 4 * slots},
             {offsets, 4 * size_t(experts + 1)}}))
    return ZC_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (const cudaError_t err = device_info(&dev); err != cudaSuccess) return finish(err);
  return finish(ex::launch_combine({tokens, hidden, k, experts, type}, rows, rows_pitch, weights, position, offsets,
                                   out, out_pitch, dev.status, stream));
}

int zc_moe_combine_grad(const void* d_out, size_t d_out_pitch, const void* rows, size_t rows_pitch, int type,
                        const float* weights, const int* position, const int* offsets, size_t tokens, int k,
                        int experts, size_t hidden, void* d_rows, size_t d_rows_pitch, float* d_weights,
                        cudaStream_t stream) {
  if (!slots_ok(tokens, k, experts) || !type_ok(type) || !matrix_ok(tokens * k, hidden) || rows_pitch < hidden ||
      d_out_pitch < hidden || d_rows_pitch < hidden)
    return ZC_ERR_INVALID_ARG;
  if (tokens == 0) return ZC_OK;
  if (!d_out || !rows || !weights || !position || !offsets || !d_rows || !d_weights) return ZC_ERR_INVALID_ARG;
  const size_t b = ex::type_bytes(type), slots = tokens * k;
  if (!aligned(rows, b) || !aligned(d_out, b) || !aligned(d_rows, b) || !aligned(weights, 4) ||
      !aligned(d_weights, 4) || !aligned(position, 4) || !aligned(offsets, 4))
    return ZC_ERR_MISALIGNED;
  if (clash({{d_rows, rows_bytes(slots, d_rows_pitch, hidden, type)}, {d_weights, 4 * slots}},
            {{rows, rows_bytes(slots, rows_pitch, hidden, type)},
             {d_out, rows_bytes(tokens, d_out_pitch, hidden, type)},
             {weights, 4 * slots},
             {position, 4 * slots},
             {offsets, 4 * size_t(experts + 1)}}))
    return ZC_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (const cudaError_t err = device_info(&dev); err != cudaSuccess) return finish(err);
  return finish(ex::launch_combine_grad({tokens, hidden, k, experts, type}, d_out, d_out_pitch, rows, rows_pitch,
                                        weights, position, offsets, d_rows, d_rows_pitch, d_weights, dev.status,
                                        stream));
}

int zc_fp8_quantize(const void* x, size_t pitch, int type, size_t rows, size_t cols, int fmt, void* values,
                    void* scales, cudaStream_t stream) {
  if (!type_ok(type) || !fmt_ok(fmt) || !matrix_ok(rows, cols) || pitch < cols) return ZC_ERR_INVALID_ARG;
  if (rows == 0) return ZC_OK;
  if (!x || !values || !scales) return ZC_ERR_INVALID_ARG;
  if (!aligned(x, ex::type_bytes(type)) || !aligned(values, 16) || !aligned(scales, 4)) return ZC_ERR_MISALIGNED;
  if (clash({{values, values_bytes(rows, cols)}, {scales, scales_bytes(rows, cols)}},
            {{x, rows_bytes(rows, pitch, cols, type)}}))
    return ZC_ERR_INVALID_ARG;
  return finish(ex::launch_quantize(x, pitch, type, rows, cols, fmt, static_cast<uint8_t*>(values),
                                    static_cast<uint8_t*>(scales), stream));
}

int zc_fp8_scale_values(const void* scales, size_t words, float* out, cudaStream_t stream) {
  if (words > kMaxRows) return ZC_ERR_INVALID_ARG;
  if (words == 0) return ZC_OK;
  if (!scales || !out) return ZC_ERR_INVALID_ARG;
  if (!aligned(scales, 4) || !aligned(out, 16)) return ZC_ERR_MISALIGNED;
  if (clash({{out, 16 * words}}, {{scales, 4 * words}})) return ZC_ERR_INVALID_ARG;
  return finish(ex::launch_scale_values(scales, words, out, stream));
}

size_t zc_fp8_column_blocks(size_t rows, int groups) {
  if (rows > kMaxRows || !groups_ok(groups)) return 0;
  return ex::column_blocks(rows, groups);
}

int zc_fp8_quantize_columns(const void* x, size_t pitch, int type, size_t rows, size_t cols, int groups,
                            const int* offsets, int fmt, void* values, void* scales, int* block_offsets,
                            cudaStream_t stream) {
  if (!type_ok(type) || !fmt_ok(fmt) || !matrix_ok(rows, cols) || pitch < cols || !groups_ok(groups) ||
      (!offsets && groups != 1) || !block_offsets)
    return ZC_ERR_INVALID_ARG;
  if (rows && (!x || !values || !scales)) return ZC_ERR_INVALID_ARG;
  if (!aligned(x, ex::type_bytes(type)) || !aligned(values, 16) || !aligned(scales, 4) || !aligned(offsets, 4) ||
      !aligned(block_offsets, 4))
    return ZC_ERR_MISALIGNED;
  const size_t wide = ex::column_blocks(rows, groups) * ZC_FP8_BLOCK;
  if (clash({{values, values_bytes(cols, wide)}, {scales, scales_bytes(cols, wide)}, {block_offsets, 4 * size_t(groups + 1)}},
            {{x, rows_bytes(rows, pitch, cols, type)}, {offsets, offsets ? 4 * size_t(groups + 1) : 0}}))
    return ZC_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (const cudaError_t err = device_info(&dev); err != cudaSuccess) return finish(err);
  return finish(ex::launch_quantize_columns(x, pitch, type, rows, cols, groups, offsets, fmt,
                                            static_cast<uint8_t*>(values), static_cast<uint8_t*>(scales),
                                            block_offsets, dev.status, stream));
}

int zc_fp8_quantize_weight(const void* w, int type, int groups, size_t rows, size_t cols, int fmt, void* values,
                           void* scales, void* values_t, void* scales_t, cudaStream_t stream) {
  if (!type_ok(type) || !fmt_ok(fmt) || rows < 1 || rows > kMaxCols || cols < 1 || cols > kMaxCols ||
      !groups_ok(groups) || !w || !values || !scales || !values_t != !scales_t)
    return ZC_ERR_INVALID_ARG;
  if (!aligned(w, ex::type_bytes(type)) || !aligned(values, 16) || !aligned(scales, 4) || !aligned(values_t, 16) ||
      !aligned(scales_t, 4))
    return ZC_ERR_MISALIGNED;
  const size_t g = groups, t = values_t ? 1 : 0;
  if (clash({{values, g * values_bytes(rows, cols)},
             {scales, g * scales_bytes(rows, cols)},
             {values_t, t * g * values_bytes(cols, rows)},
             {scales_t, t * g * scales_bytes(cols, rows)}},
            {{w, g * rows * cols * ex::type_bytes(type)}}))
    return ZC_ERR_INVALID_ARG;
  return finish(ex::launch_quantize_weight(w, type, groups, rows, cols, fmt, static_cast<uint8_t*>(values),
                                           static_cast<uint8_t*>(scales), static_cast<uint8_t*>(values_t),
                                           static_cast<uint8_t*>(scales_t), stream));
}

size_t zc_fp8_matmul_workspace(size_t rows, int groups, size_t n, size_t k) {
  if (!groups_ok(groups) || !matrix_ok(rows, k) || rows == 0 || n < 1 || n > kMaxCols) return 0;
  return ex::matmul_workspace(rows, groups, n, k);
}

int zc_fp8_matmul(const void* a, const void* a_scales, int a_fmt, size_t rows, const void* b, const void* b_scales,
                  int b_fmt, int groups, size_t n, size_t k, const int* offsets, void* out, size_t out_pitch,
                  int out_type, void* workspace, cudaStream_t stream) {
  return matmul(a, a_scales, a_fmt, rows, b, b_scales, b_fmt, groups, n, k, offsets, out, out_pitch, out_type,
                workspace, stream, ex::kWaits);
}

int zc_fp8_weight_grad(const void* a, const void* a_scales, int a_fmt, const void* b, const void* b_scales, int b_fmt,
                       size_t capacity, int groups, size_t n, size_t k, const int* block_offsets, void* out,
                       int out_type, cudaStream_t stream) {
  return weight_grad(a, a_scales, a_fmt, b, b_scales, b_fmt, capacity, groups, n, k, block_offsets, out, out_type,
                     stream, ex::kWaits);
}

int zc_fp8_matmul_stall_test(const void* a, const void* a_scales, int a_fmt, size_t rows, const void* b,
                             const void* b_scales, int b_fmt, int groups, size_t n, size_t k, const int* offsets,
                             void* out, size_t out_pitch, int out_type, void* workspace, cudaStream_t stream,
                             int stalled_cta, unsigned wait_us) {
  return matmul(a, a_scales, a_fmt, rows, b, b_scales, b_fmt, groups, n, k, offsets, out, out_pitch, out_type,
                workspace, stream, {1000ull * wait_us, stalled_cta});
}

int zc_fp8_weight_grad_stall_test(const void* a, const void* a_scales, int a_fmt, const void* b, const void* b_scales,
                                  int b_fmt, size_t capacity, int groups, size_t n, size_t k,
                                  const int* block_offsets, void* out, int out_type, cudaStream_t stream,
                                  int stalled_cta, unsigned wait_us) {
  return weight_grad(a, a_scales, a_fmt, b, b_scales, b_fmt, capacity, groups, n, k, block_offsets, out, out_type,
                     stream, {1000ull * wait_us, stalled_cta});
}

}  // extern "C"
