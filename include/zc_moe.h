/*
 * zc_moe.h -- C ABI of the operators on either side of a compressed mixture-of-experts exchange:
 * tokens sorted by expert into the send buffer and brought back with weights applied, with their
 * gradients, rows rounded to 8-bit floating point with a scale for each block of 128 values, and
 * the experts' matrix products on them.  The send buffer they fill (16-bit rows, contiguous) is
 * what zc_compress takes.
 *
 * Exported by the same library as zc.h and with its conventions: all entry points are host
 * functions, every pointer is a device address unless stated, every call is asynchronous in the
 * order of `stream`, allocates nothing and never synchronizes, host-side errors are returned
 * (ZC_ERR_INVALID_ARG, ZC_ERR_MISALIGNED, ZC_ERR_CUDA) and device-side ones are read with
 * zc_status (ZC_ERR_CORRUPT: a position or group start outside its range, the access skipped;
 * ZC_ERR_TIMEOUT: a bounded wait ran out).  The calls decide nothing on the host that depends on
 * device values, so they can be captured in a CUDA graph.
 *
 * No sum depends on the order of atomic operations: equal inputs give equal bits.
 */
#ifndef ZC_MOE_H
#define ZC_MOE_H

#include "zc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ types and limits */

#define ZC_TYPE_BF16 0
#define ZC_TYPE_FP16 1
#define ZC_TYPE_FP32 2

#define ZC_FP8_E4M3 0 /* largest value 448, no infinity */
#define ZC_FP8_E5M2 1 /* largest value 57344            */

#define ZC_MOE_MAX_EXPERTS 1024
#define ZC_MOE_MAX_K 64
#define ZC_MOE_MAX_SLOTS ((size_t)1 << 30)
#define ZC_FP8_BLOCK 128

/* ------------------------------------------------------------------ kernel timing
 *
 * The kernels' ids in the records of zc_timing_collect (zc.h). */

#define ZC_KERNEL_MOE_SORT 16         /* both kernels of a sort */
#define ZC_KERNEL_MOE_DISPATCH 17     /* with the sort, where one launch does both */
#define ZC_KERNEL_MOE_COMBINE 18      /* and the gradient of dispatch */
#define ZC_KERNEL_MOE_COMBINE_GRAD 19
#define ZC_KERNEL_FP8_ROWS 20         /* zc_fp8_quantize */
#define ZC_KERNEL_FP8_COLUMNS 21      /* and the block starts, where they take a launch of their own */
#define ZC_KERNEL_FP8_WEIGHT 22
#define ZC_KERNEL_FP8_SCALES 23       /* zc_fp8_scale_values */
#define ZC_KERNEL_FP8_PRODUCT 24      /* both products, and the clearing of a workspace */

/* ------------------------------------------------------------------ tokens sorted by expert
 *
 * T tokens with k slots each; slot s = t k + j asks for expert ids[s].  An id outside
 * [0, experts) means no expert here (a dropped token, or another rank's expert): such a slot is
 * sorted behind all experts and carries zeros.  position[s] is the place of slot s in the order
 * by expert, ties in slot order (a permutation of 0 .. T k - 1); rows offsets[e] ..
 * offsets[e + 1] - 1 belong to expert e, and rows from offsets[experts] on to no expert.
 * Rows are `hidden` values of one type; a pitch is the distance between rows in values. */

/* Bytes of workspace that zc_moe_sort and zc_moe_dispatch need: 0 for small calls (the workspace
 * may then be null) and when an argument is out of range.  Pure host function. */
size_t zc_moe_sort_workspace(size_t slots, int experts);

/* position and offsets from the ids (id_bytes 4 or 8: signed integers of that size).
 *   position  tokens x k int32;  offsets  experts + 1 int32;  workspace  16-byte aligned. */
int zc_moe_sort(const void* ids, int id_bytes, size_t tokens, int k, int experts, int* position, int* offsets,
                void* workspace, cudaStream_t stream);

/* zc_moe_sort, then rows[position[t k + j]] = x[t] for every slot (zeros for a slot without an
 * expert).  rows: tokens x k rows; must not overlap x.  One launch for small calls. */
int zc_moe_dispatch(const void* x, size_t x_pitch, int type, const void* ids, int id_bytes, size_t tokens, int k,
                    int experts, size_t hidden, void* rows, size_t rows_pitch, int* position, int* offsets,
                    void* workspace, cudaStream_t stream);

/* out[t] = sum over j of weights[t k + j] rows[position[t k + j]], over the slots that have an
 * expert, in slot order, in fp32, rounded once.  weights: tokens x k fp32, or null for ones (the
 * gradient of zc_moe_dispatch with respect to x).  A slot without an expert adds nothing,
 * whatever its weight or row holds; a token without any gets zeros. */
int zc_moe_combine(const void* rows, size_t rows_pitch, int type, const float* weights, const int* position,
                   const int* offsets, size_t tokens, int k, int experts, size_t hidden, void* out, size_t out_pitch,
                   cudaStream_t stream);

/* The gradient of zc_moe_combine: d_rows[position[s]] = weights[s] d_out[t] (zeros for a slot
 * without an expert) and d_weights[s] = <d_out[t], rows[position[s]]> in fp32 (0 for such a
 * slot).  d_rows: tokens x k rows; must not overlap rows or d_out. */
int zc_moe_combine_grad(const void* d_out, size_t d_out_pitch, const void* rows, size_t rows_pitch, int type,
                        const float* weights, const int* position, const int* offsets, size_t tokens, int k,
                        int experts, size_t hidden, void* d_rows, size_t d_rows_pitch, float* d_weights,
                        cudaStream_t stream);

/* ------------------------------------------------------------------ 8-bit blocks
 *
 * A matrix in 8-bit blocks: `rows` x `cols` values, row after row, each row padded with zeros to
 * pitch = 128 ceil(cols / 128) bytes, and a scale 2^(byte - 127) for each row and block of 128
 * columns.  The scale of row r and block b is byte [b / 4][r][b % 4] of an array
 * ceil(blocks / 4) x rows x 4 (four blocks to a word; a missing block's byte is 127).  A scale is
 * the smallest power of two that brings the block's largest finite magnitude to at most the
 * format's largest value, clamped to 2^-127 .. 2^127; 1 for a block without a finite nonzero
 * value.  Values are rounded to nearest, ties to even, after the (exact) scaling.  NaN stays NaN;
 * an infinity stays one in e5m2 and becomes NaN in e4m3, so an overflow is never hidden. */

/* Blocks along the rows of x (rows x cols of `type`, pitch in values). */
int zc_fp8_quantize(const void* x, size_t pitch, int type, size_t rows, size_t cols, int fmt, void* values,
                    void* scales, cudaStream_t stream);

/* Scale bytes as fp32: 4 `words` values 2^(byte - 127) (NaN for byte 255).  out: 16-byte aligned. */
int zc_fp8_scale_values(const void* scales, size_t words, float* out, cudaStream_t stream);

/* Blocks of 128 along the rows of each group, for products that sum over the rows: the result
 * is the transpose, `cols` rows of 128 * capacity values, capacity = zc_fp8_column_blocks(rows,
 * groups).  Group g (rows offsets[g] .. offsets[g + 1] - 1 of x) starts at block
 * block_offsets[g] and fills ceil of its rows / 128 blocks, the last one padded with zeros
 * (offsets start at 0 and do not decrease); the blocks from block_offsets[groups] on are zeros with
 * scale 1.  offsets null: one group of all the rows.  values: cols x 128 capacity bytes; scales: ceil(capacity / 4) x cols x 4;
 * block_offsets: groups + 1 int32. */
size_t zc_fp8_column_blocks(size_t rows, int groups);
int zc_fp8_quantize_columns(const void* x, size_t pitch, int type, size_t rows, size_t cols, int groups,
                            const int* offsets, int fmt, void* values, void* scales, int* block_offsets,
                            cudaStream_t stream);

/* Weights, `groups` matrices of rows x cols (contiguous), in blocks of 128 x 128 (one scale for
 * all the rows of a block): values and scales as above for each matrix, one after the other, and,
 * where values_t is not null, the transposes (cols x rows, the same 8-bit values and scales). */
int zc_fp8_quantize_weight(const void* w, int type, int groups, size_t rows, size_t cols, int fmt, void* values,
                           void* scales, void* values_t, void* scales_t, cudaStream_t stream);

/* ------------------------------------------------------------------ the experts' products */

/* out[r, i] = sum over j of a[r, j] b[g, i, j], g the group of row r: a is rows x k and b is
 * `groups` matrices of n x k, both in 8-bit blocks; offsets as above (null: one group of all the
 * rows).  Rows from offsets[groups] on get zeros.  Products of values and scales are exact; sums
 * are in fp32; out (rows x n of out_type ZC_TYPE_BF16 or ZC_TYPE_FP32) is rounded once.
 * values arrays 128-byte aligned, scales 4-byte aligned.  workspace: zc_fp8_matmul_workspace bytes,
 * 16-byte aligned, null where that is 0 (all but few rows with long sums). */
size_t zc_fp8_matmul_workspace(size_t rows, int groups, size_t n, size_t k);
int zc_fp8_matmul(const void* a, const void* a_scales, int a_fmt, size_t rows, const void* b, const void* b_scales,
                  int b_fmt, int groups, size_t n, size_t k, const int* offsets, void* out, size_t out_pitch,
                  int out_type, void* workspace, cudaStream_t stream);

/* The weights' gradient: out[g, i, j] = sum over the blocks of group g of a[i, .] b[j, .], with a
 * (n rows) and b (k rows) as zc_fp8_quantize_columns writes them, of the same `capacity` and
 * block_offsets.  out: groups x n x k; a group without rows gets zeros. */
int zc_fp8_weight_grad(const void* a, const void* a_scales, int a_fmt, const void* b, const void* b_scales, int b_fmt,
                       size_t capacity, int groups, size_t n, size_t k, const int* block_offsets, void* out,
                       int out_type, cudaStream_t stream);

/* ------------------------------------------------------------------ test hooks */

/* The products with a planted stall, for testing the bounded waits: CTA `stalled_cta` of the launch (-1: none) loads
 * nothing, so the waits for its operands run out after about wait_us microseconds (those for a whole tile after two
 * more for each of its blocks), every role gives up and zc_status reports ZC_ERR_TIMEOUT.  What the stalled CTA should
 * have computed is then missing from `out`.  The other arguments are zc_fp8_matmul's and zc_fp8_weight_grad's, whose
 * own limit is 4 s. */
int zc_fp8_matmul_stall_test(const void* a, const void* a_scales, int a_fmt, size_t rows, const void* b,
                             const void* b_scales, int b_fmt, int groups, size_t n, size_t k, const int* offsets,
                             void* out, size_t out_pitch, int out_type, void* workspace, cudaStream_t stream,
                             int stalled_cta, unsigned wait_us);
int zc_fp8_weight_grad_stall_test(const void* a, const void* a_scales, int a_fmt, const void* b, const void* b_scales,
                                  int b_fmt, size_t capacity, int groups, size_t n, size_t k,
                                  const int* block_offsets, void* out, int out_type, cudaStream_t stream,
                                  int stalled_cta, unsigned wait_us);

#ifdef __cplusplus
}
#endif

#endif /* ZC_MOE_H */
