/*
 * zc_int4.h -- C ABI of the experts' products on 4-bit weights, for decoding: a few rows for each expert, bound
 * by the weights' bytes.
 *
 * Exported by the same library and with the conventions of zc_moe.h: device pointers, asynchronous in the
 * order of `stream`, no allocation, no synchronization, nothing on the host that depends on device
 * values; equal inputs give equal bits.
 *
 * A matrix of n x k weights in 4 bits: each row in groups of 128 along k (the last one may be short), a group's
 * values q * s with whole numbers q of -7 .. 7 and a bfloat16 scale s.  It is kept as the products read it, in
 * records of 16 rows x 128 columns (rows past n and columns past k hold q = 0, rows past n a scale of 1):
 *   values  ceil(n / 16) x ceil(k / 128) records of 1024 bytes
 *   scales  ceil(n / 16) x ceil(k / 128) x 16 bfloat16, one for each row
 * Within a record, row r and column c are in byte word ((r / 8) * 32 + (r % 8) * 4 + c / 32) * 4 + c % 32 / 8,
 * 32 bits, little-endian, in the four bits from 4 * (c % 8 / 2 + 4 * (c % 2)) on, as q + 8.  Several matrices
 * (`groups`) lie one after the other.
 */
#ifndef ZC_INT4_H
#define ZC_INT4_H

#include "zc_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZC_INT4_GROUP 128
#define ZC_INT4_ROWS 16

/* The kernels' ids in the records of zc_timing_collect (zc.h). */
#define ZC_KERNEL_INT4_WEIGHT 28
#define ZC_KERNEL_INT4_VALUES 29
#define ZC_KERNEL_INT4_PRODUCT 30

/* Weights, `groups` matrices of n x k (contiguous, of `type`), in 4 bits.  A group's scale is the smallest
 * bfloat16 value of at least a seventh of its largest magnitude (1 for a group of zeros), and q is weight / s
 * rounded to nearest, ties to even (decided on the exact quotient).  A group that holds an infinity or a NaN gets
 * the scale NaN and q = 0, so all of its values are NaN.  (7 s may pass a group's largest magnitude by up to a 128th: next to
 * the type's largest number such a value is an infinity.)  values and scales: 16-byte aligned. */
int zc_int4_quantize(const void* w, int type, int groups, size_t n, size_t k, void* values, void* scales,
                     cudaStream_t stream);

/* The weights that they stand for: groups x n x k values q * s of `type`, contiguous, each rounded once. */
int zc_int4_values(const void* values, const void* scales, int groups, size_t n, size_t k, int type, void* out,
                   cudaStream_t stream);

/* out[r, i] = sum over blocks b of s[g, i, b] * (sum over j in b of x[r, j] q[g, i, j]), g the group of row r: rows
 * offsets[g] .. offsets[g + 1] - 1 of x belong to group g (null: one group of all the rows), rows from
 * offsets[groups] on to none, they get zeros.  x is rows x k of `type`, out rows x n of out_type, each with a pitch
 * in values.  Products are exact (with every bit of x, the smallest numbers too), sums are in fp32, a block's before
 * its scale; out is rounded once.  (Sums are held a 64th of their size, a 128th for fp32 and a 512th for fp16:
 * results below 2^-110 may lose bits.)
 * Offsets that do not start at 0, go back or pass `rows` are reported (ZC_ERR_CORRUPT), and nothing outside the
 * rows is touched; which rows are then written is not said.  values and scales: 16-byte aligned. */
int zc_int4_matmul(const void* x, size_t x_pitch, int type, size_t rows, const void* values, const void* scales,
                   int groups, size_t n, size_t k, const int* offsets, void* out, size_t out_pitch, int out_type,
                   cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZC_INT4_H */
