/*
 * zc_router.h -- C ABI of an expert layer's router: from logits to the experts of each token and their
 * weights, the loss that keeps the experts evenly used, and the gradients of both.  What it chooses is
 * what zc_moe_sort and zc_moe_dispatch (zc_moe.h) take.
 *
 * Exported by the same library and with the conventions of zc_moe.h: device pointers, asynchronous in the
 * order of `stream`, no allocation, no synchronization, nothing on the host that depends on device
 * values; equal inputs give equal bits.
 *
 * Logits are `tokens` rows of `experts` values of one type, a pitch (in values) apart.  -infinity means that
 * a token may not use an expert; a row of nothing but -infinity is padding.
 */
#ifndef ZC_ROUTER_H
#define ZC_ROUTER_H

#include "zc_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZC_SCORE_SOFTMAX 0 /* of the row */
#define ZC_SCORE_SIGMOID 1 /* of each logit */

/* The kernels' ids in the records of zc_timing_collect (zc.h). */
#define ZC_KERNEL_MOE_ROUTE 25
#define ZC_KERNEL_MOE_ROUTE_GRAD 26 /* and the gradient of the balance loss */
#define ZC_KERNEL_MOE_BALANCE 27    /* both kernels of the loss */

/* The k largest logits of each token, largest first, equal ones by expert: ids[t k + j] is the expert and
 * weights[t k + j] = scale * score.  normalize != 0: the scores of a token's chosen experts are divided by
 * their sum.  1 <= k <= min(experts, ZC_MOE_MAX_K).  -infinity is never chosen: where fewer than k logits are
 * left, the other slots get the id -1 and the weight 0.  A NaN counts as larger than every number, so it is
 * chosen and shows in the weights; +infinity gives a softmax of NaN.
 *   weights  tokens x k fp32;  ids  tokens x k int32. */
int zc_moe_route(const void* logits, size_t pitch, int type, size_t tokens, int experts, int k, int score,
                 int normalize, float scale, float* weights, int* ids, cudaStream_t stream);

/* The balance loss of a routing.  With p[t, e] the softmax of row t (ZC_SCORE_SIGMOID: its sigmoids divided by
 * their sum), 0 in rows of padding, n the number of the other rows, c[e] = counts[e] the number of slots with
 * id e (ids outside [0, experts) are in none) and S[e] = sum over t of p[t, e]:
 *   loss = experts / (k n^2) * sum over e of c[e] S[e]        (1 when all are used alike; 0 for n = 0)
 *   slope[e] = experts c[e] / (k n^2), the loss's derivative in each p[t, e].
 * Sums are taken in fp32.  loss: 1 fp32; counts: experts int32; slope: experts fp32.
 * workspace: zc_moe_balance_workspace bytes (0: it may be null), 16-byte aligned. */
size_t zc_moe_balance_workspace(size_t tokens, int experts);
int zc_moe_balance(const void* logits, size_t pitch, int type, const int* ids, size_t tokens, int experts, int k,
                   int score, float* loss, int* counts, float* slope, void* workspace, cudaStream_t stream);

/* The gradient with respect to the logits: of sum over slots of d_weights * weights (zc_moe_route with the same
 * score, normalize and scale, and the ids that it chose), plus d_loss times that of the balance loss with this
 * slope.  Either part may be left out: d_weights and ids null, or d_loss and slope null (not both).  Slots with an
 * id outside [0, experts), or whose logit is -infinity, add nothing, whatever their d_weights; logits of -infinity and
 * rows of padding get 0.  Sums in fp32, rounded once.
 *   d_weights  tokens x k fp32;  d_loss  1 fp32;  d_logits  rows like logits, of the same type. */
int zc_moe_route_grad(const float* d_weights, const int* ids, const float* d_loss, const float* slope,
                      const void* logits, size_t pitch, int type, size_t tokens, int experts, int k, int score,
                      int normalize, float scale, void* d_logits, size_t d_pitch, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZC_ROUTER_H */
