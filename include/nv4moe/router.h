/*
 * nv4moe/router.h -- the training side of the router (included by nv4moe.h): per-expert counts,
 * a balance loss and a z loss, the gradient of the logits, and the gradients of the combine.
 *
 * Over segments of tokens (the sequences of a batch, or the whole batch as one), p = softmax of
 * a token's logits over all E experts, lse the logarithm of its sum of exponentials; a segment s
 * counts n_s tokens (those that the mask leaves), c_se assignments to expert e and
 * P_se = sum of p_e over its tokens:
 *   balance = 1/nseg * sum_s  E / (k n_s^2) * sum_e c_se P_se     (1 where routing is even)
 *   z       = 1/nseg * sum_s  1 / n_s * sum_t lse_t^2
 * A segment that counts no token adds nothing to either.  Counts are constants for the gradient.
 *
 * A logit of -infinity gives its expert the probability 0.  A token whose logits are all
 * -infinity is counted for its assignments but has no probabilities: it adds nothing to P_s or z,
 * and its gradient is 0.  A NaN or +infinity makes its token's sums NaN and raises
 * NV4_DS_NAN_LOGIT; the logits of a token that the mask leaves out are not looked at in the loss.
 * An id outside [0, E) is not counted and raises NV4_DS_BAD_EXPERT; the same id twice counts
 * twice.
 *
 * Sums over tokens are FP32 partial sums in a fixed order: every call is deterministic.
 * The conventions of nv4moe.h hold for every call here.
 */
#ifndef NV4MOE_ROUTER_H
#define NV4MOE_ROUTER_H

#include "../nv4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * moe_balance_loss -- counts, probability sums and the two losses.
 *   logits        FP32 [T][E]
 *   topk_ids      int32 [T][k], e.g. moe_permute's
 *   mask          uint8 [T] or NULL: tokens with 0 are left out of everything here
 *   nseg, seg_offsets   device int32 [nseg+1], non-decreasing, within [0, T]: segment s is tokens
 *                 [seg_offsets[s], seg_offsets[s+1]); tokens in no segment are left out.
 *                 NULL with nseg == 1: all T tokens.
 *   counts        int32 [nseg][E]
 *   prob_sums     FP32 [nseg][E]
 *   tokens        int32 [nseg]
 *   loss          FP32 [2]: balance, z
 *   ws, ws_bytes  moe_balance_workspace() bytes, 256-byte aligned; calls that share one must
 *                 not overlap
 * counts, prob_sums and tokens are plain sums over tokens: data-parallel ranks may add theirs
 * and pass the totals to moe_balance_backward.
 * T == 0: zeros.  Errors: EINVAL, EUNSUPPORTED (E > 1024, k > 32, nseg > 65536), EALIGN,
 * EWORKSPACE, EHIP.
 */
size_t moe_balance_workspace(int64_t T, int E, int nseg);
nv4_status moe_balance_loss(const float *logits, int64_t T, int E, int k, const int32_t *topk_ids,
                            const uint8_t *mask, int nseg, const int32_t *seg_offsets, int32_t *counts,
                            float *prob_sums, int32_t *tokens, float *loss, void *ws, size_t ws_bytes,
                            int32_t *dev_status, void *stream);

/*
 * moe_balance_backward -- the gradient of the logits.
 *   logits .. seg_offsets   as above
 *   counts, tokens   as moe_balance_loss left them (or their sums over ranks)
 *   dloss         FP32 [2] on the device: the gradients of balance and z (a coefficient is
 *                 multiplied in here); NULL: neither
 *   dtopk_w       FP32 [T][k] or NULL: the gradient of the routing weights, e.g.
 *                 moe_combine_backward's.  Its part of the gradient does not go by the mask or the
 *                 segments, and takes an id outside [0, E) as none.
 *   flags         NV4_RENORM as the routing had it (matters for dtopk_w alone), or 0
 *   dlogits       FP32 [T][E], all written:
 *     mask * [ dbalance * E / (nseg k n_s^2) * p_j (c_sj - sum_i c_si p_i)
 *              + dz * 2 / (nseg n_s) * lse p_j ]
 *     + p_j * (sum of dw_m over m with id_m = j  -  sum_m dw_m p_(id_m))     without NV4_RENORM
 *     + sum of w_m (dw_m - sum_i w_i dw_i) over m with id_m = j              with it
 *   A token that the mask leaves out and whose dtopk_w are zeros or NULL gets zeros, whatever its
 *   logits hold.
 * dlogits may be logits itself.  Errors: EINVAL, EUNSUPPORTED as above, EHIP.
 */
nv4_status moe_balance_backward(const float *logits, int64_t T, int E, int k, const int32_t *topk_ids,
                                const uint8_t *mask, int nseg, const int32_t *seg_offsets, const int32_t *counts,
                                const int32_t *tokens, const float *dloss, const float *dtopk_w, int flags,
                                float *dlogits, int32_t *dev_status, void *stream);

/*
 * moe_combine_backward -- the gradients of moe_combine, out[t] = sum_j w[t][j] Y[token_row[t][j]]:
 *   dY[token_row[t][j]] = w[t][j] * dout[t]      dtopk_w[t][j] = sum_h dout[t][h] * Y[token_row[t][j]][h]
 *   dout, otype   [T][H] (row stride H), BF16 or FP32
 *   Y, ytype, ldy     expert rows [rows][ldy]
 *   token_row     int32 [T][k], every row at most once (a permutation, as moe_permute's); a row outside
 *                 [0, rows) gives dtopk_w 0 and no row of dY
 *   topk_w        FP32 [T][k]
 *   dY, lddy      [rows][lddy] of ytype, or NULL; rows that no token names are not written
 *   dtopk_w       FP32 [T][k], or NULL (Y is then not read and may be NULL)
 * Sums in FP32 in a fixed order.  dY does not overlap Y or dout.
 * Errors: EINVAL, EALIGN (H % 4, ldy % 4, lddy % 4, pointers not aligned to 4 elements), EHIP.
 */
nv4_status moe_combine_backward(const void *dout, nv4_dtype otype, const void *Y, nv4_dtype ytype, int64_t ldy,
                                int64_t rows, const int32_t *token_row, const float *topk_w, int64_t T, int k,
                                int64_t H, void *dY, int64_t lddy, float *dtopk_w, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NV4MOE_ROUTER_H */
