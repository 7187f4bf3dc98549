/*
 * mxq_scored.h -- C ABI of libmxq.so, fourth part: routing by sigmoid or
 * softmax scores, with a balancing bias and groups of experts, beside mx_route
 * (mxq_routed.h), whose outputs, padded buffer and conventions it shares.
 */
#ifndef MXQ_SCORED_H
#define MXQ_SCORED_H

#include "mxq_routed.h"

#ifdef __cplusplus
extern "C" {
#endif

enum mx_score {
    MX_SCORE_SIGMOID = 0,
    MX_SCORE_SOFTMAX = 1
};

/*
 * mx_route_scored -- routing of T tokens over E experts in `groups` groups of
 * E / groups neighbours.
 *
 *   s[e]     1 / (1 + e^-z) of the token's logit z, or its softmax
 *   u[e]     s[e] + bias[e] (bias f32 [E]; NULL: the logits' own order)
 *   groups   the top_groups groups of largest worth stay, equal ones lowest
 *            first: worth is the sum of the group_best (1 or 2) largest u (s
 *            without a bias) of the group's experts that the token may use
 *   idx      the k largest u in them, descending, equal ones lowest expert
 *            first; -1 when none is left
 *   weight   scale s[idx], divided by (the sum of the picks' s) + 1e-20 when
 *            normalize != 0; 0 where idx is -1
 *   prob     the mean over the live tokens of s[e] / (sum of s + 1e-20)
 *            (sigmoid) or s[e] (softmax)
 *
 * and slot, src, counts, offs, live, loss as mx_route's, loss with that prob.
 * u and worth are compared as the binary64 values of their formulas (formed
 * within a few units of the last place), so that picks do not depend on how fp32
 * rounds scores or loses small ones; everything else is fp32: a sigmoid score
 * within 2^-20 of itself, a softmax one as mx_route's, those below 2^-126 may be 0.
 *
 * A logit of -inf bars the expert, and so does a bias that is not finite; a
 * token that is not valid, or has no logit above -inf, takes no part.  A valid
 * token with NaN or +inf among its logits is live, picks nothing, and has NaN
 * weights; prob and loss are NaN then.
 *
 * Errors as for mx_route, plus MX_E_MODE (score), MX_E_SHAPE (groups outside
 * [1, 32] or not dividing E, top_groups outside [1, groups], group_best other
 * than 1 and 2, k above top_groups E / groups).  The workspace is
 * mx_route_workspace's.
 */
int mx_route_scored(const void *logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t *valid,
                    const float *bias, int32_t score, int32_t groups, int32_t top_groups, int32_t group_best,
                    int32_t k, int32_t normalize, float scale, int32_t align, int64_t M, int32_t *idx, float *weight,
                    int32_t *slot, int32_t *src, int32_t *counts, int32_t *offs, int32_t *live, float *prob,
                    float *loss, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * mx_route_scored_grad -- gradient of weight and loss with respect to the
 * logits, as mx_route_grad: idx, counts and live are mx_route_scored's outputs
 * (the bias decides picks alone and has no gradient).  Errors as for
 * mx_route_grad, plus MX_E_MODE (score).
 */
int mx_route_scored_grad(const void *logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t *valid,
                         int32_t score, int32_t k, int32_t normalize, float scale, const int32_t *idx,
                         const float *dweight, const int32_t *counts, const int32_t *live, const float *dloss,
                         void *dlogits, int64_t ld_d, void *stream);

/*
 * mx_route_bias_step -- out[e] = bias[e] + rate sign(mean of counts -
 * counts[e]), the sign from exact integers: the bias's step towards even
 * counts.  counts int32 [E] (of mx_route_scored, or their sums over ranks), out
 * f32 [E], may be bias.  Errors: MX_E_NULL, MX_E_SHAPE (E outside [1, 1024]),
 * MX_E_ALIGN, MX_E_OVERLAP (out with counts, or with a part of bias).
 */
int mx_route_bias_step(const float *bias, const int32_t *counts, int32_t E, float rate, float *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_SCORED_H */
