/*
 * libmoe, routing with scores: moe_gate's sibling for routers that score the
 * experts with a sigmoid or a softmax, add a balance bias for the selection,
 * choose among groups of experts first and scale the weights.
 *
 * The conventions, status codes and types are libmoe.h's.
 */
#ifndef LIBMOE_ROUTE_H
#define LIBMOE_ROUTE_H

#include "libmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/* How a group of experts is valued: by its best choice value, or by the sum of
 * its two best ones (of the only one where a group has one expert). */
typedef enum { MOE_RANK_MAX = 0, MOE_RANK_TOP2 = 1 } moe_group_rank;

/* Largest number of expert groups. */
#define MOE_MAX_EXPERT_GROUPS 64

/*
 * moe_route - k experts and their weights for every token.
 *
 *   logits   [T][E] fp32 or bf16 (`dtype`), read only.  NaN counts as -inf.
 *   bias     [E] fp32 or NULL: added to the scores for the selection only.
 *
 *   score of expert e   s_e = softmax over the E logits, or sigmoid(logit_e).
 *       (softmax: +inf logits share the mass equally; a row whose logits are
 *       all -inf has scores 0).  Scores are doubles: what rounds to 0 there (below
 *       2^-1075, a sigmoid of less than about -745.1) is 0.
 *   choice value        c_e = s_e + bias_e in double, NaN as -inf; without a
 *       bias the experts are ordered by their logits, whose order is the scores'.
 *   groups              the E experts form n_groups groups of E / n_groups
 *       consecutive ones; the top_groups groups of the largest value
 *       (`group_rank` over the c_e of the group; over the s_e for MOE_RANK_TOP2
 *       without a bias) stay, equal ones by the lower group.  n_groups = 1:
 *       every expert stays.
 *   topk_ids [T][k] int32, written: the k experts of the largest choice values
 *       among the groups that stay, in descending order, equal ones by the lower
 *       expert id.  An expert of -inf choice value comes after all others.
 *   topk_w   [T][k] fp32, written: scale * s_id (renormalize = 0), or
 *       scale * s_id / (sum of the k chosen scores) (renormalize = 1; all 0
 *       where that sum is 0).  Within 1e-6 relative of the exact value, or 2^-149
 *       where that is more (results next to fp32's subnormals).
 *
 *   Requires T >= 0, 1 <= n_groups <= 64, E a multiple of n_groups,
 *   1 <= top_groups <= n_groups, 1 <= k <= top_groups * (E / n_groups),
 *   E <= 512, a finite scale.  Nothing depends on another row, so the results do
 *   not change with the batch.
 *   Errors: MOE_ERR_INVALID_ARG for the sizes above, an unknown score or rank,
 *   renormalize not 0 or 1, a scale that is not finite, NULL or misaligned
 *   pointers (4 bytes; bf16 logits 2); MOE_ERR_UNSUPPORTED for E > 512,
 *   n_groups > 64, an unknown dtype or T * E past int32.
 */
moe_status moe_route(const void* logits, moe_dtype dtype, const float* bias, int32_t T, int32_t E, int32_t k,
                     moe_score score, int32_t n_groups, int32_t top_groups, moe_group_rank group_rank,
                     int32_t renormalize, float scale, int32_t* topk_ids, float* topk_w, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMOE_ROUTE_H */
