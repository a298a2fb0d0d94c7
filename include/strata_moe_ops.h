/* strata_moe_ops.h -- operators at the edges of the routed-expert MoE block (GB300, sm_103a).
 *
 * The calls of strata_moe.h compute the one layer whose routing is a softmax top-10 over all experts and
 * whose residual is x + moe(rmsnorm(x)).  The calls below are the same steps in the forms that other
 * mixture-of-experts layers use, to be put together with strata_moe_route, strata_moe_group and
 * strata_moe_experts:
 *   strata_moe_norm          the norm before the block
 *   strata_moe_adapters      low-rank adapters of many requests beside a shared projection (the router's
 *                            logits, or the block from its input to its output)
 *   strata_moe_select        routing from logits: softmax or sigmoid scores, a bias for balance, groups of
 *                            experts, top-k, renormalised and scaled weights
 *   strata_moe_combine_norm  the weighted sum of the experts' outputs, the norm after the block, its gates,
 *                            the scaled residual and the next block's norm in one pass
 *
 * The conventions of strata_moe.h hold: device pointers owned by the caller, work only enqueued on
 * `stream` (of the current device), host-checkable errors returned before anything is enqueued, T == 0 a
 * valid empty call, T <= STRATA_MOE_T_MAX.  No call allocates device memory or synchronises, so all of them
 * can be captured into a CUDA graph.  strata_moe_select, strata_moe_norm and strata_moe_combine_norm use no
 * workspace.  All calls repeat bit for bit.  Descriptors are host structs, read during the call.  Operands overlap
 * where a row of one shares a byte with a row of the other: rows that lie between each other, as column ranges of one
 * buffer do, are fine.
 *
 * Element types (the framework's own activations are fp32): arithmetic is in 32 bits or more whatever the
 * type, and a result is rounded once, when it is stored.  One value between is held in fewer: the adapters' A_a x has 16
 * bits where y is of a 16-bit type (strata_moe_adapters says so again). */
#ifndef STRATA_MOE_OPS_H_
#define STRATA_MOE_OPS_H_

#include "strata_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define STRATA_F32 0
#define STRATA_BF16 1
#define STRATA_F16 2

/* ---- Routing ------------------------------------------------------------------------------------- */
#define STRATA_SCORE_SOFTMAX 0
#define STRATA_SCORE_SIGMOID 1
#define STRATA_SELECT_K_MAX 32
#define STRATA_SELECT_GROUP_MAX 32

typedef struct strata_select {
  int32_t n_expert;    /* E in [1, 512] (strata_moe_route's logits: a multiple of 32) */
  int32_t top_k;       /* k in [1, 32], at most top_group * (n_expert / n_group); 10 for strata_moe_group */
  int32_t score;       /* STRATA_SCORE_SOFTMAX or STRATA_SCORE_SIGMOID */
  int32_t n_group;     /* groups of n_expert / n_group consecutive experts, in [1, 32]; divides n_expert; 1: none */
  int32_t top_group;   /* groups kept, in [1, n_group] */
  int32_t group_sum;   /* 1 or 2: a group's score is the sum of its group_sum largest values */
  int32_t renorm;      /* 1: weights divided by their sum; 0: the scores themselves */
  float scale;         /* finite; multiplies the weights */
  int32_t logits_type; /* STRATA_F32, STRATA_BF16 or STRATA_F16 */
  int32_t reserved;    /* 0 */
  int64_t logits_stride; /* elements between tokens, >= n_expert */
} strata_select_t;

/* Routing of T tokens from their logits [T][E] (rows logits_stride elements apart, aligned to the element).
 * bias fp32 [E] or NULL.  Per token:
 *   - an expert is masked when its logit is NaN or not above its type's lowest finite value (so -inf, and a
 *     mask of that lowest value), or its bias is NaN or -inf; a logit of +inf counts as the largest fp32.
 *   - score p_e = exp(l_e) / sum over the unmasked of exp(l_j), or 1 / (1 + exp(-l_e)); masked: 0.
 *   - value v_e = p_e + bias_e (p_e without a bias).  The bias moves the choice, never a weight.
 *   - n_group > 1: a group's score is the sum of the group_sum largest values of its unmasked experts (of
 *     fewer if it has fewer, -inf if it has none); the top_group groups of the largest scores are kept, equal
 *     scores: lower group first.
 *   - the k experts of the kept groups with the largest values, in descending order, equal values: lower
 *     id first; without a bias the order is that of the logits (the scores' order, finer where scores
 *     round to the same number).  Masked experts come after all others, lower id first, so the k ids are always
 *     distinct and in [0, E); their weights are 0.
 *   - weight w_i = scale * p_i / max(sum of the k p, 2^-14) with renorm, else scale * p_i.  A token whose experts
 *     are all masked gets k ids with weight 0.
 * Values that decide the choice are compared as their exact values would be: two that 32-bit arithmetic cannot
 * tell apart are evaluated in 64 bits.  ids int32 [T][k], weights fp32 [T][k]. */
strata_status strata_moe_select(const strata_select_t* sel, const void* logits, int32_t T, const float* bias,
                                int32_t* ids, float* weights, void* stream);

/* ---- Norms before and after the block -------------------------------------------------------------- */
#define STRATA_NORM_N_MAX 16384
#define STRATA_NORM_PART_MAX 32

typedef struct strata_norm {
  int32_t n;         /* width in [1, 16384] */
  float eps;         /* finite, >= 0 */
  int32_t x_type;    /* element types */
  int32_t out_type;
  int64_t x_stride;  /* elements between tokens, >= n */
  int64_t out_stride;
} strata_norm_t;

/* out[t] = x[t] / sqrt(mean(x[t]^2) + eps) * gain.  gain fp32 [n] or NULL (1).  out may be x itself (same address,
 * type and stride); other overlaps are refused.  Rows need only be aligned to their elements; calls whose rows all
 * start on boundaries of four elements and are a multiple of four wide are the fastest.  The squares and their sum are
 * fp32: a row whose sum of squares is beyond its range gives zeros, and the squares of numbers under 2^-63 lose bits or
 * count as 0, which only an eps near 0 shows.  With eps 0 a row without a square above 0 is divided by 0: infinities, and NaN where an element
 * is 0 (a row of zeros; a token whose parts all have weight 0, at the norm of the block's output). */
strata_status strata_moe_norm(const strata_norm_t* nd, const void* x, int32_t T, const float* gain, void* out,
                              void* stream);

/* flags of strata_combine_norm_t */
#define STRATA_POST_NORM 1     /* norm of the block's output (post_gain, eps) */
#define STRATA_TOKEN_SIGMOID 2 /* token_gate holds logits: the gate is their sigmoid */

typedef struct strata_combine_norm {
  int32_t n;             /* width in [1, 16384] */
  int32_t n_part;        /* parts per token in [1, 32] (10 for strata_moe_experts, 1 for a layer's output) */
  int32_t flags;         /* STRATA_POST_NORM | STRATA_TOKEN_SIGMOID */
  float eps;             /* of both norms; finite, >= 0 */
  float residual_scale;  /* finite */
  float block_scale;     /* finite */
  int32_t part_type;     /* element types; x_type is out's too */
  int32_t x_type;
  int32_t next_type;
  int32_t reserved;      /* 0 */
  int64_t part_stride;   /* elements between two parts of a token, >= n */
  int64_t token_stride;  /* elements between two tokens' first parts, >= (n_part - 1) * part_stride + n */
  int64_t x_stride;      /* elements between tokens, >= n */
  int64_t out_stride;
  int64_t next_stride;
} strata_combine_norm_t;

/* After a block, for T tokens:
 *   y    = sum over k of part_weights[t][k] * parts[t][k]             (in k order; NULL weights: 1)
 *   z    = y / sqrt(mean(y^2) + eps) * post_gain with STRATA_POST_NORM, else y
 *   r    = residual_scale * x[t] + block_scale * channel_gate * token_gate[t] * z
 *   out  = r
 *   next = r / sqrt(mean(r^2) + eps) * pre_gain                       (of r before it is rounded into out)
 * A part whose weight is 0 is not read (a masked expert's part may hold anything, or nothing yet).
 * part_weights fp32 [T][n_part]; x, post_gain, channel_gate fp32 [n], token_gate fp32 [T] and pre_gain may be
 * NULL (no residual; factors of 1); out or next may be NULL, not both.  A post_gain without STRATA_POST_NORM, a
 * pre_gain without next or STRATA_TOKEN_SIGMOID without a token_gate is refused.
 * out or next may be x itself (same address, type and stride); other overlaps are refused.  Alignment and
 * the range of both norms as for strata_moe_norm. */
strata_status strata_moe_combine_norm(const strata_combine_norm_t* cn, const void* parts, const float* part_weights,
                                      const void* x, int32_t T, const float* post_gain, const float* channel_gate,
                                      const float* token_gate, const float* pre_gain, void* out, void* next,
                                      void* stream);

/* ---- Low-rank adapters ------------------------------------------------------------------------------ */
#define STRATA_ADAPTER_RANK_MAX 128
#define STRATA_ADAPTER_DIM_MAX 16384
#define STRATA_ADAPTER_COUNT_MAX 65536

typedef struct strata_adapters {
  const uint16_t* a;   /* device bf16: A_i [rank][d_in] at a + i * a_stride */
  const uint16_t* b;   /* device bf16: B_i [d_out][rank] at b + i * b_stride */
  const float* scale;  /* device fp32 [n_adapter] or NULL (1) */
  int64_t a_stride;    /* elements, a multiple of 8, >= rank * d_in */
  int64_t b_stride;    /* elements, a multiple of 8, >= d_out * rank */
  int32_t n_adapter;   /* in [1, 65536] */
  int32_t rank;        /* a multiple of 8 in [8, 128]; an adapter of a smaller rank is padded with zeros */
  int32_t d_in;        /* multiples of 8 in [8, 16384] */
  int32_t d_out;
  int32_t x_type;      /* element types; y_type is base's too */
  int32_t y_type;
  int64_t x_stride;    /* elements between tokens, multiples of 8, >= d_in and >= d_out */
  int64_t base_stride;
  int64_t y_stride;
} strata_adapters_t;

/* y[t] = base[t] + scale[a] * B_a (A_a x[t]) for the tokens of n_seg segments (requests): segment i holds tokens
 * seg_off[i] .. seg_off[i + 1] - 1 and uses adapter seg_adapter[i], or none (-1: y[t] = base[t]).  seg_off int32
 * [n_seg + 1] (device), non-decreasing, in [0, T]; empty segments are fine; rows of y outside [seg_off[0],
 * seg_off[n_seg]) keep their contents.  base NULL: 0.  y may be base itself (same address and stride: an update in
 * place, rows without an adapter untouched); other overlaps of y with base or x are refused.
 * x, base, y, a, b on 16-byte boundaries.  Products are exact and their sums in fp32: an fp32 x enters the tensor
 * cores as three bf16 terms (24 significant bits), an fp16 x as two, and A_a x[t] likewise (three terms for
 * an fp32 y, two otherwise).  A token whose x or A_a x holds a NaN, an infinity or a number that rounds to bf16's
 * infinity may give NaN in its whole row; other tokens' rows do not change.
 * n_seg in [0, STRATA_MOE_T_MAX].  A seg_off out of order or outside [0, T], or an adapter outside
 * [-1, n_adapter), sets STRATA_E_CORRUPT in the workspace's status word and the call computes nothing (y keeps
 * its contents).  ws: the workspace of any call with T tokens (strata_moe_workspace_bytes(T), initialised once);
 * calls that share one must not overlap in time. */
strata_status strata_moe_adapters(const strata_adapters_t* ad, const int32_t* seg_off, const int32_t* seg_adapter,
                                  int32_t n_seg, const void* x, int32_t T, const void* base, void* y, void* ws,
                                  size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* STRATA_MOE_OPS_H_ */
