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
 *   strata_moe_linear        a projection of a few tokens by 4-bit weights with group scales, or by bf16 weights
 *                            (the router's logits, of any width)
 *   strata_moe_q4_experts    the routed experts of a few tokens, of any shape, with 4-bit weights: gate, up, SwiGLU,
 *                            down and the weighted sum
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
 * type, and a result is rounded once, when it is stored.  Some values between are held in fewer: the adapters' A_a x has 16
 * bits where y is of a 16-bit type, an fp32 x beside 4-bit weights and the experts' hidden values 22 (the calls say so again). */
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

/* ---- 4-bit weights with group scales ---------------------------------------------------------------- */
#define STRATA_Q4_ROWS_MAX 1048576
#define STRATA_Q4_COLUMNS_MAX 32768

/* The format of a 4-bit matrix w [n_out][d_in]: w[n][k] = scale[n][k / group] * (code[n][k] - zero[n][k / group]), codes and zero
 * points in 0 .. 15, zero points of 8 where the matrix has none.  As it comes (dense, row-major):
 *   codes  uint8 [n_out][d_in / 2], column 2i in bits 0-3 and column 2i + 1 in bits 4-7 of byte i
 *   scales bf16 or fp16 [n_out][d_in / group]
 *   zeros  uint8 [n_out][d_in / group], one to a byte (its low four bits count), or none
 * Packed, as the kernels read it: slabs of 16 rows one after the other (a last slab of fewer rows is filled up with zeros), a slab
 * in chunks of 128 columns (the last may hold 32, 64 or 96), a chunk of nb blocks of 32 columns as
 *   codes   [2 halves][32 lanes][nb blocks] 32-bit words: lane 4g + c holds row g (half 0) or g + 8 (half 1), columns 8c .. 8c + 7
 *           of the block, column 2j of them in bits 4j .. 4j + 3 and column 2j + 1 in bits 16 + 4j .. 19 + 4j
 *   scales  [8 g][128 / group]{row g, row g + 8}
 *   zeros   [8 g][128 / group]{row g, row g + 8}, bytes, each g padded to 4 of them; only with zeros
 * A paired matrix is gate and up of an expert at once: its rows are d_ff rows of gate, then d_ff of up, and a slab holds rows
 * 8s .. 8s + 7 of gate and the same rows of up. */
typedef struct strata_q4 {
  int32_t n_out;      /* rows, in [1, 1048576]; paired: 2 * d_ff, a multiple of 16 */
  int32_t d_in;       /* columns, a multiple of group in [group, 32768] */
  int32_t group;      /* 32, 64 or 128 */
  int32_t scale_type; /* STRATA_BF16 or STRATA_F16 */
  int32_t zeros;      /* 1: with zero points; 0: all are 8 */
  int32_t paired;     /* 1: gate and up of an expert */
} strata_q4_t;

/* Bytes of one packed matrix (a multiple of 32); 0 if the format is none of the above. */
size_t strata_q4_bytes(const strata_q4_t* q);

/* Packs n_matrix matrices of one format that follow one another in codes, scales and zeros (NULL without zero points, and
 * only then) into packed (strata_q4_bytes each).  strata_pack_q4: host arrays.  strata_pack_q4_device: device arrays, packed on a 16-byte
 * boundary, n_matrix in [0, 65536]; it only enqueues. */
strata_status strata_pack_q4(const strata_q4_t* q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, void* packed,
                             int64_t n_matrix);
strata_status strata_pack_q4_device(const strata_q4_t* q, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                                    void* packed, int64_t n_matrix, void* stream);

/* ---- Projections of a few tokens --------------------------------------------------------------------- */
#define STRATA_W_Q4 0
#define STRATA_W_BF16 1

typedef struct strata_linear {
  const void* w;     /* device: a packed matrix (STRATA_W_Q4), or bf16 rows of d_in elements (STRATA_W_BF16); 16-byte boundary */
  int64_t w_stride;  /* STRATA_W_BF16: elements between rows, a multiple of 8, >= d_in; STRATA_W_Q4: 0 */
  strata_q4_t q4;    /* the matrix's format, not paired; STRATA_W_BF16: n_out and d_in alone (d_in a multiple of 8 in [8, 32768]), the rest 0 */
  int32_t weight;    /* STRATA_W_Q4 or STRATA_W_BF16 */
  int32_t x_type;    /* element types */
  int32_t y_type;
  int32_t reserved;  /* 0 */
  int64_t x_stride;  /* elements between tokens, a multiple of 8, >= d_in */
  int64_t y_stride;  /* elements between tokens, >= n_out */
} strata_linear_t;

/* y[t][n] = sum over k of w[n][k] * x[t][k] + bias[n].  bias fp32 [n_out] or NULL.  x on a 16-byte boundary, y aligned to its elements;
 * y must not overlap x or bias.  No workspace.  Products are exact and their sums fp32; an fp32 x enters them with 22 bits beside 4-bit weights (24
 * beside bf16 ones), a bf16 or fp16 x with all its bits, each down to 2^-40 of the
 * largest of the 128 columns around it.  Scales are below 2^100 in magnitude: with larger ones sums may pass fp32's range where the results do not.
 * A token whose x holds a NaN or an infinity (beside bf16 weights: or a number that rounds to bf16's infinity)
 * may give NaN in its whole row; other tokens' rows do not change.
 * Built for few tokens: 4-bit weights are read once for up to 24 (16-bit x) or 12 (fp32) of them, bf16 weights for 24 (bf16), 12 (fp16) or 8 (fp32),
 * and the time of more grows in proportion. */
strata_status strata_moe_linear(const strata_linear_t* li, const void* x, int32_t T, const float* bias, void* y, void* stream);

/* ---- Routed experts of a few tokens -------------------------------------------------------------------- */
#define STRATA_Q4_EXPERTS_T_MAX 64
#define STRATA_Q4_EXPERTS_DIM_MAX 8192
#define STRATA_Q4_EXPERTS_E_MAX 1024
#define STRATA_Q4_EXPERTS_K_MAX 32

typedef struct strata_q4_experts {
  const void* gate_up;     /* device: expert e's packed gate and up (paired) at gate_up + e * gate_up_stride; 16-byte boundary */
  const void* down;        /* device: expert e's packed down at down + e * down_stride; 16-byte boundary */
  int64_t gate_up_stride;  /* bytes, multiples of 16, at least the packed matrix */
  int64_t down_stride;
  strata_q4_t gate_up_q4;  /* n_out = 2 * d_ff, d_in = d_model, paired */
  strata_q4_t down_q4;     /* n_out = d_model, d_in = d_ff, at most 8192 each; group, scale_type and zeros as gate_up_q4's */
  int32_t n_expert;        /* in [1, 1024] */
  int32_t top_k;           /* experts of a token, in [1, 32] */
  int32_t x_type;          /* element types */
  int32_t out_type;
  int64_t x_stride;        /* elements between tokens, multiples of 8, >= d_model */
  int64_t out_stride;
} strata_q4_experts_t;

/* Bytes of a workspace for T tokens; 0 if the descriptor or T is refused.  It holds strata_moe_workspace_init's words at its start and
 * may be any call's workspace that is large enough for each. */
size_t strata_moe_q4_experts_workspace_bytes(const strata_q4_experts_t* ex, int32_t T);

/* out[t] = sum over i of weights[t][i] * D_e (silu(G_e x[t]) * (U_e x[t])), e = ids[t][i], in the order of i, silu(z) = z / (1 + exp(-z)).
 * ids int32 [T][top_k], weights fp32 [T][top_k] (strata_moe_select's).  A slot with an id of -1 or a weight of 0 has no expert:
 * nothing of it is read; a token without any gets zeros.  An expert may stand twice in a token's list.  A shared expert is one more expert that every
 * token lists.  T in [0, 64].  Made for lists that spread over the experts: one that more tokens list than a block holds (8 of them with a 16-bit x, 4
 * with fp32, up to three times as many where lists are crowded) is passed over again for each further block, by the same few CTAs.  64 tokens of 512
 * experts take four times as long with a shared expert as without.  x and out on 16-byte boundaries; out must not overlap x, ids or weights.
 * Products are exact and summed in fp32 as in strata_moe_linear; the hidden values of an expert are held in fp32 and enter the
 * second product with 22 bits.  NaN and infinities as there.
 * An id outside [-1, n_expert) sets STRATA_E_CORRUPT in the workspace's status word and the call computes nothing (out keeps its contents).
 * Calls that share a workspace must not overlap in time.  One cooperative launch, whose CTAs wait for one another; a wait of more than 2 s sets
 * STRATA_E_TIMEOUT, and the workspace must then be initialised again. */
strata_status strata_moe_q4_experts(const strata_q4_experts_t* ex, const int32_t* ids, const float* weights, const void* x, int32_t T,
                                    void* out, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* STRATA_MOE_OPS_H_ */
