/*
 * eagle3_moe.h - the feed-forward part of a mixture-of-experts target (building blocks).
 *
 * The target layers that verify a tree need, in place of the dense SwiGLU feed-forward of "EAGLE-3:
 * Engineering Implementation of LLM Inference Acceleration", appendix C, the following when the
 * target is a mixture of experts:
 *   logits = x Wr^T                            eagle3_linear (EAGLE3_EPI_F32)
 *   experts of every row, rows by expert       eagle3_moe_route
 *   silu(x Wg_e^T) * (x Wu_e^T), by expert     eagle3_grouped_linear (EAGLE3_EPI_SWIGLU, rows gathered)
 *   h Wd_e^T, by expert                        eagle3_grouped_linear (EAGLE3_EPI_BF16)
 *   residual + weighted sum over the experts   eagle3_moe_combine
 *
 * Conventions as in eagle3.h: asynchronous on the stream, host-detected errors returned before any
 * launch, caller-owned device memory, scratch in a caller workspace (its contents need no
 * preparation and mean nothing between calls).  Row counts by expert are known on the device only;
 * no call reads them back, so the whole sequence can be captured into a CUDA graph.
 */
#ifndef EAGLE3_MOE_H
#define EAGLE3_MOE_H

#include "eagle3.h"
#include "eagle3_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EAGLE3_MOE_MAX_EXPERTS 512
#define EAGLE3_MOE_MAX_TOP_K 16

typedef enum {
    EAGLE3_MOE_SOFTMAX = 0, /* score = exp(z_e - max z) / sum over the row's finite logits          */
    EAGLE3_MOE_SIGMOID = 1  /* score = 1 / (1 + exp(-z_e))                                          */
} eagle3_moe_scoring_t;

/* ------------------------------------------------------------------------------------------------
 * eagle3_moe_route - the top-k experts of every row, and the rows in expert order.
 *
 * A row takes the top_k largest of its finite logits, in decreasing order, equal logits by
 * increasing expert (both scores grow with the logit, so this is the order of the scores too).  A
 * logit that is not finite (-inf, +inf, NaN) marks an expert that the row does not take; a row with
 * fewer than top_k finite logits, and a row at or past *num_rows, leaves the remaining places empty
 * (id -1, weight 0, slot -1).  The weight of a place is its score, divided by the sum of the row's
 * chosen scores if renormalize is set (0 where that sum is 0), times scale.  fp32 throughout: the
 * sigmoid of a logit below -88.7 is 0, so that a row of such logits alone has weights of 0.
 *
 * The taken places, sorted by expert and within an expert by row, are numbered from 0: these
 * numbers are the slots.  Slots [expert_offsets[e], expert_offsets[e + 1]) belong to expert e,
 * sorted_rows[slot] is the row of a slot, slots[row][j] the slot of a place; sorted_rows is -1 at
 * and past expert_offsets[n_experts].  All outputs are written whole.
 *
 * *num_rows outside [0, rows] is clamped and raises EAGLE3_DEV_CAPACITY.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t rows;             /* T >= 0                                                        */
    int32_t n_experts;        /* E, 1 .. 512                                                   */
    int32_t top_k;            /* k, 1 .. min(E, 16)                                            */
    int32_t scoring;          /* eagle3_moe_scoring_t                                          */
    int32_t renormalize;      /* 0 or 1                                                        */
    float scale;              /* factor of every weight, finite                                */
    int64_t ld_logits;        /* row pitch in elements, 0 = dense                              */
    const float *logits;      /* [T, E]                                                        */
    const int32_t *num_rows;  /* optional device word: only rows below it are routed           */
    int32_t *topk_ids;        /* [T, k]                                                        */
    float *topk_weights;      /* [T, k]                                                        */
    int32_t *expert_offsets;  /* [E + 1]                                                       */
    int32_t *sorted_rows;     /* [T * k]                                                       */
    int32_t *slots;           /* [T, k]                                                        */
    int32_t *dev_status;      /* optional EAGLE3_DEV_* word                                    */
} eagle3_moe_route_args_t;

size_t eagle3_moe_route_workspace_size(const eagle3_moe_route_args_t *args);
eagle3_status_t eagle3_moe_route(const eagle3_moe_route_args_t *args, void *workspace, size_t workspace_bytes,
                                 eagle3_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * eagle3_grouped_linear - out[s] = epilogue(x[r(s)] W[e]^T) for every slot s of every group e.
 *
 * Slots [offsets[e], offsets[e + 1]) use the weights of group e; r(s) = row_ids[s], or s itself
 * without row_ids.  Epilogues: EAGLE3_EPI_BF16 (out bf16), EAGLE3_EPI_SWIGLU
 * (out bf16 = silu(x W^T) * (x W2^T); silu of less than -87.3 is 0).  bf16 in, fp32 accumulation on the
 * tcgen05 tensor cores.
 * Groups may be empty.  Rows of out at or past offsets[n_groups] are left as they were.  With few rows
 * and columns the sum over k is cut into ranges that a thread-block cluster adds in order; the cut comes
 * from the shape and from how many CTAs the device holds, never from the offsets, so results are
 * reproducible on a given GPU model.
 *
 * EAGLE3_DEV_BAD_COUNTS (eagle3_chain.h) is raised when offsets do not start at 0, decrease or pass
 * m (out is then not written at all), and when a row id of a used slot is outside [0, n_src) (that
 * slot's output row is void).  out must not overlap x.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t n_groups;         /* E, 1 .. 512                                                   */
    int32_t m;                /* rows of out (slots), >= 0                                     */
    int32_t n, k;             /* output columns, contraction length (a multiple of 8)          */
    int32_t n_src;            /* rows of x with row_ids, >= 1 (ignored without: x has m rows)  */
    int32_t epilogue;         /* EAGLE3_EPI_BF16 or EAGLE3_EPI_SWIGLU                          */
    int64_t ld_x, ld_w, ld_out;   /* row pitches in elements, 0 = dense; ld_x, ld_w multiples of 8 */
    const uint16_t *x;        /* [n_src or m, k] bf16                                          */
    const uint16_t *w;        /* [E, n, k] bf16 (a group's rows ld_w apart, groups n * ld_w)   */
    const uint16_t *w2;       /* [E, n, k] bf16 (SWIGLU only)                                  */
    uint16_t *out;            /* [m, n] bf16                                                   */
    const int32_t *offsets;   /* [E + 1]                                                       */
    const int32_t *row_ids;   /* optional [m]                                                  */
    int32_t *dev_status;      /* optional EAGLE3_DEV_* word                                    */
} eagle3_grouped_linear_args_t;

eagle3_status_t eagle3_grouped_linear(const eagle3_grouped_linear_args_t *args, eagle3_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * eagle3_moe_combine - out[t] = residual[t] + sum over j of weights[t][j] * y[slots[t][j]].
 *
 * The sum runs over the places with slots[t][j] >= 0, in order of j, in fp32, the residual added
 * last, and is rounded to bf16 once.  An empty place adds nothing whatever its weight.  A slot at
 * or past n_slots is taken as empty and raises EAGLE3_DEV_BAD_COUNTS.  out may be the residual
 * buffer itself; it must not overlap y.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t rows;             /* T >= 0                                                        */
    int32_t n_slots;          /* rows of y, >= 0                                               */
    int32_t top_k;            /* k, 1 .. 16                                                    */
    int32_t dim;              /* d >= 1                                                        */
    int64_t ld_y, ld_res, ld_out;  /* row pitches in elements, 0 = dense                       */
    const uint16_t *y;        /* [n_slots, d] bf16                                             */
    const int32_t *slots;     /* [T, k]                                                        */
    const float *weights;     /* [T, k]                                                        */
    const uint16_t *residual; /* optional [T, d] bf16                                          */
    uint16_t *out;            /* [T, d] bf16                                                   */
    int32_t *dev_status;      /* optional EAGLE3_DEV_* word                                    */
} eagle3_moe_combine_args_t;

eagle3_status_t eagle3_moe_combine(const eagle3_moe_combine_args_t *args, eagle3_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EAGLE3_MOE_H */
