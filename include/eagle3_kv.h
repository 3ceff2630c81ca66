/*
 * eagle3_kv.h - an 8-bit paged KV cache and the rotary positions of its keys (building blocks).
 *
 * For a target whose cache is held in e4m3, what eagle3_verify_attn and eagle3_compact_kv do for a
 * bf16 cache ("Advanced speculative decoding: tree drafts and EAGLE", "Implementation"; paging as in
 * "Speculative Decoding (EAGLE3) in the vLLM Neuron Framework", "EagleProposer: Draft Model
 * Management"):
 *   rotary positions, also scaled for long contexts    eagle3_rope_table, eagle3_rope
 *   new tokens' keys and values into the cache          eagle3_append_kv
 *   attention of single tokens or of a tree's nodes     eagle3_verify_attn_fp8
 *
 * The cache.  Position p of sequence b lies on page block_table[b][p / block_size] at place
 * p % block_size.  An e4m3 pool is [pages, Hkv, block_size, D] codes, so that one head's part of a page is
 * one run of memory, with one scale byte for each page, KV head and group of 64 places,
 * [pages, Hkv, block_size / 64]: byte s stands for 2^(s - 127) (255 for NaN), and a code c for
 * e4m3(c) * 2^(s - 127).  Powers of two because e4m3 carries its precision in an exponent of its own: a
 * finer scale would gain nothing but in the subnormals, and this one moves older codes exactly when a
 * later token makes it grow.  e4m3 is the variant without infinities (largest value 448, NaN 0x7F / 0xFF).
 * A bf16 pool is [pages * block_size, Hkv, D], as eagle3_verify_attn reads it.
 *
 * Conventions as in eagle3.h: asynchronous on the stream, host-detected errors returned before any
 * launch, caller-owned device memory, scratch in a caller workspace (its contents need no preparation
 * and mean nothing between calls).  Lengths and counts are read on the device, so that a sequence of
 * calls can be captured into a CUDA graph.
 */
#ifndef EAGLE3_KV_H
#define EAGLE3_KV_H

#include "eagle3.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EAGLE3_KV_GROUP 64          /* places of a page that share a scale                          */
#define EAGLE3_ROPE_MAX_DIM 256

/* ------------------------------------------------------------------------------------------------
 * eagle3_rope_table - the angles of rotary positions: for the pairs j = 0 .. rotary_dim / 2 - 1,
 *   table[j] = 2^64 * (f_j / (2 pi)) mod 2^64, rounded: the turns of one position as a 64-bit fraction.
 * Position p then stands at p * table[j] mod 2^64, which integers give exactly at any distance (a
 * product in fp32 is off by 0.008 radians at position 131072).  With f = theta^(-2 j / rotary_dim):
 *   EAGLE3_ROPE_NONE    f_j = f
 *   EAGLE3_ROPE_LINEAR  f_j = f / factor
 *   EAGLE3_ROPE_BASE    f_j = f of the base theta * factor^(R / (R - 2)), R = rotary_dim > 2
 *   EAGLE3_ROPE_BANDS   (Llama 3.1) t = original_positions * f / (2 pi) turns over the original context;
 *                       f_j = k f + (1 - k) f / factor, k = (t - low_turns) / (high_turns - low_turns)
 *                       cut to [0, 1]
 *   EAGLE3_ROPE_RAMP    (YaRN) f_j = (1 - k) f + k f / factor, k = (j - lo) / max(hi - lo, 0.001) cut to
 *                       [0, 1], lo = max(floor(d(high_turns)), 0), hi = min(ceil(d(low_turns)), R - 1),
 *                       d(t) = R ln(original_positions / (2 pi t)) / (2 ln theta)
 * computed on the host in fp64.  A program makes it once and keeps it.
 * ---------------------------------------------------------------------------------------------- */
typedef enum {
    EAGLE3_ROPE_NONE = 0,
    EAGLE3_ROPE_LINEAR = 1,
    EAGLE3_ROPE_BASE = 2,
    EAGLE3_ROPE_BANDS = 3,
    EAGLE3_ROPE_RAMP = 4
} eagle3_rope_scaling_t;

typedef enum {
    EAGLE3_ROPE_HALF = 0,        /* pair j: dims j and j + rotary_dim / 2                             */
    EAGLE3_ROPE_INTERLEAVED = 1  /* pair j: dims 2 j and 2 j + 1                                      */
} eagle3_rope_layout_t;

typedef struct {
    int32_t rotary_dim;          /* R: even, 2 .. EAGLE3_ROPE_MAX_DIM                                 */
    int32_t scaling;             /* eagle3_rope_scaling_t                                             */
    int32_t original_positions;  /* BANDS, RAMP: >= 1                                                 */
    double theta;                /* > 1                                                               */
    double factor;               /* all but NONE: >= 1                                                */
    double low_turns, high_turns; /* BANDS, RAMP: 0 < low_turns < high_turns                          */
    uint64_t *table;             /* [R / 2] out                                                       */
} eagle3_rope_table_args_t;

eagle3_status_t eagle3_rope_table(const eagle3_rope_table_args_t *args, eagle3_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * eagle3_rope - rotary positions of rows of heads.  For row r, head h and pair j (dims a and b), with
 * the angle t = 2 pi * (positions[r] * table[j] mod 2^64) / 2^64:
 *   out[a] = amplitude * (x[a] cos t - x[b] sin t)
 *   out[b] = amplitude * (x[b] cos t + x[a] sin t)
 * and dims past rotary_dim are copied.  fp32 arithmetic, rounded once.  inverse turns by -t: with the
 * same amplitude, the gradient of x from that of out.  out may be x itself, with the same pitch (views
 * that overlap in any other way are not allowed).  Positions may be negative.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t rows;                /* >= 0                                                              */
    int32_t n_heads;             /* >= 1                                                              */
    int32_t head_dim;            /* D: a multiple of 8, <= EAGLE3_ROPE_MAX_DIM                        */
    int32_t rotary_dim;          /* R: even, 2 .. D                                                   */
    int32_t elem_bytes;          /* 2 (bf16) or 4 (fp32)                                              */
    int32_t layout;              /* eagle3_rope_layout_t                                              */
    int32_t inverse;             /* 0 or 1                                                            */
    float amplitude;             /* finite; e.g. 1 (YaRN: 0.1 ln(factor) + 1)                         */
    int64_t x_row_stride;        /* elements between rows, 0 = n_heads * D; a multiple of 16 bytes    */
    int64_t out_row_stride;
    const void *x;               /* [rows, n_heads, D], heads dense                                   */
    const int32_t *positions;    /* [rows]                                                            */
    const uint64_t *table;       /* [R / 2] from eagle3_rope_table                                    */
    void *out;                   /* [rows, n_heads, D], heads dense                                   */
} eagle3_rope_args_t;

eagle3_status_t eagle3_rope(const eagle3_rope_args_t *args, eagle3_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * eagle3_append_kv - keys and values of new tokens into a paged cache, keys rotated on the way.
 *
 * Token j < n_new[b] of sequence b goes to position p = cache_len[b] + j.  Its row of k_new / v_new is
 *   row_start[b] + j                        (row_start given: packed rows), or
 *   b * max_new + j                         (neither: rows padded to max_new), or
 *   b * rows_per_seq + row_ids[b][j]        (row_ids given; e.g. the nodes of an accepted path).
 * Without n_new a sequence's tokens end before its first negative row id.  With a rope table the first
 * rotary_dim dims of every key are turned to position p as by eagle3_rope (fp32, not rounded between);
 * without one the keys arrive rotated.  cache_len is read and not advanced: the layers of a model share it.
 *
 * EAGLE3_KV_BF16: the rows are stored rounded to bf16.
 * EAGLE3_KV_E4M3: let m be the largest magnitude of the new tokens' finite values in a group of 64
 * places of one head (keys and values apart), s the least byte >= 1 with m <= 448 * 2^(s - 127).  Where
 * the group holds older tokens (places before cache_len[b]) and their scale byte is larger, that one
 * stays; where s is larger it becomes the group's scale and the older codes are rounded again to the
 * scale that grew.  New codes are the values over the scale, rounded to nearest even.  Infinities and NaN become NaN
 * codes and take no part in m.  Places that no token goes to keep their codes.
 *
 * n_new[b] outside [0, max_new], cache_len[b] < 0 or a last position past max_blocks * block_size: the
 * sequence is left out and EAGLE3_DEV_CAPACITY raised.  A page id outside the pool: what would go there is left
 * out (E4M3: the group; BF16, whose pages may end inside a group: the tokens of that page) and
 * EAGLE3_DEV_CAPACITY raised.  A row outside [0, n_rows) (with row_ids: outside
 * [0, rows_per_seq) of its sequence): the token is left out and EAGLE3_DEV_BAD_TOKEN raised.
 * A page that is written must belong to one sequence.  batch * (groups of 64 that max_new tokens can touch) *
 * 2 * n_kv_heads must be below 2^31 - 2^16.
 * ---------------------------------------------------------------------------------------------- */
typedef enum {
    EAGLE3_KV_BF16 = 0,
    EAGLE3_KV_E4M3 = 1
} eagle3_kv_format_t;

typedef struct {
    int32_t batch;               /* B >= 0                                                            */
    int32_t n_kv_heads;          /* Hkv >= 1                                                          */
    int32_t head_dim;            /* D: a multiple of 8, <= 256                                        */
    int32_t format;              /* eagle3_kv_format_t                                                */
    int32_t n_rows;              /* rows of k_new / v_new, >= 0 (0: they may be NULL)                 */
    int32_t max_new;             /* host bound on every sequence's new tokens, >= 0                   */
    int32_t rows_per_seq;        /* row_ids only: rows of a sequence                                  */
    int32_t max_blocks;          /* columns of block_table                                            */
    int32_t block_size;          /* places of a page: >= 1; E4M3: a multiple of 64                    */
    int32_t n_pages;             /* pages of the pool                                                 */
    int32_t rotary_dim;          /* R: even, 2 .. D; read with rope_table only                        */
    int32_t rope_layout;         /* eagle3_rope_layout_t                                              */
    float rope_amplitude;        /* finite                                                            */
    int64_t row_stride;          /* elements between rows of k_new / v_new, 0 = Hkv * D; a multiple of 8 */
    const uint16_t *k_new;       /* [n_rows, Hkv, D] bf16, heads dense                                */
    const uint16_t *v_new;
    const int32_t *cache_len;    /* [B]                                                               */
    const int32_t *n_new;        /* [B]; NULL with row_ids only                                       */
    const int32_t *row_start;    /* [B] or NULL                                                       */
    const int32_t *row_ids;      /* [B, max_new] or NULL (not both)                                   */
    const int32_t *block_table;  /* [B, max_blocks] page ids                                          */
    const uint64_t *rope_table;  /* [R / 2] or NULL                                                   */
    void *k_cache;               /* BF16: [n_pages * block_size, Hkv, D]                              */
    void *v_cache;               /* E4M3: [n_pages, Hkv, block_size, D]                               */
    uint8_t *k_scale;            /* E4M3: [n_pages, Hkv, block_size / 64]                             */
    uint8_t *v_scale;
    int32_t *dev_status;         /* optional EAGLE3_DEV_* word                                        */
} eagle3_append_kv_args_t;

eagle3_status_t eagle3_append_kv(const eagle3_append_kv_args_t *args, eagle3_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * eagle3_verify_attn_fp8 - eagle3_verify_attn over an e4m3 cache, for single tokens as for trees.
 *
 * For each sequence b (L = prefix_len[b]), node i and query head h (KV head g = h / (Hq / Hkv)):
 *   out[b,i,h] = sum_j softmax_j(q_i . k_j * sm_scale) v_j over the cache positions 0 .. L - 1 and, with
 *                tree_k, the tree nodes that are i or an ancestor of i.
 * q and tree_k arrive rotated.  Without tree_k (parents and tree_v are then NULL too) the queries see the
 * cache alone, all of it: a single token whose own key has been appended, or n_nodes queries over a shared
 * prefix.  A query that sees no key gets zeros and lse = -inf.  lse (optional) is the natural logarithm of
 * the sum of exp of the scaled scores.
 * Codes and scales of positions >= L are not looked at and may be anything.  Before L a NaN code or scale of K
 * makes out and lse of the queries that see it NaN; one of V makes out NaN (a code: its dim), and lse, which has no
 * values in it, stays what the keys make it.  A page id outside the pool reads as keys and values of
 * zero.  prefix_len[b] outside [0, max_prefix_len] is cut and raises EAGLE3_DEV_CAPACITY; a tree that is
 * not one raises EAGLE3_DEV_BAD_TREE and its nodes end at the bad one.
 * Scores, softmax statistics and sums are fp32.  q and tree_k enter the tensor cores as fp16, scaled by a power
 * of two of their own, or, with many query rows a KV head (more than 16 of n_nodes * Hq / Hkv; batch and
 * max_prefix_len decide too), as two e4m3 parts: 8 bits, but no finer than 2^-17 of the row's (of the tree's)
 * largest element, and infinities as NaN.  Weights are rounded to fp16 (11 bits); V's codes are exact where their scale is above
 * 2^-21 of the sequence's largest, and at any scale no finer than 2^-31 of that.  Where work is cut depends
 * on the lengths, max_prefix_len, the shape and the number of SMs: results are reproducible for the same call on a given
 * GPU model.  Where few query rows are read at a time, a max_prefix_len far above the lengths costs time.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t batch;               /* B >= 0                                                            */
    int32_t n_nodes;             /* N in [1, 64]                                                      */
    int32_t n_heads;             /* Hq, a multiple of n_kv_heads                                      */
    int32_t n_kv_heads;          /* Hkv                                                               */
    int32_t head_dim;            /* D; 128 is supported                                               */
    int32_t max_prefix_len;      /* host bound on prefix_len[b], >= 0                                 */
    int32_t num_splits;          /* parts of the prefix (more than 512 are 512); 0 = choose automatically */
    int32_t max_blocks;          /* columns of block_table; max_blocks * block_size >= max_prefix_len */
    int32_t block_size;          /* places of a page, a multiple of 64                                */
    int32_t n_pages;             /* pages of the pool                                                 */
    float sm_scale;              /* 0 = 1/sqrt(D)                                                     */
    int64_t q_node_stride;       /* elements between nodes of q, 0 = Hq * D; a multiple of 8          */
    int64_t kv_node_stride;      /* elements between nodes of tree_k / tree_v, 0 = Hkv * D; a multiple of 8 */
    const uint16_t *q;           /* [B, N, Hq, D] bf16, rotated                                       */
    const uint16_t *tree_k;      /* [B, N, Hkv, D] bf16, rotated, or NULL                             */
    const uint16_t *tree_v;      /* [B, N, Hkv, D] bf16, or NULL                                      */
    const int32_t *parents;      /* [B, N] or NULL                                                    */
    const uint8_t *k_cache;      /* [n_pages, Hkv, block_size, D] e4m3                                */
    const uint8_t *v_cache;
    const uint8_t *k_scale;      /* [n_pages, Hkv, block_size / 64]                                   */
    const uint8_t *v_scale;
    const int32_t *block_table;  /* [B, max_blocks] page ids                                          */
    const int32_t *prefix_len;   /* [B]                                                               */
    uint16_t *out;               /* [B, N, Hq, D] bf16                                                */
    float *lse;                  /* [B, N, Hq] fp32 or NULL                                           */
    int32_t *dev_status;         /* optional                                                          */
} eagle3_verify_attn_fp8_args_t;

size_t eagle3_verify_attn_fp8_workspace_size(const eagle3_verify_attn_fp8_args_t *args);
eagle3_status_t eagle3_verify_attn_fp8(const eagle3_verify_attn_fp8_args_t *args, void *workspace,
                                       size_t workspace_bytes, eagle3_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EAGLE3_KV_H */
