/*
 * eagle3_fp8.h - 8-bit projections of libeagle3 (building blocks).
 *
 * The bias-free projections of "EAGLE-3: Engineering Implementation of LLM Inference Acceleration",
 * section VIII and appendix C (out = x W^T), for a target whose weights are held in e4m3 with one
 * fp32 scale for each 128 x 128 block: eagle3_linear's counterpart at half the weight bytes and
 * twice the tensor-core rate.  Activations are e4m3 with one scale for each row and 128 columns,
 * made by eagle3_quantize_fp8.
 *
 * Conventions as in eagle3.h: asynchronous on the stream, host-detected errors returned before any
 * launch, caller-owned device memory.  e4m3 is the variant without infinities (largest value 448,
 * NaN 0x7F / 0xFF).
 */
#ifndef EAGLE3_FP8_H
#define EAGLE3_FP8_H

#include "eagle3.h"
#include "eagle3_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------------
 * eagle3_quantize_fp8 - rows of bf16 to e4m3 with a scale for each row and 128 columns.
 *
 * For row r and columns [128 b, min(128 b + 128, k)): a = max |x|, s = a / 448 (1 where a is 0),
 * q = e4m3(x / s), both divisions and the conversion rounded to nearest even, the quotient cut to
 * +-448.  scale[b][r] = s.  A block that holds a NaN or an infinity gets the scale NaN and values
 * NaN, so that every product with it is NaN.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t rows;             /* m >= 0                                                        */
    int32_t k;                /* a multiple of 16                                              */
    int64_t ld_x, ld_q;       /* row pitches in elements, 0 = dense; multiples of 8 and 16     */
    const uint16_t *x;        /* [m, k] bf16                                                   */
    uint8_t *q;               /* [m, k] e4m3                                                   */
    float *scale;             /* [ceil(k / 128), m] fp32                                       */
} eagle3_quantize_fp8_args_t;

eagle3_status_t eagle3_quantize_fp8(const eagle3_quantize_fp8_args_t *args, eagle3_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * eagle3_linear_fp8 - out = epilogue(y),
 *   y[r][c] = sum over b of x_scale[b][r] * w_scale[c / 128][b] *
 *             (sum over i in [128 b, min(128 b + 128, k)) of x[r][i] * w[c][i]).
 *
 * The inner sums run on the tcgen05 tensor cores (products exact, fp32 accumulation over one block
 * of 128), the outer one in fp32 registers.  Epilogues as in eagle3_linear.h: EAGLE3_EPI_BF16,
 * EAGLE3_EPI_F32, EAGLE3_EPI_BF16_RESIDUAL (out may be the residual buffer itself) and
 * EAGLE3_EPI_SWIGLU (silu(y) * y2 with y2 from w2, w2_scale; silu of less than -87.3 is 0).  A NaN
 * among the values or the scales makes the outputs that read it NaN.  Scales may be 0, subnormal or
 * negative; x_scale * w_scale, and x_scale times an inner sum (at most 448 * 448 * 128), have to stay
 * below fp32's largest number, and lose bits where they fall below its smallest normal one.  Where the
 * output has few tiles the sum over b is cut into ranges that a thread-block cluster adds in order;
 * the cut comes from the shape and from how many CTAs the device holds, so results are reproducible on
 * a given GPU model.
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
    int32_t m, n, k;          /* rows of x, rows of W (= output columns), contraction (k % 16 == 0) */
    int32_t epilogue;         /* eagle3_epilogue_t, without EAGLE3_EPI_BF16_ROPE               */
    int64_t ld_x, ld_w, ld_out, ld_res;   /* row pitches in elements, 0 = dense; ld_x, ld_w multiples of 16 */
    const uint8_t *x;         /* [m, k] e4m3                                                   */
    const float *x_scale;     /* [ceil(k / 128), m]                                            */
    const uint8_t *w;         /* [n, k] e4m3                                                   */
    const float *w_scale;     /* [ceil(n / 128), ceil(k / 128)]                                */
    const uint8_t *w2;        /* [n, k] e4m3 (SWIGLU only)                                     */
    const float *w2_scale;    /* [ceil(n / 128), ceil(k / 128)] (SWIGLU only)                  */
    void *out;                /* [m, n] bf16 or fp32                                           */
    const uint16_t *residual; /* [m, n] bf16 (BF16_RESIDUAL only)                              */
    int32_t *dev_status;      /* optional EAGLE3_DEV_* word                                    */
} eagle3_linear_fp8_args_t;

eagle3_status_t eagle3_linear_fp8(const eagle3_linear_fp8_args_t *args, eagle3_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EAGLE3_FP8_H */
