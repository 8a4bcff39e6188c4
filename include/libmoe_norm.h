/*
 * libmoe, norm: the root-mean-square norm in front of the router and the
 * experts, with the residual's addition before it and 8-bit codes behind it.
 *
 * The conventions, status codes and types are libmoe.h's.
 */
#ifndef LIBMOE_NORM_H
#define LIBMOE_NORM_H

#include "libmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Codes that moe_rmsnorm writes: none, int8 with one scale per row (the rows of
 * moe_grouped_linear_i8), or E4M3 with one scale per 128 columns (the rows of
 * moe_grouped_linear_fp8 and moe_grouped_ffn_fp8). */
typedef enum { MOE_CODE_NONE = 0, MOE_CODE_I8 = 1, MOE_CODE_FP8 = 2 } moe_code;

/*
 * moe_rmsnorm - of every row
 *     r    = x + residual in fp32, rounded to residual_dtype (r = x without a residual)
 *     rstd = 1 / sqrt(mean of r^2 + eps)                      in fp32
 *     p    = r * weight in fp32
 *     y    = p * rstd, rounded to y_dtype
 * and codes of p whose scales are multiplied by rstd, so that code * scale stands for
 * the same values (rstd multiplies the whole row and does not change its codes):
 *     MOE_CODE_I8   of each row        base = max |p| * fl(1 / 127) (1 where the product is 0)
 *                   code = p / base to the nearest integer, halves to even, the quotient
 *                   exact, held to [-127, 127]
 *     MOE_CODE_FP8  of each 128 columns (the last ones may be fewer)
 *                   base = max |p| * fl(1 / 448) (1 where the product is below 2^-100)
 *                   code = fl(p / base) to the nearest E4M3 value, halves to even
 *     scale = base * rstd in fp32.
 *
 *   x         [T][d] of x_dtype, read only.
 *   residual  [T][d] of residual_dtype or NULL.  residual_out [T][d] of the same type
 *             receives r; it may be `residual` itself (the sum in place) and is
 *             NULL exactly where residual is.
 *   weight    [d] of weight_dtype.
 *   y         [T][d] of y_dtype, or NULL: not written.
 *   q, s      codes [T][d] (int8, or E4M3 bytes) and scales [T] (MOE_CODE_I8) or
 *             [T][ceil(d / 128)] (MOE_CODE_FP8); unused with MOE_CODE_NONE.
 *   A row with a value that is not finite, or whose sum of squares is not in fp32,
 *   gives NaN in y and in its scales.  A row of zeros gives zeros.
 *   Apart from residual_out, outputs must not alias inputs.
 *   Requires T >= 0, d a positive multiple of 8, eps positive and finite; types bf16
 *   or fp32; x, residual, weight, y 16-byte aligned, q 8-byte, s 4-byte.  T * d may
 *   pass int32.
 *   Errors: MOE_ERR_INVALID_ARG for negative sizes, eps, an unknown code, nothing to
 *   write (no y and no codes), NULL or misaligned pointers, one of residual and
 *   residual_out alone; MOE_ERR_UNSUPPORTED for d not a multiple of 8, an unknown type (of
 *   a tensor that is given), T * ceil(d / 128) past int32.
 */
moe_status moe_rmsnorm(const void* x, moe_dtype x_dtype, const void* residual, moe_dtype residual_dtype,
                       const void* weight, moe_dtype weight_dtype, int32_t T, int32_t d, float eps,
                       void* residual_out, void* y, moe_dtype y_dtype, moe_code code, void* q, float* s,
                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMOE_NORM_H */
