/*
 * libmoe, int8 experts: products of int8 rows with int8 expert matrices on the
 * integer matrix instructions, with one scale per token and per output
 * channel, and the grouped SwiGLU FFN built from them.
 *
 * The conventions, status codes and types are libmoe.h's.
 *
 * Quantisation, the same everywhere: of a row of values v (a token's hidden
 * state, or 128 columns of the SwiGLU product)
 *     scale = max |v| * c in fp32, c the fp32 number nearest to 1 / 127 (1 where the
 *             product is 0)
 *     code  = v / scale rounded to the nearest integer, halves to even, the
 *             quotient exact, held to [-127, 127].
 * Values that are not all finite give the scale NaN and codes 0, so that what is
 * computed from them is NaN.
 *
 * Packed int8 matrices: a matrix C [R][K] of an expert (R and K multiples of 16
 * and 64) is stored as blocks of 16 rows x 64 codes (1 KiB), block (r / 16,
 * k / 64) at byte ((r / 16) * (K / 64) + k / 64) * 1024 of the expert's matrix
 * and C[r][k] at (((k % 64) / 16) * 16 + r % 16) * 16 + k % 16 inside it: the
 * layout of moe_grouped_ffn_fp8w_packed, so that one load instruction of a
 * wavefront reads one contiguous KiB, which is one matrix-instruction operand.
 */
#ifndef LIBMOE_INT8_H
#define LIBMOE_INT8_H

#include "libmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns of the SwiGLU product that share one scale in moe_grouped_ffn_i8. */
#define MOE_I8_BLOCK 128

/*
 * moe_quantize_rows_i8 - int8 codes and one scale per row.
 *
 *   x  [T][d] bf16 or fp32 (`dtype`), read only.
 *   q  [T][d] int8, written: the codes.    s  [T] fp32, written: the scales.
 *   Requires T >= 0, d a positive multiple of 8; x and q 16- and 8-byte
 *   aligned, s 4-byte.
 *   Errors: MOE_ERR_INVALID_ARG for negative sizes, NULL or misaligned
 *   pointers; MOE_ERR_UNSUPPORTED for d not a multiple of 8, an unknown dtype,
 *   T * d past int32.
 */
moe_status moe_quantize_rows_i8(const void* x, moe_dtype dtype, int32_t T, int32_t d, int8_t* q, float* s,
                                hipStream_t stream);

/*
 * moe_grouped_linear_i8 - the product of each group's int8 rows with its
 * expert's int8 matrix:
 *     y[n][o] = x_scale[r] * w_scale[e][o] * sum_k xq[r][k] * w[e][o][k],
 * r = x_rows[n] (n without a row list), e the expert of sorted row n's group.
 * The sums are exact int32; the two scales multiply in fp32 and the result is
 * rounded once to `out_dtype`.
 *
 *   xq       [n_x][K] int8 (n_x = n_rows without a row list), read only.
 *   x_scale  [n_x] fp32.
 *   x_rows   [n_rows] int32 or NULL, as in moe_grouped_ffn; entries are clamped
 *            to [0, n_x).
 *   group_offsets [G+1] int32, G = nseg*E + n_shared, as in moe_grouped_ffn:
 *            rows before group_offsets[0] or from group_offsets[G] on are left as
 *            they were.  E = 1, n_shared = 0, nseg = 1 with offsets {0, n_rows} is
 *            an ordinary linear map.
 *   w        [E+n_shared][O][K] int8, packed (above).  w_scale [E+n_shared][O].
 *   y        [n_rows][O] of `out_dtype` (bf16 or fp32), written.
 *   Requires n_rows <= 2^24, K and O positive multiples of 64, K <= 131072 (the
 *   sums of codes in [-127, 127] stay in int32), nseg in {1, 2}, 1 <= E <= 512, n_shared <= 256; tensors of codes and
 *   values 16-byte aligned, w_scale 16-byte, x_scale 4-byte.
 *   Errors: MOE_ERR_INVALID_ARG for negative sizes, nseg, NULL or misaligned
 *   pointers, n_x < 1 with a row list; MOE_ERR_UNSUPPORTED for the other
 *   requirements and element counts of xq and y past int32.
 */
moe_status moe_grouped_linear_i8(const int8_t* xq, const float* x_scale, const int32_t* x_rows, int32_t n_x,
                                 const int32_t* group_offsets, int32_t n_rows, int32_t E, int32_t n_shared,
                                 int32_t nseg, int32_t K, int32_t O, const int8_t* w, const float* w_scale,
                                 moe_dtype out_dtype, void* y, hipStream_t stream);

/*
 * moe_grouped_ffn_i8 - the grouped SwiGLU expert FFN of moe_grouped_ffn on int8
 * weights and int8 activations (bf16 in and out):
 *     xq, sx = the token rows quantised per row
 *     g = sx * s_gate * (xq . W_gate),  u = sx * s_up * (xq . W_up)   exact int32 sums
 *     a = silu(g) * u in fp32, quantised per row and MOE_I8_BLOCK columns -> aq, sa
 *     h = s_down * sum over the blocks b of sa[b] * (aq . W_down over b)  (fp32 over the
 *         blocks, exact int32 inside one), rounded once to bf16.
 * A block of the SwiGLU product whose scale is below 2^-126 counts as zeros.
 * g, u, silu and the scales are fp32 steps (the hardware's exponential and
 * reciprocal among them), so a code whose exact quotient lies within
 *     2^-16 * (22 + 2.2 * (n + m)) codes,  n = max(0, -g), m the largest n of the block,
 * of a border may be the neighbour (measured: 1.4e-4 near g = -20, 3.2e-4 near
 * -55), and a value of g below -87 may count as 0.
 *
 *   x_sorted, x_rows, n_x, group_offsets, n_rows, E, n_shared, nseg, h_sorted: as
 *                  moe_grouped_ffn with dtype MOE_BF16.  All n_x token rows are
 *                  quantised, once each however many sorted rows read them (a
 *                  batch of few rows quantises them where it multiplies).
 *   w_gate, w_up   [E+n_shared][I][d] int8, packed; s_gate, s_up [E+n_shared][I].
 *   w_down         [E+n_shared][d][I] int8, packed; s_down [E+n_shared][d].
 *   workspace      of the queried size, whose contents need no preparation: the
 *                  token codes and scales, the SwiGLU product in codes and block
 *                  scales (few rows: in fp32).  The size depends on n_rows, n_x
 *                  (where a row list is given; the query takes x_rows' presence
 *                  from n_x > 0), d and I only.  Calls that share a workspace,
 *                  replayed graphs among them, must not overlap in time.
 *   Requires n_rows <= 2^24, d and I positive multiples of 64, d <= 131072.
 *   Errors: as moe_grouped_ffn_fp8w_packed.
 */
moe_status moe_grouped_ffn_i8(const void* x_sorted, const int32_t* x_rows, int32_t n_x,
                              const int32_t* group_offsets, int32_t n_rows, int32_t E, int32_t n_shared,
                              int32_t nseg, int32_t d, int32_t I, const int8_t* w_gate, const float* s_gate,
                              const int8_t* w_up, const float* s_up, const int8_t* w_down, const float* s_down,
                              void* h_sorted, void* workspace, size_t* workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMOE_INT8_H */
