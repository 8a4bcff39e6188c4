/*
 * libmoe, block-scaled FP8 experts: products of E4M3 rows with E4M3 expert
 * matrices on the matrix instructions of gfx950 that multiply 128 codes at
 * once, a scale for each 128 columns of a row and for each 128 x 128 block of a
 * matrix, and the grouped SwiGLU FFN built from them.
 *
 * The conventions, status codes and types are libmoe.h's.  Codes are E4M3 bytes
 * (the finite ones with NaN at 0x7f and 0xff).
 *
 * Quantisation, the same everywhere: of 128 neighbouring columns v of a row (the
 * row's last ones may be fewer)
 *     scale = max |v| * c in fp32, c the fp32 number nearest to 1 / 448 (1 where
 *             the product is below 2^-100)
 *     code  = fl(v / scale) in fp32, to the nearest E4M3 value, halves to even.
 * Values that are not all finite give the scale NaN and codes 0, so that what is
 * computed from them is NaN.
 *
 * Packed matrices: a matrix C [R][K] of an expert (R and K multiples of 16 and
 * 64) is stored as blocks of 16 rows x 64 codes (1 KiB), block (r / 16, k / 64) at
 * byte ((r / 16) * (K / 64) + k / 64) * 1024 of the expert's matrix and C[r][k] at
 * (((k % 64) / 16) * 16 + r % 16) * 16 + k % 16 inside it: the layout of
 * moe_grouped_ffn_fp8w_packed and of the int8 products.
 */
#ifndef LIBMOE_FP8_H
#define LIBMOE_FP8_H

#include "libmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns of a row, and rows and columns of a matrix, that share one scale. */
#define MOE_FP8_BLOCK 128

/*
 * moe_quantize_blocks_fp8 - E4M3 codes of rows, a scale for each 128 columns.
 *
 *   x  [T][d] bf16 or fp32 (`dtype`), read only.
 *   q  [T][d] E4M3 bytes, written.    s  [T][ceil(d / 128)] fp32, written.
 *   Requires T >= 0, d a positive multiple of 8; x and q 16- and 8-byte
 *   aligned, s 4-byte.  T * d may pass int32.
 *   Errors: MOE_ERR_INVALID_ARG for negative sizes, NULL or misaligned
 *   pointers; MOE_ERR_UNSUPPORTED for d not a multiple of 8, an unknown dtype,
 *   T * ceil(d / 128) past int32.
 */
moe_status moe_quantize_blocks_fp8(const void* x, moe_dtype dtype, int32_t T, int32_t d, void* q, float* s,
                                   hipStream_t stream);

/*
 * moe_grouped_linear_fp8 - the product of each group's E4M3 rows with its
 * expert's E4M3 matrix:
 *     y[n][o] = sum over blocks b of 128 columns of
 *               x_scale[r][b] * w_scale[e][o / 128][b] * sum over k in b of xq[r][k] * w[e][o][k],
 * r = x_rows[n] (n without a row list), e the expert of sorted row n's group.
 * Sums are fp32 (a block's inside the matrix instruction, then over the blocks),
 * and the result is rounded once to `out_dtype`.  With a bf16 result the products of
 * large groups may be those of the FP8 matrix instructions, which cut each product to
 * a multiple of 2^(e - 13), e the exponent of the largest of eight neighbouring columns'
 * products: an error of some 2^-15 of a sum, where bf16's rounding is 2^-9.
 *
 *   xq       [n_x][K] E4M3 (n_x = n_rows without a row list), read only.
 *   x_scale  [n_x][ceil(K / 128)] fp32.
 *   x_rows   [n_rows] int32 or NULL, as in moe_grouped_ffn; entries are clamped
 *            to [0, n_x).
 *   group_offsets [G+1] int32, G = nseg*E + n_shared, as in moe_grouped_ffn:
 *            rows before group_offsets[0] or from group_offsets[G] on are left as
 *            they were.  E = 1, n_shared = 0, nseg = 1 with offsets {0, n_rows} is
 *            an ordinary linear map.
 *   w        [E+n_shared][O][K] E4M3, packed (above).
 *   w_scale  [E+n_shared][ceil(O / 128)][ceil(K / 128)] fp32.
 *   y        [n_rows][O] of `out_dtype` (bf16 or fp32), written.
 *   More than 800 groups (512 experts with a priority segment) run on the kernel of
 *   small groups however many rows they have: fp32 sums, at a lower rate.
 *   Requires n_rows <= 2^24, K and O positive multiples of 64, nseg in {1, 2},
 *   1 <= E <= 512, n_shared <= 256; tensors of codes and values 16-byte aligned,
 *   scales 4-byte.
 *   Errors: MOE_ERR_INVALID_ARG for negative sizes, nseg, NULL or misaligned
 *   pointers, n_x < 1 with a row list; MOE_ERR_UNSUPPORTED for the other
 *   requirements and element counts of xq and y past int32.
 */
moe_status moe_grouped_linear_fp8(const void* xq, const float* x_scale, const int32_t* x_rows, int32_t n_x,
                                  const int32_t* group_offsets, int32_t n_rows, int32_t E, int32_t n_shared,
                                  int32_t nseg, int32_t K, int32_t O, const void* w, const float* w_scale,
                                  moe_dtype out_dtype, void* y, hipStream_t stream);

/*
 * moe_grouped_ffn_fp8 - the grouped SwiGLU expert FFN on block-scaled E4M3 rows
 * and weights (moe_rmsnorm or moe_quantize_blocks_fp8 make the rows), bf16 out:
 *     g = x . W_gate,  u = x . W_up   as in moe_grouped_linear_fp8 with an fp32 result
 *     a = silu(g) * u in fp32, as codes and a scale for each 128 columns
 *     h = a . W_down                  as in moe_grouped_linear_fp8 with a bf16 result.
 * g, u, silu, the scales and the quotients are fp32 steps whatever the batch (the
 * hardware's exponential and reciprocal among them), so a code whose quotient lies
 * next to a border between two codes may be the neighbour.  A block of the SwiGLU product
 * whose scale is below 2^-100 counts as zeros.
 *
 *   xq, x_scale    as in moe_grouped_linear_fp8 with K = d.
 *   x_rows, n_x, group_offsets, n_rows, E, n_shared, nseg: likewise.
 *   w_gate, w_up   [E+n_shared][I][d] E4M3, packed; s_gate, s_up
 *                  [E+n_shared][ceil(I / 128)][ceil(d / 128)].
 *   w_down         [E+n_shared][d][I] E4M3, packed; s_down
 *                  [E+n_shared][ceil(d / 128)][ceil(I / 128)].
 *   h_sorted       [n_rows][d] bf16, written.
 *   workspace      of the queried size, whose contents need no preparation: the
 *                  SwiGLU product in codes and block scales (few rows: in fp32).  The
 *                  size depends on n_rows and I only.  Calls that share a
 *                  workspace, replayed graphs among them, must not overlap in time.
 *   Requires n_rows <= 2^24, d and I positive multiples of 64.
 *   Errors: as moe_grouped_linear_fp8 (the element counts are those of xq, of the
 *   SwiGLU product and of h_sorted); MOE_ERR_WORKSPACE for too small a workspace.
 */
moe_status moe_grouped_ffn_fp8(const void* xq, const float* x_scale, const int32_t* x_rows, int32_t n_x,
                               const int32_t* group_offsets, int32_t n_rows, int32_t E, int32_t n_shared,
                               int32_t nseg, int32_t d, int32_t I, const void* w_gate, const float* s_gate,
                               const void* w_up, const float* s_up, const void* w_down, const float* s_down,
                               void* h_sorted, void* workspace, size_t* workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMOE_FP8_H */
