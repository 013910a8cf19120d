/*
 * qgmm_mm.h -- C ABI of the grouped products without dequantisation or combine
 * (libqgmm_mm.so): rows sorted by expert times their expert's weights in bf16, fp16
 * or MXFP4, the two gradients of the bf16 / fp16 product, and the MXFP4 quantiser
 * that leads from one to the other.  (No counterpart on the pages, which cover
 * quantised inference: these are the products in which the experts are trained, and
 * the cast to the 4-bit form whose E2M1 weights page 1's MxA8W4 mode reads.)
 *
 *   off[] as in qgmm.h (group_list_type 0: cumulative ends, 1: counts); for every
 *   expert g and row i in [off[g], off[g+1]):
 *     y[i][j]   = sum_kk x[i][kk] * W(g, kk, j)             qgmm_grouped_mm
 *     dx[i][kk] = sum_j  dy[i][j] * W(g, kk, j)             qgmm_grouped_mm_dgrad
 *     dW(g, kk, j) = sum_i x[i][kk] * dy[i][j]              qgmm_grouped_mm_wgrad
 *
 * W(g, kk, j) is w[g][kk][j] (transpose_w 0) or w[g][j][kk] (transpose_w 1).  Sums
 * are f32 in the tensor core, which truncates, rounded once to out_type at the end (nearest
 * even); f32 outputs are added up outside it from sums of 512 terms (MXFP4: 8192), rounded, and
 * 16-bit y and dx of more than 8192 bf16 or fp16 terms from sums of 2048, fp16 dw of more than 8192
 * rows from sums of 8192, bf16 dw of more than 32768 from such.  A sum of n terms in the tensor
 * core comes out smaller by some 1e-9 n of itself, by 6e-9 n where all terms have one sign.
 * MXFP4 operands stand for q * 2^(s - 127), q an E2M1 value and s its block's E8M0
 * code (32 consecutive kk share one); a code of 255 stands for NaN.
 *
 * The conventions are those of qgmm.h: device pointers on the current device, memory
 * owned by the caller, nothing allocated, every call asynchronous on `cuda_stream`
 * and capturable in a CUDA graph, host checks before any launch, bad group lists
 * reported through the workspace's status word (qgmm_device_status) with the rows
 * they cover sanitised, bounded waits inside the kernels.  Calls that may overlap
 * need workspaces of their own, and no output may overlap an input or the workspace.
 */
#ifndef QGMM_MM_H
#define QGMM_MM_H

#include <stddef.h>
#include <stdint.h>

#include "qgmm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QGMM_T_BF16 = 0, QGMM_T_F16 = 1, QGMM_T_F32 = 2, QGMM_T_MXFP4 = 3 };   /* element types */

/*
 * One problem serves the product and both gradients.
 *   m    rows of x, 0 <= m <= 2^24.  Rows at or past the groups' total are neither
 *        read into a result nor written: y's and dx's stay as they were.
 *   k,n  8 <= k, n <= 65536, multiples of 8 (k a multiple of 32 for MXFP4)
 *   e    experts, 1 <= e <= 1024
 *   x_type      element type of x, w and dy: BF16, F16 or MXFP4 (both x and w)
 *   out_type    element type of the call's output: x_type or F32; with MXFP4 BF16, F16 or F32
 *   group_list_type   QGMM_GROUP_CUMSUM | QGMM_GROUP_COUNTS
 *   transpose_w 0: w (and dw) stored (e, k, n); 1: (e, n, k).  MXFP4 needs 1.
 *   accumulate  qgmm_grouped_mm_wgrad only: 1 adds to what dw holds (the sum in f32,
 *               rounded once), an expert without rows leaving its dw as it was; 0
 *               overwrites dw, an expert without rows getting zeros
 *   ld_x, ld_w, ld_y   elements from one row to the next of x (and dx), of w (and dw)
 *               and of y (and dy); 0 = dense.  Multiples of 8 (ld_x and ld_w of 32 with
 *               MXFP4, whose scale rows are then ld_x / 32 and ld_w / 32 apart), at
 *               least the row's length, ld_x and ld_y at most 2^32, ld_w at most 2^22.
 */
typedef struct {
    int64_t m, k, n, e;
    int32_t x_type, out_type, group_list_type, transpose_w, accumulate;
    int64_t ld_x, ld_w, ld_y;
} qgmm_mm_problem;

/*
 * Workspace bytes of any of the three calls with `p` (host pointers).  The first word
 * is the status word; the workspace needs no initialisation and carries nothing from
 * one call to the next.  The rest holds f32 parts of the sums of calls with few tiles and a
 * long sum, f32 sums of 16-bit weight gradients of more rows than that, and arranged scales of
 * MXFP4 calls with many rows.  What is returned is enough for the same problem with fewer rows, too
 * (a call is refused only below what it needs itself, which may be less).
 * 20 MB are enough for any bf16 or fp16 problem.
 * Errors: NULL_PTR, SHAPE, DTYPE, UNSUPPORTED (MXFP4 without transpose_w).
 */
qgmm_status qgmm_grouped_mm_workspace(const qgmm_mm_problem *p, size_t *ws_bytes);

/*
 * y = x W.  x [m, k], w [e, k, n] or [e, n, k], y [m, n] of out_type; x_scale and
 * w_scale are NULL except for MXFP4: E8M0 bytes [m, k/32] and [e, n, k/32], x and w
 * then E2M1 pairs [m, k/2] and [e, n, k/2], lower kk in the low nibble.  x, w, y and the
 * scales 16-byte aligned, workspace 256-byte.  x and
 * y may be NULL when m = 0 (only group_list is read then, and the status word written).
 * Errors: NULL_PTR, SHAPE, DTYPE, ALIGNMENT, WORKSPACE_TOO_SMALL, UNSUPPORTED (also
 * accumulate), CUDA.
 */
qgmm_status qgmm_grouped_mm(const qgmm_mm_problem *p, const void *x, const uint8_t *x_scale, const void *w,
                            const uint8_t *w_scale, const int64_t *group_list, void *y, void *workspace,
                            size_t ws_bytes, void *cuda_stream);

/*
 * dx = dy W^T: dy [m, n] of x_type, dx [m, k] of out_type.  As qgmm_grouped_mm
 * otherwise.  Errors: as qgmm_grouped_mm, UNSUPPORTED for MXFP4.
 */
qgmm_status qgmm_grouped_mm_dgrad(const qgmm_mm_problem *p, const void *dy, const void *w, const int64_t *group_list,
                                  void *dx, void *workspace, size_t ws_bytes, void *cuda_stream);

/*
 * dW = x^T dy for every expert, the expert's rows summed in an order that the problem and
 * group_list fix (bitwise reproducible): x [m, k] and dy [m, n] of x_type, dw
 * of out_type in w's layout.  With m = 0 and accumulate 0, dw is zeroed.
 * Errors: as qgmm_grouped_mm, UNSUPPORTED for MXFP4.
 */
qgmm_status qgmm_grouped_mm_wgrad(const qgmm_mm_problem *p, const void *x, const void *dy, const int64_t *group_list,
                                  void *dw, void *workspace, size_t ws_bytes, void *cuda_stream);

/*
 * MXFP4 quantisation, the 4-bit sibling of qgmm_per_token_quant_mxfp8.  For each 32
 * consecutive elements of a row:
 *   a  = max |x|;  sf = max(0, biased f32 exponent of a - 2)     (E8M0 code)
 *   q  = E2M1(x * 2^(127 - sf)), round to nearest even, magnitudes past 6 saturate
 * so the largest magnitude lands in E2M1's top binade.  x * 2^(127 - sf) is exact
 * (what f32 cannot hold of it rounds to 0 anyway); the conversion is the only
 * rounding.  A NaN in a block makes its code 255 and its q 0: the block stands for
 * NaN.  An infinity makes sf 253 and its q 6, whose value overflows f32 to infinity.
 *   x       [rows, k] BF16, F16 or F32 by x_type, 16-byte aligned
 *   q_out   E2M1 pairs [rows, k/2], lower index in the low nibble, 4-byte aligned
 *   sf_out  E8M0 bytes [rows, k/32]
 * 0 <= rows <= 2^31-1, 32 <= k <= 65536, k % 32 == 0, rows * k <= 2^42.  (Pointers may be NULL
 * when rows = 0.)
 * Weights (e, n, k) are e * n rows.
 * Errors: NULL_PTR, SHAPE, DTYPE, ALIGNMENT, UNSUPPORTED, CUDA.
 */
qgmm_status qgmm_per_token_quant_mxfp4(const void *x, int32_t x_type, int64_t rows, int64_t k, uint8_t *q_out,
                                       uint8_t *sf_out, void *cuda_stream);

/*
 * The values MXFP4 codes stand for: out[i][c] = q[i][c] * 2^(sf[i][c/32] - 127), computed
 * in f32 and rounded to out_type (BF16, F16 or F32; BF16 and F32 hold every value
 * that is not below their smallest subnormal or past their largest number exactly).
 * Layouts, limits and errors as qgmm_per_token_quant_mxfp4; out 16-byte aligned.
 */
qgmm_status qgmm_mxfp4_dequant(const uint8_t *q, const uint8_t *sf, int64_t rows, int64_t k, void *out,
                               int32_t out_type, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* QGMM_MM_H */
