/*
 * tsenor_ops.h -- dense operators of masked models (part of libtsenor.so).
 *
 * A mask with M = 8, 16 or 32 (tsenor.h) has no matrix core of its own: its
 * layers run as dense products of masked weights.  These entry points carry
 * such a layer through a training step and through serving: products grouped
 * by expert (forward, data gradient, masked weight gradient), products of
 * 8-bit integers with a scale for each token and channel, and the clipping of
 * a model's gradients, masked ones by what their masks keep.
 *
 * Groups.  The rows of a grouped operand are sorted by expert.  `ends` (device,
 * int32 [experts]) holds for each expert the row behind its last one: expert e
 * owns rows ends[e-1] .. ends[e]-1 (from 0 for e = 0), which may be none.  Rows
 * from ends[experts-1] on belong to no expert; their results are zeros.  The
 * host never reads `ends`: entries below 0 count as 0, above `rows` as `rows`,
 * and one below an earlier one as that one.
 *
 * 8-bit integer operands [rows][k]: values int8 [rows][kpad], kpad = k rounded up
 * to a multiple of 128, the entries behind k zeros; scales fp32 [rows].  A row
 * stands for value * scale.  Values lie in -127 .. 127.  A batch of operands is
 * stacked without gaps, and so are its scales.  k <= 2^17, so that sums of
 * products fit 32 bits.
 *
 * Conventions are those of tsenor_fp8.h: device pointers, no reference kept,
 * asynchronous on `stream`, argument errors found on the host before any HIP
 * call, nothing allocated or kept between calls, calls may overlap and may be
 * captured into graphs, outputs must not overlap inputs (but for the gradients
 * of tsenor_clip_grads).  Operands of more than 2^40 entries and grids past one
 * launch are _SHAPE.  Matrices are row-major with a leading dimension in
 * elements; any alignment of their type is allowed (16-byte aligned rows are
 * faster).  Results are deterministic.  A NaN in one row touches the results
 * that the row enters only.
 */
#ifndef TSENOR_OPS_H
#define TSENOR_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "tsenor.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more element type, for the operands of tsenor_gemm_int8. */
enum { TSENOR_INT8 = 3 };

/* Y[r] = X[r] W_e^T (transpose 0, W_e [m][ldw], ldw >= k) or Y[r] = X[r] W_e
 * (transpose 1, W_e [k][ldw], ldw >= m) for the expert e that owns row r; sums
 * in fp32, rounded once.
 *   X      bf16 [rows][ldx], ldx >= k;  W  bf16, expert e at W + e * stride;
 *   Y      ytype f32 or bf16, [rows][ldy], ldy >= m.
 * rows == 0 is a no-op.  Errors: _NULL, _DTYPE, _PARAM (transpose not 0 or 1,
 * experts < 1 or > 1024), _SHAPE (rows < 0 or >= 2^30, m, k <= 0, k >= 2^30,
 * leading dimensions, stride, alignment).                                     */
int tsenor_grouped_mm(const uint16_t* X, int64_t rows, int64_t ldx, const uint16_t* W,
                      int transpose, int64_t experts, int64_t stride, int64_t ldw, int64_t m,
                      int64_t k, const int* ends, void* Y, int ytype, int64_t ldy, void* stream);

/* C_e = dY_e^T X_e for every expert: its weight gradient over the rows that it
 * owns (none: zeros), sums in fp32, rounded once.
 *   dY     bf16 [rows][lddy], lddy >= m;  X  bf16 [rows][ldx], ldx >= k;
 *   mask   [experts][m][ceil(k/32)] words (layout of tsenor_mask): entries that
 *          it removes are written as 0; or NULL;
 *   C      ctype f32 or bf16, expert e at C + e * stride, [m][ldc], ldc >= k.
 * Errors: _NULL, _DTYPE, _PARAM (experts), _SHAPE (as above).                 */
int tsenor_grouped_wgrad(const uint16_t* dY, int64_t lddy, const uint16_t* X, int64_t ldx,
                         int64_t rows, int64_t experts, int64_t m, int64_t k, const int* ends,
                         const uint32_t* mask, void* C, int ctype, int64_t stride, int64_t ldc,
                         void* stream);

/* `batch` matrices (f32 or bf16; matrix b at X + b * stride elements, [rows][ldx])
 * to stacked 8-bit integer operands.  For a row with largest magnitude amax:
 * scale = amax / 127 in fp32, values the integers nearest to x * 127 / amax
 * (taken exactly), ties to even.  A row of zeros has scale 0; a row with an
 * infinity or a NaN has values 0 and scale NaN, so that its products are NaN.
 * Errors: _NULL, _DTYPE, _SHAPE (batch, rows < 0, cols <= 0 or > 2^17, ldx < cols,
 * stride < rows * ldx, alignment).  No rows are a no-op.                        */
int tsenor_quant_int8(const void* X, int dtype, int64_t batch, int64_t stride, int64_t rows,
                      int64_t cols, int64_t ldx, int8_t* values, float* scales, void* stream);

/* Y[r][j] = xs[r] as_e[j] sum_i x[r][i] a_e[j][i]: 8-bit integer operands X
 * [rows][k] and A (a batch of `experts` operands [m][k]), sums exact in 32 bits;
 * Y[r][j] = round(float(sum) * xs[r] * as[j]), left to right in fp32.
 *   X      xtype TSENOR_INT8: values of an operand, and its scales;
 *          xtype TSENOR_BF16: [rows][ldx] with rows <= 16, rows * kpad <= 2^15 and ends
 *          NULL, quantised on the way as tsenor_quant_int8 does, xscales NULL;
 *   ldx    kpad for TSENOR_INT8, >= k for TSENOR_BF16;
 *   ends   as above, or NULL: one weight (experts 1) for all rows;
 *   Y      ytype f32 or bf16, [rows][ldy], ldy >= m.
 * rows == 0 is a no-op.  Errors: _NULL, _DTYPE, _PARAM (experts < 1 or > 1024,
 * experts != 1 without ends), _SHAPE (rows < 0 or >= 2^30, m <= 0 or >= 2^30,
 * k <= 0 or > 2^17, leading dimensions, more rows than allowed for bf16, alignment: values 16 bytes). */
int tsenor_gemm_int8(const void* X, int xtype, const float* xscales, int64_t rows, int64_t ldx,
                     const int8_t* A, const float* ascales, int64_t experts, int64_t m, int64_t k,
                     const int* ends, void* Y, int ytype, int64_t ldy, void* stream);

/* One gradient of a list: [rows][ld] of dtype (f32 or bf16); out (same type,
 * [rows][ldo], for tsenor_clip_grads) may be grad itself (ldo == ld) and must not overlap
 * it otherwise, nor anything else of the list; mask words [rows][ceil(cols/32)] or NULL (all kept). */
typedef struct {
    const void* grad;
    void* out;
    const uint32_t* mask;
    int dtype;
    int64_t rows, cols, ld, ldo;
} tsenor_grad;

/* The norm of a list of gradients, sqrt(sum of squares of the kept entries), in
 * 64 bits, written as fp32 to *norm (device).  tsenor_clip_grads also writes
 *   out = kept entry * f, removed entry 0;   f = 1 if norm <= max_norm, else
 * fp32(max_norm / norm), the product rounded once to the gradient's type.
 * An infinite norm gives f = 0 and NaN at the infinite entries, a NaN norm gives NaN everywhere
 * (at kept entries).
 *   grads  HOST array of `count` >= 0 entries, not needed after the call;
 *   max_norm  >= 0, may be infinite (nothing is scaled);
 *   workspace device memory of at least tsenor_grads_workspace(count) bytes, 8-byte
 *          aligned, not shared by calls that may overlap.
 * Errors: _NULL (norm, workspace, grads, an entry's grad or out), _DTYPE, _PARAM
 * (count < 0, max_norm), _SHAPE (rows, cols < 0, ld, ldo < cols, in place with
 * ldo != ld, alignment of the type, workspace_bytes).                              */
size_t tsenor_grads_workspace(int count);
int tsenor_grad_norm(const tsenor_grad* grads, int count, void* workspace, size_t workspace_bytes,
                     float* norm, void* stream);
int tsenor_clip_grads(const tsenor_grad* grads, int count, float max_norm, void* workspace,
                      size_t workspace_bytes, float* norm, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSENOR_OPS_H */
