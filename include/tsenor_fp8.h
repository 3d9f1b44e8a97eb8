/*
 * tsenor_fp8.h -- 8-bit operators of 2:4-masked weights (part of libtsenor.so).
 *
 * With a transposable 2:4 mask (tsenor.h, N = 2, M = 4) both W and W^T are 2:4
 * along their rows.  These entry points hold them as 8-bit floats with a scale
 * for each block of 128 and multiply with them: quantise the activations or
 * gradients, compress the masked weight, the product (forward and data
 * gradient), the masked weight gradient, and a mixture-of-experts layer for a
 * few tokens.
 *
 * Numbers.  A value is e4m3 (OCP: 4 exponent bits, 3 fraction bits, largest
 * 448, no infinity, NaN 0x7F/0xFF).  The scale of a block is a power of two
 * 2^s, held as the byte s + 127 (e8m0): s is the least integer >= -127 with
 * amax <= 448 * 2^s, amax being the largest finite magnitude of the block, and
 * 0 for a block without one (all zeros).  An element x becomes the e4m3 number
 * nearest to x * 2^-s, ties to even; infinities and NaN become NaN.
 *
 * Operands.  kpad = k rounded up to a multiple of 128; the entries behind k
 * are zeros.  All bases are 16-byte aligned.
 *   dense [rows][k]: values uint8 [rows][kpad]; scales uint8 [kpad/128][rows],
 *            one for each block of 1 x 128 along a row, block index first.
 *   2:4 [rows][k]: values uint8 [rows][kpad/2], the two kept entries of every
 *            aligned group of four along the row in ascending position, unused
 *            slots 0; meta uint32 [rows][kpad/32] as in tsenor_compress24; and
 *            scales uint8 [ceil(rows/128)][kpad/128], one for each 128 x 128 block.
 *   A batch of 2:4 operands is stacked without gaps, operand after operand.
 *
 * Conventions are those of tsenor.h: device pointers, no reference kept,
 * asynchronous on `stream`, argument errors found on the host before any HIP
 * call.  No entry point allocates, keeps or shares any memory between calls,
 * records an event, or waits: calls may overlap on several streams and may be
 * captured into graphs.  Outputs must not overlap inputs.  An operand of more
 * than 2^40 entries, or more threads than one launch counts (2^32; 2^35 entries
 * of X in tsenor_quant_fp8 along the rows), is _SHAPE.  Results are
 * deterministic.  A NaN in one row of X touches that row of the result only.
 */
#ifndef TSENOR_FP8_H
#define TSENOR_FP8_H

#include <stddef.h>
#include <stdint.h>

#include "tsenor.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more element type, for the operands of tsenor_spmm24_fp8. */
enum { TSENOR_E4M3 = 2 };

/* X (dtype f32 or bf16, [rows][ldx], ldx >= cols) to 8 bits, read once.
 *   values, scales      the dense operand X  [rows][cols], or both NULL;
 *   values_t, scales_t  the dense operand X^T [cols][rows], or both NULL.
 * rows == 0 is a no-op.  Errors: _NULL (X, or neither operand asked for, or
 * half of one), _DTYPE, _SHAPE (rows < 0, cols <= 0, ldx < cols, alignment). */
int tsenor_quant_fp8(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                     uint8_t* values, uint8_t* scales, uint8_t* values_t, uint8_t* scales_t,
                     void* stream);

/* `batch` weights (f32 or bf16; matrix b at W + b * stride elements, [rows][ld])
 * under their 2:4 masks ([batch][rows][ceil(cols/32)] words) to 2:4 8-bit
 * operands, read once.  amax runs over the entries that the mask keeps.
 *   values, meta, scales        the operand W   [rows][cols], or all NULL;
 *   values_t, meta_t, scales_t  the operand W^T [cols][rows], or all NULL:
 *            the same 8-bit numbers, since a block is square.
 * Groups with more than two kept entries keep their first two and are counted
 * into *bad (of W) and *bad_t (of W^T), device ints, added to; NULL = no count.
 * The mask may be any; for a transposable 2:4 mask both counts stay 0.
 * Errors: _NULL, _DTYPE, _SHAPE (batch < 0, rows or cols <= 0 or not multiples
 * of 4, ld < cols, stride < rows * ld, alignment).  batch == 0 is a no-op.    */
int tsenor_compress24_fp8(const void* W, int dtype, int64_t batch, int64_t stride, int64_t rows,
                          int64_t cols, int64_t ld, const uint32_t* mask, uint8_t* values,
                          uint32_t* meta, uint8_t* scales, uint8_t* values_t, uint32_t* meta_t,
                          uint8_t* scales_t, int* bad, int* bad_t, void* stream);

/* Y = X A^T with A [m][k] a 2:4 operand.  Per block of 128 along k the kept
 * products are summed on the sparse matrix cores, the sum is scaled by
 * 2^(sx + sa) and added in fp32.  (A factor above 2^127 counts as 2^127; a block
 * whose factor is below 2^-149, or 2^100 below another's in the same row of Y,
 * may be lost.)  The 8-bit matrix cores add eight products at a time
 * and drop what lies more than about 2^-12 below the largest of the eight; for
 * entries of similar size a sum is good to about 2^-15.  Entries that the mask
 * removed are not multiplied, but the unused slots of a group with fewer than two
 * kept entries are: zeros times the entries of X at the positions 0 and 1 of an empty
 * group, at 3 beside one kept entry (2 if that is itself at 3).  A NaN there makes
 * the result NaN (in tsenor_moe24_fp8 an infinite entry of the hidden vector too).
 *   X      xtype TSENOR_E4M3: values [n][ldx] of a dense operand (ldx >= kpad, a
 *          multiple of 16) and its scales [kpad/128][n];
 *          xtype TSENOR_BF16: [n][ldx] with n <= 16, quantised on the way as
 *          tsenor_quant_fp8 does, xscales NULL.
 *   Y      ytype f32 or bf16, [n][ldy], ldy >= m; columns behind m are not written.
 * n == 0 is a no-op.  Errors: _NULL, _DTYPE, _SHAPE (n < 0, n > 16 for bf16 X,
 * m, k <= 0, leading dimensions, alignment).                                 */
int tsenor_spmm24_fp8(const void* X, int xtype, const uint8_t* xscales, int64_t n, int64_t ldx,
                      const uint8_t* values, const uint32_t* meta, const uint8_t* scales,
                      int64_t m, int64_t k, void* Y, int ytype, int64_t ldy, void* stream);

/* C = A B^T for dense operands A [p][k] and B [q][k], on the scaled matrix
 * cores with fp32 sums; with a mask ([p][ceil(q/32)] words, layout of
 * tsenor_mask) the entries that it removes are written as 0.  With A and B
 * quantised along the tokens (values_t of dY and X) this is the masked weight
 * gradient dY^T X.  k == 0 (no tokens) gives zeros.
 *   C      ctype f32 or bf16, [p][ldc], ldc >= q.
 * Errors: _NULL, _DTYPE, _SHAPE (p, q <= 0, k < 0, ldc < q, alignment).        */
int tsenor_gemm_fp8(const uint8_t* A, const uint8_t* a_scales, int64_t p, const uint8_t* B,
                    const uint8_t* b_scales, int64_t q, int64_t k, const uint32_t* mask, void* C,
                    int ctype, int64_t ldc, void* stream);

/* A mixture-of-experts layer for a few tokens, weights 2:4 in 8 bits,
 * activations bf16, sums fp32:
 *   logits = x R^T (products exact, sums in fp64); each token takes the `topk`
 *   largest (ties to the lowest index, NaN below every number) with weights
 *   softmax over those; y = sum_e w_e Down_e (silu(Gate_e x) * (Up_e x)).  The
 *   hidden vector is held as the sum of two bf16 numbers (2^-16 of each entry
 *   at most is lost), y is rounded once.  Weights are multiplied as bf16 numbers:
 *   they lose bits below 2^-133, and a magnitude of 2^128 or more is infinite.
 *   X [n][ldx] bf16, 0 <= n <= 64;  router [experts][ldr] bf16;
 *   gate, up  batches of `experts` 2:4 operands [f][d];  down  [d][f];
 *   workspace device memory of at least tsenor_moe24_fp8_workspace(...) bytes,
 *            16-byte aligned, not shared by calls that may overlap;
 *   Y [n][ldy] bf16;  ids int32 [n][topk] (largest logit first) and weights
 *            fp32 [n][topk]: the routing, or NULL.
 * Errors: _NULL, _PARAM (topk < 1, topk > experts, topk > 16, experts > 512), _SHAPE
 * (n < 0 or > 64, d or f <= 0 or > 2^20, leading dimensions, alignment, workspace_bytes). */
size_t tsenor_moe24_fp8_workspace(int64_t n, int64_t d, int64_t f, int64_t experts, int topk);
int tsenor_moe24_fp8(const uint16_t* X, int64_t n, int64_t ldx, int64_t d, const uint16_t* router,
                     int64_t ldr, int64_t experts, int topk, const uint8_t* gate_values,
                     const uint32_t* gate_meta, const uint8_t* gate_scales,
                     const uint8_t* up_values, const uint32_t* up_meta, const uint8_t* up_scales,
                     const uint8_t* down_values, const uint32_t* down_meta,
                     const uint8_t* down_scales, int64_t f, void* workspace,
                     size_t workspace_bytes, uint16_t* Y, int64_t ldy, int* ids, float* weights,
                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TSENOR_FP8_H */
