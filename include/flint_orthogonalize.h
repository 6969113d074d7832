/* Orthogonalised updates of the matrices that are trained (adapters, routers,
 * dense blocks) by Newton-Schulz steps: C ABI.
 *
 * For each matrix M [rows][cols] of a batch, with X X^T taken over the shorter
 * side (X^T X and X on the left where rows > cols):
 *   X = M / (|M| + eps)                        |M|: Frobenius norm
 *   for each step (a, b, c):  S = X X^T,  X <- a X + (b S + c S S) X
 *   out = bf16(scale X)
 * The steps act on the singular values alone, s <- a s + b s^3 + c s^5: with
 * (3.4445, -4.7750, 2.0315) five times, values of 0.01 to 1 end between 0.7
 * and 1.2, the singular vectors as they were.
 *
 * Numerics: sums are FP32; of the norm's squares a thread adds up to 4096 in
 * FP32, FP64 adds the threads'. X is kept as the sum of two f16 values, to 2^-22
 * of a value or to 2^-35 where that is more (in one kernel's registers, up to
 * 128 rows, as FP32), because what its rounding adds to the weak directions the
 * later steps amplify by up to a^steps. Up to 32 rows the products take X, S and
 * P = b S + c S S as two f16 values too: with the steps above results are the
 * exact ones rounded to bf16 (2^-9.2 of the norm), to 2^-16 of the norm. Above,
 * where a relative error stays relative, X, S and P (from 65 rows on) are single
 * f16 values in the products, to 2^-11 of a value or to 2^-35 (P: 2^-33), and
 * results are within 2^-8 of the exact ones in the norm, 2^-8.5 as a rule;
 * singular values that all pass near 1.2, where a step multiplies a relative
 * error by up to 5, were found to give 0.004. What is kept of an X far below one
 * (|M| far below eps) is a power of two times it, so that all of this holds down
 * to |M| = 2^-100 eps. Singular values must stay below 8 during the steps (S)
 * and b s^2 + c s^4 below 255 (P), as any useful steps' do: beyond, results are
 * not finite.
 *
 * Conventions as in flint_moe.h: device pointers, caller-owned memory, no
 * allocation, asynchronous on `stream`, status codes. Matrices are contiguous,
 * the batch's one behind the other; the first is 16-byte aligned, the workspace
 * 256-byte aligned (FLINT_MOE_EALIGN). Inputs must be finite; a matrix of zeros
 * gives zeros. A workspace needs no initialisation, holds nothing between
 * calls, and must not be shared by calls in flight at the same time. Results do
 * not depend on timing, nor a matrix's on the others of its batch; the batch's
 * size decides how long sums are split, and with it the last bits of larger
 * matrices. A device-side wait that gave up sets
 * FLINT_MOE_DEV_ERR_TIMEOUT in the workspace's status word
 * (flint_moe_read_status), which each call with matrices clears.
 */
#ifndef FLINT_ORTHOGONALIZE_H_
#define FLINT_ORTHOGONALIZE_H_

#include "flint_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FLINT_ORTHOGONALIZE_MAX_STEPS 16
#define FLINT_ORTHOGONALIZE_MAX_SIDE 65536  /* the longer side; the shorter one is at most 16384 */
#define FLINT_ORTHOGONALIZE_MAX_MATRICES 65535

typedef enum { FLINT_ORTHOGONALIZE_F32 = 0, FLINT_ORTHOGONALIZE_BF16 = 1 } flint_orthogonalize_fmt;

/* Bytes of the workspace for batches of n_mat matrices [rows][cols]; 0 if the
 * arguments are not supported. */
size_t flint_orthogonalize_workspace_bytes(int32_t n_mat, int32_t rows, int32_t cols);

/* in: float32 or bf16 (in_fmt) [n_mat][rows][cols], out: bf16, the same shape;
 * out may be in (bf16), any other overlap of the two is refused
 * (FLINT_MOE_EINVAL). coeffs: HOST memory, float [steps][3] = a, b, c of each
 * step, finite, read before the call returns; 1 <= steps <= FLINT_ORTHOGONALIZE_MAX_STEPS. eps > 0 and scale
 * finite. n_mat = 0 is a no-op; rows and cols from 1. The workspace must not
 * overlap in or out (FLINT_MOE_EINVAL). */
flint_moe_status flint_orthogonalize(const void* in, int32_t in_fmt, int32_t n_mat, int32_t rows, int32_t cols,
                                     const float* coeffs, int32_t steps, float eps, float scale, uint16_t* out,
                                     void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FLINT_ORTHOGONALIZE_H_ */
