/* Low-rank adapters of many requests beside a shared projection: C ABI.
 *
 * The packed NVFP4 matrices are frozen: four-bit weights are neither trained
 * nor exchanged per request. What a request or a fine-tune changes is a
 * low-rank adapter beside the matrix. For token row x_t (bf16 [K]) with
 * adapter a = adapter[t], and the projection's own output row base_t:
 *   y_t = bf16(base_t + s_a B_a (A_a x_t))
 * with A_a bf16 [R][K], B_a bf16 [N][R] and the FP32 scale s_a. Tokens of
 * different adapters share one call in any order. An index outside
 * 0 .. num_adapters - 1 (by custom -1) means no adapter: y_t = bf16(base_t).
 *
 * Every sum is FP32. The low-rank row h_t = s_a A_a x_t enters the second product
 * as the sum of two bf16 values (hi = bf16(h), lo = bf16(h - hi)), 16 significant
 * bits: each term is within 2^-16 of its value, where the output's rounding is
 * 2^-8. The same holds for g_t of the gradients.
 * Values that are not finite: infinite values of h and g, and finite ones above
 * bf16's largest, go through; where x, dy or an adapter itself holds an infinity,
 * an output that it makes infinite by the formula may be NaN (x: its columns of
 * da, dy: its rows of db, an adapter: its outputs). Outputs that the formula
 * makes finite stay as they are.
 *
 * Conventions as in flint_moe.h: device pointers, caller-owned memory, no
 * allocation, asynchronous on `stream`, status codes. Matrices, rows and row
 * strides are 16-byte aligned, index and scale arrays 4-byte aligned,
 * workspaces 256-byte aligned (FLINT_MOE_EALIGN). A workspace needs no
 * initialisation, holds nothing between calls, and must not be shared by calls
 * in flight at the same time. Results do not depend on timing: every sum has a
 * fixed order. A device-side wait that gave up sets FLINT_MOE_DEV_ERR_TIMEOUT in
 * the workspace's status word (flint_moe_read_status), which each call clears.
 */
#ifndef FLINT_LORA_H_
#define FLINT_LORA_H_

#include "flint_gemv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FLINT_LORA_MAX_TOKENS 65536
#define FLINT_LORA_MAX_ADAPTERS 1024
#define FLINT_LORA_MAX_RANK 128

/* A pool of adapters of one projection: plain device pointers, no ownership.
 * in_dim K, out_dim N: multiples of 8, 8 .. 65536. rank R: multiple of 8,
 * 8 .. 128; an adapter of lower rank is stored with zero rows of A and zero
 * columns of B (their gradients are zero too). num_adapters: 1 .. 1024. */
typedef struct flint_lora {
  int32_t in_dim;
  int32_t out_dim;
  int32_t rank;
  int32_t num_adapters;
  const uint16_t* a;   /* bf16 [num_adapters][R][K] */
  const uint16_t* b;   /* bf16 [num_adapters][N][R] */
  const float* scale;  /* float32 [num_adapters] */
} flint_lora;

/* Fills a handle (host struct) after checking shapes (FLINT_MOE_EUNSUPPORTED)
 * and alignment. */
flint_moe_status flint_lora_init(int32_t in_dim, int32_t out_dim, int32_t rank, int32_t num_adapters,
                                 const uint16_t* a, const uint16_t* b, const float* scale, flint_lora* out_lora);

/* Bytes of the workspace of flint_lora_apply for up to max_tokens tokens
 * (1 .. FLINT_LORA_MAX_TOKENS); 0 if the arguments are not supported. */
size_t flint_lora_workspace_bytes(const flint_lora* lora, int32_t max_tokens);

/* y_out[t] = bf16(y_in[t] + s_a B_a (A_a x[t])) for t < T, 0 <= T <=
 * FLINT_LORA_MAX_TOKENS (0 is a no-op). x bf16 [T] rows of K, ldx elements
 * apart; y_in, y_out bf16 [T] rows of N, ldy elements apart (ldx >= K, ldy >=
 * N, multiples of 8 below 2^31). adapter: int32 [T]. y_in NULL means zero. y_out may be
 * y_in (rows without an adapter are then left untouched); any other overlap of
 * y_out with x or y_in is refused (FLINT_MOE_EINVAL). Rows count as overlapping
 * where their extents, first element to last, do: also the columns of one
 * buffer side by side. */
flint_moe_status flint_lora_apply(const flint_lora* lora, const uint16_t* x, int64_t ldx, const int32_t* adapter,
                                  int32_t T, const uint16_t* y_in, uint16_t* y_out, int64_t ldy, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/* Bytes of the workspace of flint_gemv_lora for up to max_batch rows (1 .. 32). */
size_t flint_gemv_lora_workspace_bytes(const flint_lora* lora, int32_t max_batch);

/* flint_gemv with adapters beside the matrix, for 0 <= B <= 32 rows:
 *   y[t] = bf16(G c x[t] + s_a B_a (A_a x[t])),   one rounding.
 * packed, N, K, weight_fmt, x, B, y, dev_status as flint_gemv (without its
 * norm prologue: x is the projection's input as it is); the adapters' out_dim
 * and in_dim must be N and K (FLINT_MOE_EINVAL). x, y contiguous, not
 * overlapping. dev_status NULL: the workspace's status word instead. Two
 * kernels: the adapters' part in FP32 into the workspace, and the GEMV, launched
 * with programmatic dependent launch so that it runs beside it up to its last
 * step, the sum of both. */
flint_moe_status flint_gemv_lora(const void* packed, int32_t N, int32_t K, int32_t weight_fmt, const uint16_t* x,
                                 int32_t B, uint16_t* y, const flint_lora* lora, const int32_t* adapter,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status, cudaStream_t stream);

/* Bytes of the workspace of flint_lora_backward for up to max_tokens tokens. */
size_t flint_lora_backward_workspace_bytes(const flint_lora* lora, int32_t max_tokens);

/* Gradients of flint_lora_apply from dy bf16 [T] rows of N (lddy apart):
 *   g_t = s_a B_a^T dy_t,  h_t = s_a A_a x_t
 *   dx_out[t] = bf16(dx_in[t] + A_a^T g_t)      rows of K, lddx apart
 *   da[a] = bf16(sum_t g_t x_t^T),  db[a] = bf16(sum_t dy_t h_t^T)
 * with the sums over the tokens of adapter a (zero for an adapter without
 * tokens; all num_adapters gradients are written, also for T = 0). dx_in: the
 * projection's own part of the gradient, NULL means zero; dx_out may be dx_in,
 * or NULL (then only da and db are computed; dx_in and lddx are not read). x rows are ldx
 * apart. da, db: bf16, the shapes of a and b. Overlaps are refused
 * (FLINT_MOE_EINVAL): dx_out with x, dy or (otherwise) dx_in; da and db with
 * one another, the adapters, x, dy or dx. */
flint_moe_status flint_lora_backward(const flint_lora* lora, const uint16_t* x, int64_t ldx, const uint16_t* dy,
                                     int64_t lddy, const int32_t* adapter, int32_t T, const uint16_t* dx_in,
                                     uint16_t* dx_out, int64_t lddx, uint16_t* da, uint16_t* db, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FLINT_LORA_H_ */
