/* Dense gated feed-forward block on BF16 weights, for many tokens, with its
 * gradients: C ABI.
 *
 * "Day-0 Support for Flint on vLLM", section "Model architecture": the first
 * layers of the stack are dense gated blocks instead of experts. For token row
 * x (bf16 [H]) and the matrices Wg, Wu [I][H], Wd [H][I]:
 *   g = Wg x,  u = Wu x                    FP32 accumulation
 *   h = bf16(silu(g) * u)                  BF16 rounding point, as in flint_moe.h
 *   y = bf16(Wd h)                         FP32 accumulation
 * Up to 32 tokens on packed (NVFP4 or BF16) matrices, a decode step has
 * flint_gemv_glu and flint_gemv (flint_gemv.h).
 *
 * Conventions as in flint_moe.h: device pointers, caller-owned memory, no
 * allocation, asynchronous on `stream`, status codes. Matrices, rows and row
 * strides are 16-byte aligned, workspaces 256-byte aligned (FLINT_MOE_EALIGN).
 * Inputs must be finite. A workspace needs no initialisation, holds nothing
 * between calls, and must not be shared by calls in flight at the same time.
 * Results do not depend on timing: every sum has a fixed order. A device-side
 * wait that gave up sets FLINT_MOE_DEV_ERR_TIMEOUT in the workspace's status
 * word (flint_moe_read_status), which each call clears that has anything to
 * compute (tokens, and an output).
 */
#ifndef FLINT_FFN_H_
#define FLINT_FFN_H_

#include "flint_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FLINT_FFN_MAX_TOKENS 65536

/* A block's weights: plain device pointers, no ownership. hidden H and inter I:
 * multiples of 8, 8 .. 65536. */
typedef struct flint_ffn {
  int32_t hidden;
  int32_t inter;
  const uint16_t* gate; /* bf16 [I][H] */
  const uint16_t* up;   /* bf16 [I][H] */
  const uint16_t* down; /* bf16 [H][I] */
} flint_ffn;

/* Fills a handle (host struct) after checking shapes (FLINT_MOE_EUNSUPPORTED)
 * and alignment. */
flint_moe_status flint_ffn_init(int32_t hidden, int32_t inter, const uint16_t* gate, const uint16_t* up,
                                const uint16_t* down, flint_ffn* out_ffn);

/* Bytes of the workspace of flint_ffn_forward for up to max_tokens tokens
 * (1 .. FLINT_FFN_MAX_TOKENS); 0 if the arguments are not supported. */
size_t flint_ffn_workspace_bytes(const flint_ffn* ffn, int32_t max_tokens);

/* y[t] = block(x[t]) for t < T, 0 <= T <= FLINT_FFN_MAX_TOKENS (0 is a no-op).
 * x, y: bf16 [T] rows of H, ldx and ldy elements apart (>= H, multiples of 8
 * below 2^31). gate_out, up_out: bf16 [T][I], receive bf16(g) and bf16(u),
 * which the gradients take; both or neither (FLINT_MOE_EINVAL). y, gate_out,
 * up_out and the workspace must not overlap one another, x or the weights
 * (FLINT_MOE_EINVAL; rows count from the first element to the last). */
flint_moe_status flint_ffn_forward(const flint_ffn* ffn, const uint16_t* x, int64_t ldx, int32_t T, uint16_t* y,
                                   int64_t ldy, uint16_t* gate_out, uint16_t* up_out, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/* Bytes of the workspace of flint_ffn_backward for up to max_tokens tokens. */
size_t flint_ffn_backward_workspace_bytes(const flint_ffn* ffn, int32_t max_tokens);

/* Gradients from dy (bf16 [T] rows of H, lddy apart) and the products that the
 * forward call kept (gate_act, up_act: bf16 [T][I]):
 *   dh = Wd^T dy,  s = sigmoid(g)                        FP32
 *   dg = bf16(dh u s (1 + g (1 - s))),  du = bf16(dh g s),  h = bf16(g s u)
 *   dx = bf16(Wg^T dg + Wu^T du)                         rows of H, lddx apart
 *   dgate = bf16(sum_t dg_t x_t^T), dup = bf16(sum_t du_t x_t^T),
 *   ddown = bf16(sum_t dy_t h_t^T)                       shapes of the weights
 * dx NULL skips the gradient of x; dgate, dup and ddown all NULL skip those of
 * the weights (frozen), one of them alone is refused (FLINT_MOE_EINVAL); what is
 * left has the same bits. T = 0
 * writes zeros to the weights' gradients. Outputs and workspace must not overlap
 * one another or an input (FLINT_MOE_EINVAL). */
flint_moe_status flint_ffn_backward(const flint_ffn* ffn, const uint16_t* x, int64_t ldx, const uint16_t* gate_act,
                                    const uint16_t* up_act, const uint16_t* dy, int64_t lddy, int32_t T, uint16_t* dx,
                                    int64_t lddx, uint16_t* dgate, uint16_t* dup, uint16_t* ddown, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FLINT_FFN_H_ */
