/* Balance loss of the router, per-expert counts, and the router's gradient:
 * C ABI, for training the bf16 router of a layer.
 *
 * The router of flint_moe.h scores token t with s_te = sigmoid(z_te) and picks
 * k experts. For n_seq sequences of tokens, sequence b with T_b counted tokens
 * and c_be picks of expert e among them:
 *   p_te = s_te / sum_e' s_te'                        (the scores' shares)
 *   f_be = E c_be / (k T_b)                           (1 for an even load)
 *   loss = alpha / n_seq  sum_b 1/T_b  sum_{t in b} sum_e f_be p_te
 * f is a count and carries no gradient. A sequence without counted tokens adds
 * nothing. Shares are defined for every row of finite logits as the softmax of
 * log sigmoid(z), also where every s underflows FP32; a row whose logits are all
 * -infinity has shares of zero.
 *
 * Sequences: seq_start int32 [n_seq + 1] (device), not decreasing, within
 * 0 .. T; sequence b is the tokens seq_start[b] .. seq_start[b + 1] - 1 (none
 * is allowed). Tokens before the first or behind the last sequence are in no
 * sequence. seq_start NULL (n_seq = 1) means one sequence of all T tokens.
 * Picks: idx int32 [T][k] as the router returns them. A token whose first pick
 * is negative is padding: it is not counted. Another pick outside 0 .. E - 1
 * is dropped.
 * cfg gives E, k, renormalize and routed_scale (flint_moe_check_config).
 *
 * Conventions as in flint_moe.h: device pointers, caller-owned memory, no
 * allocation, asynchronous on `stream`, status codes; pointers 4-byte aligned
 * (logits and gradients of E % 4 == 0 experts, and workspaces, 16-byte), else
 * FLINT_MOE_EALIGN. Counts are whole numbers and sums have a fixed order: the
 * same inputs give the same bits.
 */
#ifndef FLINT_MOE_BALANCE_H_
#define FLINT_MOE_BALANCE_H_

#include "flint_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FLINT_MOE_BALANCE_MAX_TOKENS (1 << 20)
#define FLINT_MOE_BALANCE_MAX_SEQS 65536

/* Bytes of the workspace of flint_moe_balance for up to max_tokens tokens in
 * up to max_seqs sequences; 0 if the arguments are not supported. It needs no
 * initialisation, holds nothing between calls, and must not be shared by calls
 * in flight at the same time. */
size_t flint_moe_balance_workspace_bytes(const flint_moe_config* cfg, int32_t max_tokens, int32_t max_seqs);

/* logits float32 [T][E], idx int32 [T][k], 0 <= T <=
 * FLINT_MOE_BALANCE_MAX_TOKENS, 1 <= n_seq <= FLINT_MOE_BALANCE_MAX_SEQS.
 * Writes loss float32 [1], counts int32 [E] (over all sequences: what an
 * update of the selection bias goes by), seq_counts int32 [n_seq][E] (c_be)
 * and seq_tokens int32 [n_seq] (T_b), which the backward call takes. T = 0
 * writes zeros. Outputs and workspace that overlap one another or an input are
 * refused (FLINT_MOE_EINVAL), counts and seq_counts of one sequence too. */
flint_moe_status flint_moe_balance(const flint_moe_config* cfg, const float* logits, const int32_t* idx, int32_t T,
                                   const int32_t* seq_start, int32_t n_seq, float alpha, float* loss,
                                   int32_t* counts, int32_t* seq_counts, int32_t* seq_tokens, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/* The logits' gradient, of the loss and of the routing weights together:
 *   dz_tj  = dloss alpha / (n_seq T_b) p_tj (f_bj - sum_e f_be p_te) (1 - s_tj)
 *   dz_tj += routed_scale w_tj (dw_tj - sum_i dw_ti w_ti) (1 - s_tj)  at the
 *            token's picks, w_tj = s_tj / sum_picks s (renormalize), or
 *            routed_scale s_tj dw_tj (1 - s_tj)
 * dloss: float32 [1] on the device, NULL means 1. dw: float32 [T][k], the
 * gradient of the routing weights, NULL for none. seq_counts and seq_tokens as
 * flint_moe_balance wrote them. dlogits float32 [T][E] (refused where it
 * overlaps an input: FLINT_MOE_EINVAL): padding tokens get zeros; rows of tokens in no sequence are left as
 * they were. An expert picked twice by a token gets both gradients. */
flint_moe_status flint_moe_balance_backward(const flint_moe_config* cfg, const float* logits, const int32_t* idx,
                                            int32_t T, const int32_t* seq_start, int32_t n_seq, float alpha,
                                            const int32_t* seq_counts, const int32_t* seq_tokens,
                                            const float* dloss, const float* dw, float* dlogits,
                                            cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FLINT_MOE_BALANCE_H_ */
