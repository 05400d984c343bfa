/*
 * gbattn_bwd.h -- C ABI of the attention gradients (sm_103a), beside gbattn.h.
 *
 * For the forward calls of gbattn.h (attn_fwd_dense, attn_fwd_padded,
 * attn_fwd_varlen) with
 *     s_ij = softmax_scale * q_i . k_j   over the visible pairs,
 * and out, lse as the forward call returned them, these calls compute
 *     p_ij    = exp(s_ij - lse_i)
 *     delta_i = dout_i . out_i - dlse_i
 *     ds_ij   = p_ij (dout_i . v_j - delta_i)
 *     dv_j = sum_i p_ij dout_i
 *     dk_j = softmax_scale sum_i ds_ij q_i
 *     dq_i = softmax_scale sum_j ds_ij k_j
 * where dout is the gradient of out and dlse that of lse (NULL: lse is not
 * used further on).  dk and dv of a KV head are the sums over the query heads
 * that share it.  A row that sees no key (lse = -inf) gives nothing and gets
 * dq = 0, whatever its rows of dout and out hold.
 *
 * Conventions are those of gbattn.h (ownership, streams, errors, dev_status,
 * head sizes, masks), and:
 *  - q, k, v, dout and the gradients are bf16; out is bf16 or fp32
 *    (out_dtype), lse and dlse fp32 in the forward call's layout.  All are
 *    contiguous (an out that is not: gbattn_bwd_strided.h).
 *  - Sums are kept in fp32 and rounded once; the probabilities and ds are
 *    rounded to bf16 as operands of the second products.
 *  - Documents and batch entries are apart: nothing that one of them holds, NaN
 *    and infinity included, reaches another's gradients.  Within a document a
 *    value that is not finite may reach rows that do not see it: p and ds of a
 *    hidden pair are 0, and 0 times it is NaN, as in the forward product p v.
 *    (Rows that see no key, and rows past an entry's lengths, may hold anything.)
 *  - The same inputs give the same bits: each gradient row is summed in one
 *    order, without atomics.
 *  - dq, dk and dv are written whole but for the rows that belong to no
 *    document.  They and the workspace must not overlap the inputs or each
 *    other (GBATTN_ERR_INVALID_ARG).
 *  - workspace: device buffer of at least attn_bwd_workspace_size bytes,
 *    256-byte aligned, needing no initialisation; calls that can overlap
 *    (other streams, graphs replayed together) need one each.
 */
#ifndef GBATTN_BWD_H
#define GBATTN_BWD_H

#include "gbattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * attn_bwd_workspace_size -- bytes of workspace for num_docs documents (or
 * batch entries) of Tq query rows in all (B * Sq of a batch).  Pure host
 * arithmetic; 0 for invalid sizes.
 */
size_t attn_bwd_workspace_size(int num_docs, int Tq, int Hq);

/*
 * attn_bwd_dense -- gradients of attn_fwd_dense.
 *   q, out, dout, dq   device [B, Sq, Hq, D]
 *   k, v, dk, dv       device [B, Sk, Hkv, D]
 *   lse, dlse          device fp32 [B, Hq, Sq]; dlse may be NULL
 * B, Sq or Sk equal to 0 is allowed; the side without rows may be NULL.
 * Errors: GBATTN_ERR_INVALID_ARG, GBATTN_ERR_UNSUPPORTED (head size,
 * out_dtype, B > 65535, rows or tiles past 2^31 - 1), GBATTN_ERR_ALIGNMENT,
 * GBATTN_ERR_WORKSPACE, GBATTN_ERR_DEVICE / GBATTN_ERR_CUDA.
 */
gbattn_status attn_bwd_dense(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                             const float* lse, const void* dout, const float* dlse, int B, int Sq, int Sk, int Hq,
                             int Hkv, int D, float softmax_scale, int causal, void* dq, void* dk, void* dv,
                             void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream);

/*
 * attn_bwd_padded -- gradients of attn_fwd_padded: entry b uses its first
 * lens_q[b] query rows and lens_k[b] keys (device int32 [B], or NULL for all).
 * The rows past them get zeros in dq, dk and dv, and never reach a result,
 * whatever q, k, v, out, dout, lse and dlse hold there.  A length outside
 * [0, S] sets GBATTN_DEV_BAD_SEQLEN and is clamped.
 */
gbattn_status attn_bwd_padded(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                              const float* lse, const void* dout, const float* dlse, const int32_t* lens_q,
                              const int32_t* lens_k, int B, int Sq, int Sk, int Hq, int Hkv, int D, float softmax_scale,
                              int causal, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                              uint32_t* dev_status, void* stream);

/*
 * attn_bwd_varlen -- gradients of attn_fwd_varlen: packed documents.
 *   q, out, dout, dq   device [Tq, Hq, D]
 *   k, v, dk, dv       device [Tk, Hkv, D]
 *   lse, dlse          device fp32 [Hq, Tq]; dlse may be NULL
 *   cu_seqlens_q/k, num_docs, max_seqlen_q/k  as for attn_fwd_varlen
 * Rows that belong to no document are neither read into a result nor written.
 * A document whose boundaries decrease, run past Tq / Tk or exceed
 * max_seqlen sets GBATTN_DEV_BAD_SEQLEN; its rows are left unwritten.  (Where
 * boundaries decrease, two other documents can claim the same rows; those
 * two's results are undefined.)  A document with keys and no queries gets
 * dk = dv = 0.
 */
gbattn_status attn_bwd_varlen(const void* q, const void* k, const void* v, const void* out, gbattn_dtype out_dtype,
                              const float* lse, const void* dout, const float* dlse, const int32_t* cu_seqlens_q,
                              const int32_t* cu_seqlens_k, int num_docs, int Tq, int Tk, int max_seqlen_q,
                              int max_seqlen_k, int Hq, int Hkv, int D, float softmax_scale, int causal, void* dq,
                              void* dk, void* dv, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBATTN_BWD_H */
