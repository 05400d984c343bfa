/*
 * gbattn_bwd_strided.h -- the calls of gbattn_bwd.h for an `out` that is not
 * contiguous: a transposed view, as attention computed by other code leaves it
 * ([B, Hq, Sq, D] in memory), or a part of a wider tensor.
 *
 * attn_bwd_padded_strided and attn_bwd_varlen_strided are attn_bwd_padded and
 * attn_bwd_varlen (and, with no lengths, attn_bwd_dense) reading row i, head h
 * of entry b at out + b * out_bstride + i * out_rstride + h * out_hstride, D
 * values side by side.  The same values give the same bits wherever they lie.
 *
 * Strides count elements of out's type, are not negative (zero: the same values
 * again) and are multiples of 16 bytes; one whose dimension has a single index
 * is not used.  Rows of a packed `out` are those of the whole tensor
 * (out_rstride from row to row, Tq of them).  Everything else is contiguous, as
 * in gbattn_bwd.h.  From its first byte to its last, `out` must not meet the
 * gradients or the workspace.
 *
 * Errors beside those of gbattn_bwd.h: GBATTN_ERR_INVALID_ARG (a negative
 * stride), GBATTN_ERR_ALIGNMENT (a stride off 16 bytes),
 * GBATTN_ERR_UNSUPPORTED (a dimension that reaches past 2^58 elements).
 */
#ifndef GBATTN_BWD_STRIDED_H
#define GBATTN_BWD_STRIDED_H

#include "gbattn_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

gbattn_status attn_bwd_padded_strided(const void* q, const void* k, const void* v, const void* out,
                                      gbattn_dtype out_dtype, long long out_bstride, long long out_rstride,
                                      long long out_hstride, const float* lse, const void* dout, const float* dlse,
                                      const int32_t* lens_q, const int32_t* lens_k, int B, int Sq, int Sk, int Hq, int Hkv,
                                      int D, float softmax_scale, int causal, void* dq, void* dk, void* dv,
                                      void* workspace, size_t workspace_bytes, uint32_t* dev_status, void* stream);

gbattn_status attn_bwd_varlen_strided(const void* q, const void* k, const void* v, const void* out,
                                      gbattn_dtype out_dtype, long long out_rstride, long long out_hstride,
                                      const float* lse, const void* dout, const float* dlse, const int32_t* cu_seqlens_q,
                                      const int32_t* cu_seqlens_k, int num_docs, int Tq, int Tk, int max_seqlen_q,
                                      int max_seqlen_k, int Hq, int Hkv, int D, float softmax_scale, int causal, void* dq,
                                      void* dk, void* dv, void* workspace, size_t workspace_bytes, uint32_t* dev_status,
                                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBATTN_BWD_STRIDED_H */
