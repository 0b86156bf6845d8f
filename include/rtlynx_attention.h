/*
 * rtlynx_attention.h - attention of the queries, keys and values that a
 * block's projections and rotary positions make, and its gradients.
 *
 *   s = scale * q k^T,  p = softmax(s) over the keys that a query sees,  o = p v
 *
 * Query head h reads key head h / (heads_q / heads_k).  A causal query i of a
 * sequence with len_q queries and len_k keys sees keys j <= i + len_k - len_q
 * (the last query sees every key).  A query that sees no key gets zeros, and
 * -inf for its log-sum-exp.
 *
 * Sequences are either rows of a batch, [batch, tokens, heads, head_dim], all
 * of the same length or with fewer keys filled (k_lens: a cache, a padded
 * batch), or lie one after another, [tokens, heads, head_dim], from
 * q_starts[i] to q_starts[i + 1] (k_starts likewise).
 *
 * Scores, the softmax's running maximum and sum and all products accumulate
 * in fp32; the weights p (relative to a running maximum) and, backward, ds
 * enter the matrix cores in the tensors' type; results are rounded once.
 *
 * Conventions are those of rtlynx.h, with these differences: tensors are
 * strided (strides in elements, multiples of 8, the channel stride is 1;
 * heads may be slices of one projection's output) and may pass 2 GiB.
 * Values in the rows of a sequence are finite; what lies outside (behind a
 * filled length, between or behind sequences) is never read into a result.
 */
#ifndef RTLYNX_ATTENTION_H
#define RTLYNX_ATTENTION_H

#include "rtlynx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type (exactly one; the backward pass is bf16 only: fp16 has no room
 * for ds, whose size depends on the loss). */
#define RTL_ATTN_BF16 0x0u
#define RTL_ATTN_FP16 0x1u
#define RTL_ATTN_CAUSAL 0x10u
/* Rows of o that lie in no sequence are set to zero; without this flag they
 * are left as they were. */
#define RTL_ATTN_ZERO_REST 0x20u

#define RTL_ATTN_MAX_HEAD_DIM 128

/* One tensor [sequences, tokens, heads, head_dim]; the batch stride is
 * ignored when sequences are packed. */
typedef struct {
  void* data;
  int64_t batch_stride, token_stride, head_stride; /* elements */
} rtl_attn_tensor;

typedef struct {
  int64_t sequences;          /* batch, or the number of packed sequences      */
  int64_t tokens_q, tokens_k; /* of one sequence, or packed: of all together   */
  int64_t heads_q, heads_k;   /* heads_q a multiple of heads_k                 */
  int64_t head_dim;           /* a multiple of 8, at most RTL_ATTN_MAX_HEAD_DIM */
  const int32_t* q_starts;    /* device, [sequences + 1], or NULL: a batch     */
  const int32_t* k_starts;    /* device, [sequences + 1], or NULL: a batch     */
  const int32_t* k_lens;      /* device, [sequences], a batch only; may be NULL */
  float scale;                /* finite, >= 0                                  */
} rtl_attn_shape;

/*
 * rtl_attention - the forward pass.
 *
 *   q, o     [.., heads_q, head_dim]; k, v [.., heads_k, head_dim].
 *   lse      fp32, may be NULL: log of the sum of exp(s), natural logarithm,
 *            [sequences, heads_q, tokens_q], packed: [heads_q, tokens_q].
 *   workspace  rtl_attention_workspace_bytes(shape, flags) bytes, 16-byte aligned:
 *            where there are fewer queries than the card needs, keys are shared
 *            out over workgroups and the parts joined (0: not for this shape; packed
 *            sequences and causal batches of more than 32 queries never are).
 *
 * q_starts and k_starts go together and must rise; starts and lengths outside
 * the tensors are cut to them.  No tokens, heads or sequences is a no-op.
 * tokens < 2^31, token strides < 2^23, other strides < 2^40, none negative.
 * tokens_q * heads_q * sequences < 2^38.
 */
size_t rtl_attention_workspace_bytes(const rtl_attn_shape* shape, uint32_t flags);

rtl_status rtl_attention(const rtl_attn_tensor* q, const rtl_attn_tensor* k, const rtl_attn_tensor* v,
                         const rtl_attn_tensor* o, float* lse, const rtl_attn_shape* shape,
                         void* workspace, size_t workspace_bytes, uint32_t flags, void* hip_stream);

/*
 * rtl_attention_backward - with p from lse, D = sum over channels of d_o o
 * (for a query that sees up to 128 keys formed as the sum over them of p d_o v^T,
 * without o's rounding):
 *
 *   dv = p^T d_o,  ds = p * (d_o v^T - D),  dq = scale ds k,  dk = scale ds^T q
 *
 * dk and dv sum over the query heads that share a key head.  Nothing is added
 * atomically: the results have the same bits in every run.  Rows of dq, dk and
 * dv that lie in no sequence, or behind a filled length, are set to zero.  No
 * sequences is a no-op, as in the forward pass.
 */
size_t rtl_attention_backward_workspace_bytes(const rtl_attn_shape* shape);

rtl_status rtl_attention_backward(const rtl_attn_tensor* d_o, const rtl_attn_tensor* q, const rtl_attn_tensor* k,
                                  const rtl_attn_tensor* v, const rtl_attn_tensor* o, const float* lse,
                                  const rtl_attn_tensor* dq, const rtl_attn_tensor* dk, const rtl_attn_tensor* dv,
                                  const rtl_attn_shape* shape, void* workspace, size_t workspace_bytes,
                                  uint32_t flags, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RTLYNX_ATTENTION_H */
