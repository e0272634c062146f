/*
 * fadam_seq.h - C ABI of the sequence operators that stand next to the
 * training operators of fadam_ops.h: what a block's rows come from and how
 * they see one another.
 *
 *   fadam_embed_*       the token embedding, and the gradient of its weight
 *   fadam_attention_*   attention over packed documents, forward and backward
 *
 * Conventions, workspaces, statuses and messages are those of fadam_ops.h
 * (fadam_ops_last_error, fadam_ops_status).  No output overlaps an input, another
 * output or the workspace: a launch may still read one where another part of it
 * has written the other.
 */
#ifndef FADAM_SEQ_H_
#define FADAM_SEQ_H_

#include <stddef.h>
#include <stdint.h>

#include "fadam_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- token embedding ----------------------------------------------------------- */

#define FADAM_EMBED_PADDING 1u    /* padding_index counts */
#define FADAM_EMBED_ACCUMULATE 2u /* the gradient is added to out, else written */

/* out_t = scale * weight_tokens[t] in fp32, rounded to out_dtype; zero where tokens[t] ==
 * padding_index, NaN where a token lies outside [0, vocab) (the loss turns into
 * NaN, and the shard's screen or norm into a skipped step).
 *   tokens [rows]           int64
 *   weight [vocab, width]   of weight_dtype (any)
 *   out [rows, width]       of out_dtype: weight_dtype or fp32 */
typedef struct {
  const int64_t* tokens;
  const void* weight;
  void* out;
  int64_t rows, width, vocab;
  int64_t weight_stride, out_stride;
  int64_t padding_index;
  float scale; /* finite */
  int32_t weight_dtype;
  int32_t out_dtype;
  uint32_t flags;
} fadam_embed;

/* Errors: FADAM_EINVAL, FADAM_EDTYPE, FADAM_EALIGN, FADAM_ELIMIT (a size
 * beyond 2^30), FADAM_ECUDA. */
fadam_status fadam_embed_forward(const fadam_embed* desc, fadam_stream stream);

/* out_v (+)= scale * sum of grad_t over the t with tokens[t] == v.  Without
 * FADAM_EMBED_ACCUMULATE rows of no token are zero; with it they are not
 * touched.  Tokens that are padding_index or outside [0, vocab) are left out.
 * The sum is fp32, over a token's rows in their order (by groups of up to 64
 * rows, then over the groups), and rounded once.
 *   grad [rows, width]      of grad_dtype (any)
 *   out [vocab, width]      of out_dtype: grad_dtype, fp32, or any where
 *                           grad_dtype is fp32
 * rows and vocab up to 2^30. */
typedef struct {
  const int64_t* tokens;
  const void* grad;
  void* out;
  int64_t rows, width, vocab;
  int64_t grad_stride, out_stride;
  int64_t padding_index;
  float scale; /* finite */
  int32_t grad_dtype;
  int32_t out_dtype;
  uint32_t flags;
} fadam_embed_grad;

fadam_status fadam_embed_grad_workspace(const fadam_embed_grad* desc, size_t* bytes);
fadam_status fadam_embed_grad_run(const fadam_embed_grad* desc, void* workspace, size_t bytes,
                                  fadam_stream stream);

/* ---- attention ------------------------------------------------------------------- */

#define FADAM_ATTENTION_CAUSAL 1u

/* Largest width of a head; widths are multiples of 8. */
#define FADAM_ATTENTION_MAX_WIDTH 128

/* Tokens lie one after another, those of documents (or sequences) together.
 * For a query i and a key j of one document, of query head h:
 *   s_ij = scale q_i . k_j
 *   s_ij = softcap tanh(s_ij / softcap)          where softcap > 0
 *   s_ij = s_ij - slopes[h] |i - j|              where slopes is not NULL
 * i sees j when the call is not causal, when j <= i, or when j is one of the
 * first prefix[d] tokens of their document d.
 *   lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j
 * over the keys that i sees.  A token that sees none (one outside all
 * documents) gets out 0 and lse -infinity.
 *   q [tokens, heads, width]        of dtype (bf16 or fp16)
 *   k, v [tokens, kv_heads, width]  of dtype; kv_heads divides heads, query
 *                                   head h reads k and v head h / (heads / kv_heads)
 *   out [tokens, heads, width]      of dtype, contiguous
 *   lse [tokens, heads]             fp32, contiguous
 *   slopes [heads]                  fp32, or NULL
 *   documents [n_documents + 1]     int32: where documents start, and the last
 *                                   one's end, not decreasing, within [0,
 *                                   tokens]; or NULL: every `sequence` tokens
 *                                   are one (tokens is a multiple of it)
 *   prefix [n_documents]            int32 (one for each sequence where
 *                                   documents is NULL), or NULL: none
 * q, k, v (and grad_out) start on 16 bytes, and their token and head strides
 * are multiples of 8 elements.  tokens up to 2^24, heads up to 2^14, and tokens
 * / 128 times heads up to 2^30.
 * Scores and sums are fp32; exp(s - m), for a running m, is rounded to dtype
 * for the product with v.  Documents that share 128 consecutive tokens (from a
 * multiple of 128) share tensor-core operands: an infinity or a NaN in a k or
 * v row can reach other rows of those, and rows before it of its own document
 * (backward one in a q or grad_out row their grad_k and grad_v, too).  What is
 * finite changes no bit of a row that does not see it (fp16's gradients: of one of
 * another document).  Rows outside all documents reach nothing, whatever they hold.
 * A row that sees keys, all of whose scores are -infinity, gets NaN and lse
 * -infinity.  Documents that
 * decrease or lie outside give undefined results, within the outputs. */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const float* slopes;
  const int32_t* documents;
  const int32_t* prefix;
  int64_t tokens, sequence, n_documents;
  int64_t q_stride, k_stride, v_stride;                /* token to token */
  int64_t q_head_stride, k_head_stride, v_head_stride; /* head to head */
  int32_t heads, kv_heads, width;
  float scale;   /* finite, > 0 */
  float softcap; /* 0: none; else 1e-15 to 1e15, and scale^7 / softcap^6 at most 1e37 */
  int32_t dtype;
  uint32_t flags;
  uint32_t reserved; /* set to 0 */
} fadam_attention;

fadam_status fadam_attention_workspace(const fadam_attention* desc, size_t* bytes);
/* Errors: as fadam_embed_forward; FADAM_ELIMIT for more than 2^24 tokens or a
 * width beyond FADAM_ATTENTION_MAX_WIDTH. */
fadam_status fadam_attention_run(const fadam_attention* desc, void* workspace, size_t bytes,
                                 fadam_stream stream);

/* The gradients of q, k and v, from that of out and from what the forward
 * pass left: forward.out and forward.lse are read, out by its own strides.
 *   grad_out [tokens, heads, width]      of dtype
 *   grad_q [tokens, heads, width], grad_k, grad_v [tokens, kv_heads, width]
 *                                        of dtype, contiguous
 * grad_k and grad_v are summed over the query heads that share a head, in fp32
 * and in a fixed order.  p = exp(s - lse) and ds, its product with (grad_out . v
 * - grad_out . out), are rounded to dtype for the products; in fp16 after
 * multiplication by powers of two: p by 2^10, ds by one of its row.  That brings a
 * bound of the row's ds (max |grad_out| times the largest sum of a |v| row, and
 * |grad_out . out|) to [2^14, 2^15), so that no ds overflows, and those of 2^-28 of
 * the bound and more keep fp16's precision.  The bound is the query's own for
 * grad_q; for grad_k it is that of the key head's queries in the key's document:
 * other documents do not matter.  Nothing is summed by atomics: results are
 * deterministic. */
typedef struct {
  fadam_attention forward;
  const void* grad_out;
  void* grad_q;
  void* grad_k;
  void* grad_v;
  int64_t out_stride, out_head_stride;
  int64_t grad_out_stride, grad_out_head_stride;
} fadam_attention_grad;

fadam_status fadam_attention_backward_workspace(const fadam_attention_grad* desc, size_t* bytes);
fadam_status fadam_attention_backward(const fadam_attention_grad* desc, void* workspace,
                                      size_t bytes, fadam_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* FADAM_SEQ_H_ */
