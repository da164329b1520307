/*
 * kda_attn.h -- C ABI of softmax attention on MI355X (gfx950): full
 * attention layers with grouped heads, one width of 64 or 128 for queries, keys
 * and values, beside the layers of kda.h and kda_ssm.h, in the same library,
 * with the same conventions.  Whole prompts with their gradients, and new
 * tokens of requests over a paged cache of keys and values (whose pages
 * kda_pages.h looks after).
 *
 * Row i is a token with a query head h; group g = h / (H / G) holds the keys
 * and values that the H / G consecutive heads of the group share:
 *
 *     s_ij  = scale q_i . k_j          for the tokens j that row i sees
 *     lse_i = log sum_j e^{s_ij}
 *     o_i   = sum_j e^{s_ij - lse_i} v_j
 *
 * With causal != 0 a row sees the tokens of its sequence up to its own; with
 * 0 all of them.  A row that sees no token has o = 0 and lse = -infinity; one
 * whose query, or a key that it sees, holds a NaN has NaN in both.
 *
 * Common contract (beside that of kda.h, which holds here too: device
 * pointers, 16-byte alignment (lse, cu_seqlens, table, lengths 4-byte),
 * validation before anything is enqueued, nothing allocated, no host
 * synchronisation, deterministic results without atomics, `stream` on the
 * current device):
 *   - Sizes: head dimension D 64 or 128, H a multiple of G, H <=
 *     KDA_MAX_HEADS, H * D <= KDA_ATTN_MAX_STRIDE, H / G times the tokens of
 *     a sequence (packed: of the batch) at most 2^30, scale log2 e within
 *     float32 (anything else -> KDA_ERR_BAD_SHAPE / _TOO_LARGE).
 *   - in_dtype (KDA_BF16 or KDA_F32) is the type of q, k, v, o and of their
 *     gradients; lse is float32.
 *   - Token rows: a `_stride` is the number of elements from one token row to
 *     the next (a multiple of 16 bytes, at most KDA_ATTN_MAX_STRIDE), so q, k
 *     and v, and their gradients, can be columns of one projection's rows.
 *     Row b * T + t holds token t of sequence b; a row [heads, D] itself is
 *     contiguous.  Tensors without a stride are contiguous.
 *   - Packed batches: cu_seqlens int32 [n_seqs + 1] on the device, with T the
 *     number of token rows.  Rows before cu_seqlens[0] and from
 *     cu_seqlens[n_seqs] on belong to no sequence: they affect nothing and
 *     their outputs keep what they held.  The device clamps each range into
 *     [0, T].  Sequences may be empty.
 *   - Scores (times log2 e) must be within float32.  A NaN or an infinity in q
 *     reaches its own row only, one in k or v the rows that see its token (an
 *     infinity perhaps as a NaN): rows that do not, but share a tile of keys
 *     with it, are computed once more key by key.  In the backward pass a
 *     masked weight of zero is multiplied with whatever stands there: a NaN or
 *     an infinity in any input can also reach gradients of tokens up to 94 away
 *     in its own sequence and group, on the side that does not see it.  What
 *     lies outside a sequence, behind a request's length or in pages that it
 *     does not hold is never part of a product.
 *   - Numerics: scores, softmax statistics and sums in float32.  With
 *     KDA_BF16 the weights (and in the backward pass the score gradients)
 *     are rounded to bf16 once, as operands of the matrix cores: a half step
 *     of the output's own type.  grad_q's delta is that of o as it was rounded,
 *     grad_k's is exact to float32.  With KDA_F32 nothing is rounded below
 *     float32.
 */
#ifndef KDA_ATTN_H_
#define KDA_ATTN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ATTN_MAX_STRIDE (1 << 20)   /* elements */

/*
 * Attention over whole sequences.
 *   q [rows, H, D] (q_stride), k, v [rows, G, D] (k_stride, v_stride),
 *   o [rows, H, D] contiguous, lse float32 [rows, H] or NULL.
 */
int kda_attn_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                 int64_t v_stride, int in_dtype, const int32_t* cu_seqlens, int32_t n_seqs,
                 int64_t T, int32_t H, int32_t G, int32_t D, float scale, int causal, void* o,
                 float* lse, hipStream_t stream);

/*
 * Backward pass of kda_attn_fwd: inputs as for that call, with the o and lse
 * that it gave, and grad_o = dL/do (in_dtype, contiguous).  Writes grad_q,
 * grad_k, grad_v (in_dtype, with row strides; they may be columns of the same
 * rows).  With P the softmax weights:
 *     delta_i = grad_o_i . o_i
 *     dS_ij   = P_ij (grad_o_i . v_j - delta_i)
 *     grad_q_i = scale sum_j dS_ij k_j
 *     grad_k_j = scale sum_i dS_ij q_i,   grad_v_j = sum_i P_ij grad_o_i
 * summed over the group's heads in float32 and rounded once.
 *   workspace: kda_attn_bwd_workspace_bytes(...), 16-byte aligned, clobbered.
 */
size_t kda_attn_bwd_workspace_bytes(int in_dtype, int32_t n_seqs, int64_t T, int32_t H, int32_t G,
                                    int32_t D, int varlen);
int kda_attn_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                 int64_t v_stride, int in_dtype, const int32_t* cu_seqlens, int32_t n_seqs,
                 int64_t T, int32_t H, int32_t G, int32_t D, float scale, int causal, const void* o,
                 const float* lse, const void* grad_o, void* grad_q, int64_t grad_q_stride,
                 void* grad_k, int64_t grad_k_stride, void* grad_v, int64_t grad_v_stride,
                 void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * A paged cache: k_pages, v_pages [n_pages, G, page_size, D] in in_dtype, each
 * page contiguous and page_stride elements after the one before it (a
 * multiple of 16 bytes; pages of several layers can share one pool).
 * page_size is 16, 32, 64, 128 or 256.  Token x of request b lies in row x %
 * page_size of page table[b, x / page_size]; table int32 [n_seqs, max_pages],
 * lengths int32 [n_seqs] the tokens of each request (clamped into [0,
 * max_pages * page_size]).  A table entry outside [0, n_pages) stands for no
 * page: its tokens are seen by no row, and appended to nowhere.
 *
 * The new tokens of request b are its last ones: with T_b of them (T, or in a
 * packed batch cu_seqlens[b + 1] - cu_seqlens[b]), new token t has position
 * lengths[b] - T_b + t.  One with a negative position is not there.
 *
 * kda_kv_append writes the new tokens' k and v (rows with k_stride, v_stride)
 * into their pages.  No two of them may share a place: which is kept is
 * undefined.  A page is written to whoever else holds it (kda_pages.h says when
 * an open page can be shared).
 */
int kda_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int in_dtype,
                  void* k_pages, void* v_pages, int64_t page_stride, int32_t n_pages,
                  int32_t page_size, const int32_t* table, int32_t max_pages,
                  const int32_t* lengths, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                  int32_t G, int32_t D, hipStream_t stream);

/*
 * Attention of the new tokens' queries over all tokens of their requests up to
 * their own (the pages hold the new tokens' k and v already: kda_kv_append).
 * Any number of new tokens per request: one, drafts, a chunk of a prompt.
 *   q [rows, H, D] (q_stride), o [rows, H, D] contiguous, lse [rows, H] or NULL.
 *   workspace: kda_attn_paged_workspace_bytes(...), 16-byte aligned, clobbered:
 *   results over parts of long requests, which a second launch joins.
 */
size_t kda_attn_paged_workspace_bytes(int in_dtype, int32_t n_seqs, int64_t T, int32_t H,
                                      int32_t G, int32_t D, int32_t page_size, int32_t max_pages,
                                      int varlen);
int kda_attn_paged_fwd(const void* q, int64_t q_stride, int in_dtype, const void* k_pages,
                       const void* v_pages, int64_t page_stride, int32_t n_pages,
                       int32_t page_size, const int32_t* table, int32_t max_pages,
                       const int32_t* lengths, const int32_t* cu_seqlens, int32_t n_seqs,
                       int64_t T, int32_t H, int32_t G, int32_t D, float scale, void* o, float* lse,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTN_H_ */
