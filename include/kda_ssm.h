/*
 * kda_ssm.h -- C ABI of the selective state space scan and its short causal
 * convolution on MI355X (gfx950): the scalar-decay sibling of the operators
 * in kda.h, in the same library, with the same conventions.
 *
 * Scan, per head h with state S in R^{N x P}, token t:
 *
 *     dt_t = softplus(dt_raw_t + dt_bias_h)      (or dt_raw_t + dt_bias_h)
 *     a_t  = dt_t A_h                            (log decay, <= 0)
 *     S_t  = e^{a_t} S_{t-1} + dt_t B_t x_t^T
 *     y_t  = S_t^T C_t + D_h x_t                 (read after the update)
 *
 * B_t, C_t in R^N are shared by the H / G consecutive heads of a group,
 * x_t, y_t in R^P are the head's own.  Short convolution, per channel c:
 *
 *     z_t = bias + sum_{j<W} w_j x_{t-W+1+j},    y_t = z_t sigmoid(z_t)
 *
 * Common contract (beside that of kda.h, which holds here too: device
 * pointers, 16-byte alignment (dt, A, D, dt_bias, bias, cu_seqlens, n_replay
 * 4-byte), validation before anything is enqueued, nothing allocated, no
 * host synchronisation, deterministic results, `stream` on the current
 * device):
 *   - Sizes: head dimension P 64 or 128, state dimension N 64 or 128, H a
 *     multiple of G, H <= KDA_MAX_HEADS; convolution width W 2, 3 or 4 and
 *     channels a multiple of 8 (anything else -> KDA_ERR_BAD_SHAPE).
 *   - in_dtype (KDA_BF16 or KDA_F32) is the type of x, B, C, y and of their
 *     gradients; everything else is float32.
 *   - A must be <= 0 and dt >= 0 (softplus gives that); larger values can
 *     overflow but never address memory out of bounds.  Inputs must be
 *     finite: tokens are evaluated 64 at a time, so a NaN or infinity in one
 *     token can reach outputs of the 63 tokens before it as well as all
 *     later ones of that head's sequence (not other sequences).
 *   - Token rows: tensors with a `_stride` argument may be parts of wider
 *     rows; the argument is the number of elements from one token row to the
 *     next (a multiple of 16 bytes, at most KDA_SSM_MAX_STRIDE elements), so
 *     x, B and C can be the channels that one convolution put out.  Row
 *     b * T + t holds token t of sequence b; the row itself is contiguous.
 *     Tensors without one are contiguous.
 *   - Packed batches: cu_seqlens int32 [n_seqs + 1] on the device, as in
 *     kda.h, with T the number of token rows.  Rows before cu_seqlens[0] and
 *     from cu_seqlens[n_seqs] on belong to no sequence: they affect nothing,
 *     and outputs keep what they held there.  The device clamps each range
 *     into [0, T].
 *   - Sequences of length zero are allowed: S_T is S0, the cache stays.
 */
#ifndef KDA_SSM_H_
#define KDA_SSM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest row stride (elements) of a token row.  Sequences of the scan have at
 * most 2^30 tokens (KDA_ERR_TOO_LARGE). */
#define KDA_SSM_MAX_STRIDE (1 << 23)

/*
 * Short causal convolution of whole sequences.
 *   x [rows, channels] (x_stride), y [rows, channels] contiguous, w float32
 *   [channels, width] (tap width-1 applies to the token itself), bias
 *   float32 [channels] or NULL; activation 0: y = z, 1: y = z sigmoid(z).
 *   cache float32 [n_seqs, width-1, channels] or NULL (zeros): the inputs
 *   before each sequence's first token, oldest first; afterwards it holds
 *   the last width-1 inputs of each sequence (older entries shift in for
 *   sequences shorter than that).
 */
int kda_ssm_conv_fwd(const void* x, int64_t x_stride, int in_dtype, const float* w,
                     const float* bias, float* cache, const int32_t* cu_seqlens, int32_t n_seqs,
                     int64_t T, int32_t channels, int32_t width, int activation, void* y,
                     hipStream_t stream);

/*
 * The same for 0..64 new tokens of each of B requests, for decoding: the
 * cache first takes in the first n_replay[b] (clamped into [0, Tr]; NULL:
 * all) of the Tr <= 64 replay tokens, whose outputs an earlier call gave;
 * then the T tokens are convolved; then the cache holds the inputs up to
 * the replayed ones (commit == 0) or up to the last token (commit != 0).
 * These are the semantics of kda_recurrent_fwd: the replay tokens are the
 * previous step's drafts and n_replay the accepted counts.
 *   x [B, T, channels] (x_stride), rx [B, Tr, channels] (rx_stride) or NULL
 *   when Tr == 0, cache as above with n_seqs = B (required).
 */
int kda_ssm_conv_step(const void* x, int64_t x_stride, int in_dtype, const float* w,
                      const float* bias, float* cache, const void* rx, int64_t rx_stride,
                      const int32_t* n_replay, int32_t B, int32_t T, int32_t Tr,
                      int32_t channels, int32_t width, int activation, int commit, void* y,
                      hipStream_t stream);

/*
 * Backward pass of kda_ssm_conv_fwd: given grad_y = dL/dy (in_dtype,
 * grad_y_stride), writes grad_x (in_dtype, contiguous), grad_w, grad_bias
 * (float32; grad_bias may be NULL) and, if not NULL, grad_cache.  `cache` is
 * the one before the forward call (which overwrites it), or NULL; the cache
 * that the forward call leaves behind carries no gradient.  Sums over
 * tokens run in float32, in an order that depends on the sizes only.
 * Rows of grad_x outside every sequence are not written.
 * workspace: kda_ssm_conv_bwd_workspace_bytes(...), contents clobbered.
 */
size_t kda_ssm_conv_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t width);
int kda_ssm_conv_bwd(const void* x, int64_t x_stride, int in_dtype, const float* w,
                     const float* bias, const float* cache, const int32_t* cu_seqlens,
                     int32_t n_seqs, int64_t T, int32_t channels, int32_t width, int activation,
                     const void* grad_y, int64_t grad_y_stride, void* grad_x, float* grad_w,
                     float* grad_bias, float* grad_cache, void* workspace,
                     size_t workspace_bytes, hipStream_t stream);

/*
 * Scan over whole sequences, in chunks of 64 tokens (32 with KDA_F32).
 *   x [rows, H, P] (x_stride), B, C [rows, G, N] (B_stride, C_stride),
 *   dt [rows, H], dt_bias [H] or NULL, A [H], D [H] or NULL,
 *   S0 [n_seqs, H, N, P] or NULL (zeros), y [rows, H, P] contiguous,
 *   S_T [n_seqs, H, N, P] or NULL; S_T may be S0 itself.
 *   softplus != 0 applies softplus to dt + dt_bias.
 * With few (sequence, head) pairs and long sequences each sequence is cut
 * into segments that run side by side: their local final states come first,
 * a merge gives each segment's incoming state, then all outputs run.  That
 * needs at most kda_ssm_chunk_fwd_workspace_bytes(...), the larger need of the
 * two types (0: neither is cut); with less than its own type's need (or NULL)
 * every sequence runs as one chain, with the same result up to rounding.
 * Numerics: decay sums in float64 within a chunk, everything else
 * accumulated in float32.  The products run on bf16 matrix cores.  The state
 * update takes its float32 operands (and, with KDA_F32, the inputs) as sums
 * of three bf16 parts, so S_T is accurate to float32 rounding; so is y with
 * KDA_F32.  With KDA_BF16, the weighted products C . B within a chunk are
 * rounded to bf16, a half step of the output's type; S enters S^T C as the sum
 * of two bf16 parts (2^-16 of it is lost), and D x is added in float32.
 * A token with dt A < -104 (a reset) ends all memory.  One with dt = 0 (the
 * softplus of a large negative number) leaves the state as it is, so a batch
 * may be padded at its end with finite tokens of such dt.
 */
size_t kda_ssm_chunk_fwd_workspace_bytes(int32_t n_seqs, int64_t T, int32_t H, int32_t G,
                                         int32_t N, int32_t P, int varlen);
int kda_ssm_chunk_fwd(const void* x, int64_t x_stride, const void* B, int64_t B_stride,
                      const void* C, int64_t C_stride, int in_dtype, const float* dt,
                      const float* dt_bias, int softplus, const float* A, const float* D,
                      const float* S0, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                      int32_t H, int32_t G, int32_t N, int32_t P, void* y, float* S_T,
                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Backward pass of kda_ssm_chunk_fwd: inputs as for that call, grad_y =
 * dL/dy (in_dtype, contiguous), grad_S_T float32 or NULL (zero).  Writes
 *   grad_x, grad_B, grad_C (in_dtype, with row strides; they may be parts
 *   of the same rows), grad_dt [rows, H], grad_A, grad_D, grad_dt_bias [H]
 *   (the last two may be NULL) and grad_S0 [n_seqs, H, N, P] or NULL (it may
 *   be grad_S_T itself).
 * grad_B and grad_C are summed over a group's heads in float32 and rounded
 * once.  grad_dt is the gradient of the raw dt.
 * Numerics: as for the forward call, the float32 gradients to float32
 * rounding.  With KDA_BF16, the weighted products C . B (for grad_x) and
 * grad_y . x (for grad_B and grad_C, per head) within a chunk and the state
 * gradient in grad_x are rounded to bf16 once each; D grad_y is added in
 * float32.
 * workspace: at least kda_ssm_chunk_bwd_workspace_bytes(..., 1) and at most
 * useful kda_ssm_chunk_bwd_workspace_bytes(..., G) bytes, 16-byte aligned,
 * clobbered: it holds the state at every chunk's start (64 tokens; 32
 * with KDA_F32) and the state gradient at its end for as many groups of
 * heads at a time as fit.
 */
size_t kda_ssm_chunk_bwd_workspace_bytes(int in_dtype, int32_t n_seqs, int64_t T, int32_t H,
                                         int32_t G, int32_t N, int32_t P, int varlen,
                                         int32_t groups);
int kda_ssm_chunk_bwd(const void* x, int64_t x_stride, const void* B, int64_t B_stride,
                      const void* C, int64_t C_stride, int in_dtype, const float* dt,
                      const float* dt_bias, int softplus, const float* A, const float* D,
                      const float* S0, const int32_t* cu_seqlens, int32_t n_seqs, int64_t T,
                      int32_t H, int32_t G, int32_t N, int32_t P, const void* grad_y,
                      const float* grad_S_T, void* grad_x, int64_t grad_x_stride, void* grad_B,
                      int64_t grad_B_stride, void* grad_C, int64_t grad_C_stride, float* grad_dt,
                      float* grad_A, float* grad_D, float* grad_dt_bias, float* grad_S0,
                      void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * The scan for 0..64 new tokens of each of B requests, states in place, with
 * replay: the state takes in the first n_replay[b] (clamped into [0, Tr];
 * NULL: all) of the Tr <= 64 replay tokens, then the T tokens run with their
 * outputs, and the state is stored after the replay (commit == 0) or after
 * all tokens (commit != 0), as in kda_recurrent_fwd.
 *   x [B, T, H, P] (x_stride), Bm, C [B, T, G, N] (B_stride, C_stride),
 *   dt [B, T, H]; rx [B, Tr, H, P] (rx_stride), rB [B, Tr, G, N]
 *   (rB_stride), rdt [B, Tr, H] (NULL when Tr == 0); S [B, H, N, P];
 *   y [B, T, H, P] contiguous, in_dtype.
 * Numerics: float32 throughout.
 */
int kda_ssm_recurrent_fwd(const void* x, int64_t x_stride, const void* Bm, int64_t B_stride,
                          const void* C, int64_t C_stride, int in_dtype, const float* dt,
                          const float* dt_bias, int softplus, const float* A, const float* D,
                          const void* rx, int64_t rx_stride, const void* rB, int64_t rB_stride,
                          const float* rdt, const int32_t* n_replay, float* S, int32_t B,
                          int32_t T, int32_t Tr, int32_t H, int32_t G, int32_t N, int32_t P,
                          int commit, void* y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_SSM_H_ */
