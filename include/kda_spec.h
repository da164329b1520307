/*
 * kda_spec.h -- verification of drafted tokens against the target's
 * probabilities (MI355X, gfx950): the step of speculative decoding between
 * the model's outputs for the drafts and the next call's replay.  The next
 * kda_recurrent_fwd, kda_ssm_recurrent_fwd and kda_ssm_conv_step replay the
 * token before the drafts, if it ran with them, and the accepted drafts:
 * n_replay is n_accepted + 1.  Same library and conventions as kda.h.
 */
#ifndef KDA_SPEC_H_
#define KDA_SPEC_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_SPEC_MAX_DRAFTS 64

/*
 * For each request b with K_b = min(K, n_draft[b]) drafted tokens d_i:
 *
 *   draft i stands while  u_i q_i(d_i) < p_i(d_i),   i = 0, 1, ...
 *   n_accepted = the number of drafts before the first that does not;
 *   the token after them comes from r(v) = max(p_n(v) - q_n(v), 0) at the
 *   first draft that does not stand (n = n_accepted < K_b), or from p_n
 *   after the last draft (n = K_b): the lowest v with
 *   sum_{v' <= v} r(v') > u_next sum r.
 *
 * so that, with u and u_next uniform in [0, 1), the tokens follow the
 * target's distribution.  p_target [B, K + 1, V] and p_draft [B, K, V] are
 * in in_dtype and need not be normalised exactly; entries that are not
 * greater than zero (NaN among them) count as zero.  p_draft NULL: the
 * drafts were chosen, not sampled, and q is one at the draft, zero
 * elsewhere.  If r has no positive entry, p_n takes its place, and if that
 * has none either, the token is 0.  A draft outside [0, V) does not stand
 * and takes nothing from r.
 *   drafts int32 [B, K]; n_draft int32 [B] (clamped into [0, K]) or NULL for
 *   K; u float32 [B, K]; u_next float32 [B]; n_accepted int32 [B];
 *   tokens int32 [B, K + 1]: the accepted drafts, the token after them, then
 *   -1.  0 <= K <= KDA_SPEC_MAX_DRAFTS, 1 <= V < 2^31.
 * Products and sums run in float64, so that rounding does not move a border;
 * products of float32 values are exact there.
 *   workspace: kda_verify_drafts_workspace_bytes(...), 16-byte aligned,
 *   contents clobbered.
 * Tensor alignment: 16 bytes for p_target and p_draft, 4 for the others.
 */
size_t kda_verify_drafts_workspace_bytes(int32_t B, int32_t K, int64_t V);
int kda_verify_drafts(const void* p_target, const void* p_draft, int in_dtype,
                      const int32_t* drafts, const int32_t* n_draft, const float* u,
                      const float* u_next, int32_t B, int32_t K, int64_t V, int32_t* n_accepted,
                      int32_t* tokens, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_SPEC_H_ */
