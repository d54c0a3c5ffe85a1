/*
 * spec_beam.h -- C ABI of beam search in libspecverify.so: the selection over the beams
 * and the vocabulary, and the beams' states in the order of the selected.
 *
 * A sequence has K beams with log-probabilities s_k.  The candidates of a beam
 * are its continuations by every token x, with
 *   score(k, x) = s_k + logits[k][x] - ln sum_y exp(logits[k][y]);
 * a beam that has ended (finished) has one candidate, end_token at score s_k.
 * They are compared by score / norm_k (a power of the length, say), and the n
 * best are given in that order; of equal ones the lower k * V + x comes first.
 * The comparison is that of 64 bits: where fp32 statistics of two beams leave an
 * order open, the beams' sums are taken again exactly.
 *
 * Candidates with a logit of -inf, and all of a beam at s_k = -inf, do not count (logits
 * of such a beam, and of one that has ended, are not read); where fewer than n are left, tokens and beams are
 * -1 and scores -inf.  A sequence with a NaN or +inf logit in a row that counts, a
 * NaN or +inf s_k or a norm that is not positive and finite is in error: tokens and beams -1,
 * scores NaN.
 */
#ifndef SPEC_BEAM_H
#define SPEC_BEAM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_BEAM_MAX 64 /* beams, and candidates selected */

/*
 *   logits    device, [B, K, V] of dtype (SPEC_F32 or SPEC_BF16), contiguous, 16-byte aligned
 *   scores    device float [B, K]
 *   finished  device int32 [B, K] or NULL (none): not 0 for a beam that has ended
 *   norm      device float [B, K] or NULL (1)
 *   end_token in [0, V): the candidate of an ended beam
 *   out_tokens, out_beams  device int32 [B, n]; out_scores device float [B, n]: score(k, x)
 *   No output shares memory with an input or another output (SPEC_EINVAL): where an order is open the
 *   scores are read again after the outputs have been written.
 * 0 <= B <= 65535, 1 <= K, n <= SPEC_BEAM_MAX, 2 <= V <= SPEC_MAX_V.  The
 * workspace has spec_beam_workspace_size bytes (0 for sizes out of range),
 * 256-byte aligned, was zeroed once (spec_verify_workspace_reset does) and
 * resets itself; calls in flight must not share it.  Two kernels on
 * `stream`, no allocation.
 */
typedef struct spec_beam_select_args {
    const void *logits;
    const float *scores, *norm;
    const int32_t *finished;
    int32_t *out_tokens, *out_beams;
    float *out_scores;
    int32_t B, K, V, n, end_token, dtype;
} spec_beam_select_args;

size_t spec_beam_workspace_size(int32_t B, int32_t K, int32_t V, int32_t n, int32_t dtype);
int32_t spec_beam_select(const spec_beam_select_args *args, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * States in the order of the selected beams: out[l][b][j] = in[l][b][beams[b][j]],
 * rows of row_bytes bytes; 0 where beams[b][j] is outside [0, K) (-1: none).
 *   in [lead, B, K, row_bytes], out [lead, B, n, row_bytes], contiguous, apart from each other
 *   beams device int32 [B, n]
 * lead, B, K, n and row_bytes >= 0, lead * B * n < 2^31.  One kernel on `stream`.
 */
int32_t spec_beam_reorder(const void *in, const int32_t *beams, void *out, int32_t lead,
                          int32_t B, int32_t K, int32_t n, int64_t row_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_BEAM_H */
