/*
 * spec_logits.h -- C ABI of logits processing in libspecverify.so: penalties for
 * repeated tokens, biases and grammar masks, applied to the rows that
 * spec_verify, spec_verify_tree or spec_sample read next.
 *
 * Row r of sequence b holds the logits after the sequence's history and the
 * drafted tokens on the way to r, so its token counts include them:
 *   chain (parent NULL): row r follows draft_tokens[b][0 .. r-1];
 *   tree: row r follows the tokens of node r and its ancestors except the
 *   root (spec_tree.h; entry 0 of draft_tokens and parent is ignored).
 * With c the occurrences of token x in the generated part of the history
 * (positions prompt_len .. history_len - 1) and on the row's drafted path, and
 * s whether x occurs there or in the prompt, in this order:
 *   y = s ? (x > 0 ? x / repetition : x * repetition) : x
 *   y = y - frequency * c - presence * [c > 0]
 *   y = y + (the sum of the sequence's biases for the token, in their order)
 *   y = -inf where the token's bit in `allowed` is 0
 * in fp32, rounded to the dtype once.  A logit that nothing touches keeps its
 * bits.  A row whose mask allows nothing becomes -inf throughout (which the
 * verification reports as a sequence error when it reads the row).
 *
 * Sequence errors fill the sequence's rows with NaN: repetition not finite or
 * not positive, frequency or presence not finite, lengths outside
 * 0 <= prompt_len <= history_len <= H, n_nodes outside [1, R], a history,
 * drafted or bias token outside [0, V) (bias -1 marks an unused entry), a
 * parent outside [0, n).
 */
#ifndef SPEC_LOGITS_H
#define SPEC_LOGITS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_LOGITS_MAX_ROWS 1024
#define SPEC_LOGITS_MAX_BIAS 4096

/*
 *   logits       device, [B, R, V] of dtype (SPEC_F32 or SPEC_BF16), contiguous
 *   out          the same shape; may be `logits` itself
 *   history      device int32 [B, H] or NULL (H = 0); history_len, prompt_len int32 [B] (not
 *                read where H = 0)
 *   draft_tokens device int32 [B, draft_cols] or NULL (draft_cols = 0): chain, draft_cols
 *                R - 1 or R; tree, draft_cols = R
 *   parent       device int32 [B, R] or NULL (a chain)
 *   n_nodes      device int32 [B] or NULL (R): rows from n_nodes[b] on are neither read nor
 *                written
 *   repetition, frequency, presence  device float [B] or NULL (1, 0, 0)
 *   bias_tokens  device int32 [B, bias_cols] or NULL (bias_cols = 0), bias_values float
 *                likewise
 *   allowed      device uint32 words, ceil(V / 32) for each mask, bit x % 32 of word x / 32
 *                for token x, or NULL; the mask of row (b, r) starts at word
 *                b * allowed_stride_b + r * allowed_stride_r (0: shared)
 * B >= 0 (0 is a no-op), 1 <= R <= SPEC_LOGITS_MAX_ROWS, 2 <= V <= SPEC_MAX_V,
 * 0 <= H <= 2^24, 0 <= bias_cols <= SPEC_LOGITS_MAX_BIAS.  logits and out 16-byte
 * aligned, the other arrays 4-byte aligned.  One kernel on `stream`, no
 * workspace and no allocation.  Returns SPEC_OK once launched, SPEC_EINVAL
 * for a size, pointer or alignment error, SPEC_ECUDA if the launch failed.
 */
typedef struct spec_process_logits_args {
    const void *logits;
    void *out;
    const int32_t *history, *history_len, *prompt_len;
    const int32_t *draft_tokens, *parent, *n_nodes;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_tokens;
    const float *bias_values;
    const uint32_t *allowed;
    int64_t allowed_stride_b, allowed_stride_r;
    int32_t B, R, V, H, draft_cols, bias_cols, dtype;
} spec_process_logits_args;

int32_t spec_process_logits(const spec_process_logits_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGITS_H */
