/*
 * spec_chunk.h -- C ABI of chunks of new tokens in libspecverify.so: their keys
 * and values appended to a key/value cache, and their causal attention over it.
 * A prompt goes into the caches this way, in chunks of any length; sequences of
 * a batch may have any numbers of new tokens, single ones among them.
 *
 * The new tokens of all sequences lie one behind the other ("rows"): sequence
 * b's are rows row_start[b] .. row_start[b + 1] - 1, so row_start has B + 1
 * entries that do not decrease.  Rows before row_start[0] and from
 * row_start[B] on belong to no sequence and are left as they are.
 *
 * The cache of one layer is spec_attn.h's: [num_pages, page_size, Hkv, D] with
 * a page table [B, pages_per_seq], or without one (NULL) sequence b owns page b
 * (num_pages >= B, pages_per_seq = 1).  Positions that no sequence has yet, and
 * pages that none of its positions needs, may hold anything, NaN and invalid
 * page numbers included.
 *
 * Sequence errors mark only that sequence: plan status -1, attention rows NaN,
 * no append and length -1.  A row_start that decreases, or leaves 0 .. rows,
 * is an error of every sequence: all rows become NaN.
 */
#ifndef SPEC_CHUNK_H
#define SPEC_CHUNK_H

#include <stddef.h>
#include <stdint.h>

#include "spec_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_CHUNK_MAX_ROWS (1 << 24)

/*
 * Append rows' keys and values: row r of sequence b goes to position
 * cache_len[b] + r - row_start[b], for one layer or for all of them in one
 * launch; out_len[b] = cache_len[b] + the sequence's rows.
 * A sequence error (cache_len negative, a position past pages_per_seq *
 * page_size, a page of a new position outside [0, num_pages), a bad row_start)
 * leaves the sequence's cache as it is and writes out_len[b] = -1.
 *   k_new   [layers, rows, Hkv, D], strides (layer, row, head) in elements
 *   k_cache [layers, num_pages, page_size, Hkv, D], strides (layer, page, slot, head)
 *   row_start device int32 [B + 1]; cache_len, out_len device int32 [B]
 *   out_len shares no word with the int32 inputs
 * Two sequences' new positions must not share a slot.  elem_size 2 or 4 bytes;
 * any D >= 1, page_size >= 1, Hkv * D up to 2^24 and up to 2^20 heads that do
 * not lie one after the other, 0 <= rows <=
 * SPEC_CHUNK_MAX_ROWS, 0 <= B <= 65535; base addresses aligned to the element.
 * One kernel on `stream`, no allocation.
 */
typedef struct spec_chunk_append_args {
    const void *k_new, *v_new;
    void *k_cache, *v_cache;
    int64_t k_new_stride[3], v_new_stride[3], k_cache_stride[4], v_cache_stride[4];
    const int32_t *row_start, *cache_len, *page_table;
    int32_t *out_len;
    int32_t layers, B, rows, Hkv, D, page_size, pages_per_seq, num_pages, elem_size;
} spec_chunk_append_args;

int32_t spec_chunk_append(const spec_chunk_append_args *args, void *stream);

/*
 * The plan of a step, made once for all layers: device memory of
 * spec_chunk_plan_size(B, rows, group) bytes (0 for sizes out of range), 256-byte
 * aligned.  group = Hq / Hkv, 1 .. 128.
 *   kv_len  device int32 [B]: positions in the cache, the new tokens' included;
 *           row r of sequence b stands at position kv_len[b] - row_start[b + 1] + r
 * A sequence error is kv_len out of range or below the sequence's rows, a page
 * that a position below kv_len needs outside [0, num_pages), or a bad row_start.
 * Sequences without rows read nothing of their cache.  spec_chunk_plan_status
 * gives the byte offset of the statuses int32 [B] (0, or -1 for a sequence error).
 */
size_t spec_chunk_plan_size(int32_t B, int32_t rows, int32_t group);
size_t spec_chunk_plan_status(int32_t B, int32_t rows, int32_t group);
int32_t spec_chunk_plan(const int32_t *row_start, const int32_t *kv_len, const int32_t *page_table,
                        int32_t B, int32_t rows, int32_t group, int32_t page_size,
                        int32_t pages_per_seq, int32_t num_pages, void *plan, size_t plan_bytes,
                        void *stream);

/*
 * Attention of every row over its sequence's positions up to its own:
 *   out[r][h] = sum_j w_j v[j][h / G],  w = softmax_j(scale * q[r][h] . k[j][h / G]),
 *   G = Hq / Hkv, j = 0 .. the row's position.
 * Keys and values behind a row's position have no effect on it, NaN and
 * infinities included.
 *   q       [rows, Hq, D], strides q_stride (row, head) in elements
 *   k_cache [num_pages, page_size, Hkv, D], strides (page, slot, head); v_cache likewise
 *   plan    spec_chunk_plan's, of the same B, rows, G and cache geometry
 *   out     [rows, Hq, D] contiguous, of q's dtype
 *   out_lse float [rows, Hq] or NULL: ln sum_j exp(scale * q . k_j)
 * out may be q itself, where that is contiguous; otherwise the outputs share no memory with the
 * inputs (by their extents, strides included) or each other (SPEC_EINVAL).
 * dtype SPEC_BF16 or SPEC_F16, one for all tensors.  D a multiple of 8 up to
 * SPEC_ATTN_MAX_HEAD_DIM, Hq a multiple of Hkv, Hq / Hkv <= 128, scale finite
 * and positive; page_size a multiple of 128, or a power of two from 8, or,
 * without a page table, anything.  Base addresses 16-byte aligned, strides
 * multiples of 8 elements, none 0 along a dimension of more than one entry.
 * Scores, statistics and sums are fp32; weights are rounded to the dtype for
 * their product with v as spec_tree_attention's are.
 * The workspace has spec_chunk_attention_workspace_size bytes, 256-byte
 * aligned; it need not be cleared, and calls in flight must not share it.  Up
 * to two kernels on `stream`, no allocation.  A wait inside the kernel that
 * gives up marks the plan (spec_verify_read_status(plan, ..) reads
 * SPEC_DEV_WAIT_TIMEOUT until it is made again) and makes the rows concerned NaN.
 */
typedef struct spec_chunk_attention_args {
    const void *q, *k_cache, *v_cache;
    int64_t q_stride[2], k_cache_stride[3], v_cache_stride[3];
    const int32_t *page_table;
    const void *plan;
    void *out;
    float *out_lse;
    float scale;
    int32_t B, rows, Hq, Hkv, D, page_size, pages_per_seq, num_pages, dtype;
} spec_chunk_attention_args;

size_t spec_chunk_attention_workspace_size(int32_t Hq, int32_t Hkv, int32_t D);
int32_t spec_chunk_attention(const spec_chunk_attention_args *args, void *workspace,
                             size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CHUNK_H */
