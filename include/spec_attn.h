/*
 * spec_attn.h -- C ABI of tree attention over a key/value cache in
 * libspecverify.so: the attention of a batch of drafted trees (or chains, or
 * single tokens) over each sequence's cache, the plan it reads, and the
 * commit of the accepted path's keys and values once spec_verify or
 * spec_verify_tree has answered.
 *
 * Trees are spec_tree.h's: node 0 is the root (the last committed token, whose
 * key and value are not in the cache yet), node n >= 1 hangs below
 * parent[n] < n.  A chain of k drafts is parent[n] = n - 1 with k + 1 nodes, a
 * plain decoding step one node.
 *
 * The cache of one layer is [num_pages, page_size, Hkv, D] for keys and the
 * same for values, any strides with the last dimension contiguous.  With a
 * page table [B, pages_per_seq] position t of sequence b lies in page
 * page_table[b][t / page_size], slot t % page_size.  Without one (NULL) the
 * cache is contiguous: sequence b owns page b (num_pages >= B, pages_per_seq
 * = 1).  Positions from cache_len[b] on, and pages that no position below it
 * needs, may hold anything, NaN and invalid page numbers included.
 *
 * Sequence errors mark only that sequence: its plan status is -1, its
 * attention rows are NaN (which spec_verify reports as a sequence error), and
 * a commit leaves its cache alone and writes -1 for its length.
 */
#ifndef SPEC_ATTN_H
#define SPEC_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_F16 2 /* IEEE half: the attention's and the commit's dtypes only */
#define SPEC_ATTN_MAX_NODES 1024
#define SPEC_ATTN_MAX_HEAD_DIM 128

/*
 * The plan of a step: what every layer's attention needs of the trees and the
 * lengths, made once.  Device memory of spec_tree_plan_size(B, N) bytes (0 for
 * sizes out of range: 0 <= B <= 65535, 1 <= N <= SPEC_ATTN_MAX_NODES), 256-byte
 * aligned.  spec_tree_plan_offset gives the byte offset of a part that a caller
 * may read:
 *   SPEC_PLAN_POSITIONS int32 [B, N]: cache_len + depth of a node; -1 past n_nodes and in
 *                       sequences with an error
 *   SPEC_PLAN_STATUS    int32 [B]: 0, or -1 for a sequence error
 *   SPEC_PLAN_MASK      uint32 [B, N, W], W = 4 * ceil(N / 128): bit j % 32 of word j / 32 of
 *                       row n is set when node j is n or an ancestor of n
 */
enum { SPEC_PLAN_POSITIONS = 0, SPEC_PLAN_STATUS = 1, SPEC_PLAN_MASK = 2 };
size_t spec_tree_plan_size(int32_t B, int32_t N);
size_t spec_tree_plan_offset(int32_t B, int32_t N, int32_t part);

/*
 * Make the plan (one kernel on `stream`, no allocation).
 *   parent      device int32 [B, N]; entry 0 and entries from n_nodes[b] on are ignored
 *   n_nodes     device int32 [B], 0 .. N (0: an idle sequence, whose attention rows are 0)
 *   cache_len   device int32 [B], 0 .. pages_per_seq * page_size
 *   page_table  device int32 [B, pages_per_seq], or NULL (contiguous)
 * A sequence error is n_nodes or cache_len out of range, a parent outside
 * [0, n), or a page that a position below cache_len needs outside
 * [0, num_pages).  Returns SPEC_OK once launched, SPEC_EINVAL for a size,
 * pointer or alignment error, SPEC_ENOSPACE for a short plan, SPEC_ECUDA if
 * the launch failed.  B = 0 is a no-op, which writes no status word either.
 */
int32_t spec_tree_plan(const int32_t *parent, const int32_t *n_nodes, const int32_t *cache_len,
                       const int32_t *page_table, int32_t B, int32_t N, int32_t page_size,
                       int32_t pages_per_seq, int32_t num_pages, void *plan, size_t plan_bytes,
                       void *stream);

/*
 * Attention of every tree node over the cache and over its ancestors:
 *   out[b][n][h] = sum_j w_j v[j][h / G],  w = softmax_j(scale * q[b][n][h] . k[j][h / G]),
 *   G = Hq / Hkv, j over the cache positions below cache_len[b] and over the
 *   new keys of node n and its ancestors (the plan's mask).
 * Rows past n_nodes[b] are 0, and so is a row that sees no key.  Keys and
 * values that no row sees have no effect, NaN and infinities included; a
 * new key or value that some rows see affects those rows only.
 *   q       [B, N, Hq, D], strides q_stride (sequence, node, head) in elements
 *   k_new   [B, N, Hkv, D], v_new likewise: the new tokens' keys and values
 *   k_cache [num_pages, page_size, Hkv, D], strides (page, slot, head); v_cache
 *           likewise
 *   plan    spec_tree_plan's, of the same B, N and cache geometry
 *   out     [B, N, Hq, D] contiguous, of q's dtype
 *   out_lse float [B, N, Hq] or NULL: ln sum_j exp(scale * q . k_j), -inf where a row
 *           sees no key
 * dtype SPEC_BF16 or SPEC_F16, one for all tensors.  D a multiple of 8 up to
 * SPEC_ATTN_MAX_HEAD_DIM, Hq a multiple of Hkv, Hq / Hkv <= 128, scale finite
 * and positive; page_size a multiple of 128, or a power of two from 8, or, without a page
 * table, anything.  Base addresses 16-byte aligned, strides multiples of 8 elements.
 * Scores, the softmax's statistics and the weighted sum are held in fp32;
 * each weight is rounded to the dtype before its product with v (SPEC_F16: in
 * units of 2^-11 of the row's largest weight or less, so weights down to 2^-25
 * of it keep all of their bits).
 * The workspace has spec_tree_attention_workspace_size bytes (0 for sizes out
 * of range), 256-byte aligned; it need not be cleared, and calls in flight
 * must not share it.  Up to two kernels on `stream`, no allocation.
 * A wait inside the kernel that gives up marks the plan:
 * spec_verify_read_status(plan, ..) reads SPEC_DEV_WAIT_TIMEOUT until the
 * plan is made again (SPEC_DEV_OK otherwise).  Rows that the CTA of that wait
 * had a part in are then NaN, the other rows what they always are.
 */
typedef struct spec_tree_attention_args {
    const void *q, *k_new, *v_new, *k_cache, *v_cache;
    int64_t q_stride[3], k_new_stride[3], v_new_stride[3];
    int64_t k_cache_stride[3], v_cache_stride[3];
    const int32_t *page_table;
    const void *plan;
    void *out;
    float *out_lse;
    float scale;
    int32_t B, N, Hq, Hkv, D, page_size, pages_per_seq, num_pages, dtype;
} spec_tree_attention_args;

size_t spec_tree_attention_workspace_size(int32_t N, int32_t Hq, int32_t Hkv, int32_t D);
int32_t spec_tree_attention(const spec_tree_attention_args *args, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * Append the accepted path's keys and values to the cache, for one layer or
 * for all of them in one launch: with a = out_num_accepted[b], node 0 goes to
 * position cache_len[b] and node out_nodes[b][i - 1] (i itself when out_nodes
 * is NULL: a chain) to position cache_len[b] + i, i = 1 .. a;
 * out_len[b] = cache_len[b] + a + 1.
 * A sequence error (a outside [0, N), a node outside [0, N), a position past
 * pages_per_seq * page_size, a page outside [0, num_pages)) leaves the
 * sequence's cache as it is and writes out_len[b] = -1.
 *   k_new   [layers, B, N, Hkv, D], strides (layer, sequence, node, head) in elements
 *   k_cache [layers, num_pages, page_size, Hkv, D], strides (layer, page, slot, head)
 *   out_len device int32 [B], no word of it in cache_len or another int32 input
 * elem_size 2 or 4 bytes; any D >= 1, page_size >= 1, Hkv * D up to 2^24, and up to
 * 2^29 / N heads that do not lie one after the other; base addresses aligned
 * to the element.  One kernel on `stream`, no allocation.
 */
typedef struct spec_tree_commit_args {
    const void *k_new, *v_new;
    void *k_cache, *v_cache;
    int64_t k_new_stride[4], v_new_stride[4], k_cache_stride[4], v_cache_stride[4];
    const int32_t *cache_len, *out_num_accepted, *out_nodes, *page_table;
    int32_t *out_len;
    int32_t layers, B, N, Hkv, D, page_size, pages_per_seq, num_pages, elem_size;
} spec_tree_commit_args;

int32_t spec_tree_commit(const spec_tree_commit_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ATTN_H */
