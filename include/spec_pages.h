/*
 * spec_pages.h -- C ABI of a cache's pages in libspecverify.so: page tables forked
 * when sequences become beams or branches, pages taken, shared and freed, pages
 * copied, and the pages in use moved to the front of the pool.
 *
 * The pool's state is one array, ref_count int32 [num_pages]: how many entries of
 * page tables (the caller's, or others') refer to a page.  A page with count 0
 * is free.  A table row [pages_per_seq] holds its pages in order, then -1; a row
 * of length L needs ceil(L / page_size) of them and may hold more, for tokens to come.
 *
 * Results go to arrays of their own: no output shares a word with an input, so a
 * caller keeps two tables and two counts and lets them change places.  All
 * rules are deterministic: pages are taken in ascending order, by the rows in
 * order and within a row by position.
 */
#ifndef SPEC_PAGES_H
#define SPEC_PAGES_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_PAGES_MAX (1 << 24)

/*
 * New rows from old ones.  Row r of the new table takes over row parent[r] of the
 * old one with length[parent[r]], and room for reserve[r] more tokens:
 * It holds ceil((length + reserve) / page_size) pages:
 *   - those before page length / page_size are whole, and shared;
 *   - of the others ("private", written next) the first new row of a parent keeps those that
 *     nobody else refers to, and each of the rest is a free page (free before the call);
 *   - where the last page in use (length % page_size tokens) is replaced so, it is
 *     listed to be copied: copies[0][r], copies[1][r], copies[2][r] are its old page, its
 *     new page and its tokens; -1, -1, 0 where there is nothing to copy.
 * parent[r] = -1: a row of length 0, with pages for reserve[r] tokens.  Every old row gives up its
 * references, so pages that no new row has taken over lose them and may become free.
 *   table_in   device int32 [rows_in, pages_per_seq], length_in [rows_in]
 *   parent     device int32 [rows_out]; reserve likewise or NULL (0)
 *   table_out  [rows_out, pages_per_seq], length_out [rows_out], ref_out [num_pages],
 *              copies [3, rows_out]
 * Errors.  A parent outside [-1, rows_in), a reserve that is negative or that pages_per_seq does
 * not hold, and a parent row in error make a row of -1 with length_out -1 (which the other
 * operators report in their turn).  An old row in error (a length outside
 * 0 .. pages_per_seq * page_size, fewer pages than the length needs, a page
 * outside [0, num_pages)) keeps its references.  Where the free pages do not
 * suffice, every row is in error, and ref_out is ref_in.
 * 0 <= rows_in, rows_out <= 65535, 0 <= num_pages <= SPEC_PAGES_MAX, pages_per_seq * page_size <
 * 2^31.  Rows look for one another in `parent`, so the time grows with the square of
 * their number where there are many (512 rows: 19 us, 65535: 1.8 ms).  The
 * workspace has spec_pages_workspace_size bytes (0 for sizes out of range), 256-byte
 * aligned, need not be cleared and belongs to one call at a time.  One or two kernels
 * on `stream`, no allocation.
 */
typedef struct spec_pages_fork_args {
    const int32_t *table_in, *length_in, *parent, *reserve, *ref_in;
    int32_t *table_out, *length_out, *ref_out, *copies;
    int32_t rows_in, rows_out, pages_per_seq, page_size, num_pages;
} spec_pages_fork_args;

size_t spec_pages_workspace_size(int32_t rows_out, int32_t num_pages);
int32_t spec_pages_fork(const spec_pages_fork_args *args, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * Pages in use (count above 0) to the front: with n of them, the k-th page in use from n on
 * moves to the k-th free page below n.
 *   table_in   device int32 [rows, pages_per_seq]; entries outside [0, num_pages) are
 *              taken over as they are
 *   table_out, ref_out  the table and the counts after the moves
 *   copies     int32 [3, num_pages / 2]: source, destination, page_size of each
 *              move in order; then -1, -1, 0
 *   used       int32 [1]: n
 * Tables of other owners have to be in the same call.  Workspace as
 * spec_pages_fork's (rows_out = rows).  One to three kernels on `stream`.
 */
typedef struct spec_pages_compact_args {
    const int32_t *table_in, *ref_in;
    int32_t *table_out, *ref_out, *copies, *used;
    int32_t rows, pages_per_seq, page_size, num_pages;
} spec_pages_compact_args;

int32_t spec_pages_compact(const spec_pages_compact_args *args, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * Copy pages within the caches, in every layer: entry i copies the first
 * copies[2][i] slots of page copies[0][i] to page copies[1][i].  Entries with
 * a source, a destination or a number of slots out of range copy nothing (-1,
 * -1, 0 among them).  No entry's destination is another's source or destination.
 *   k_cache, v_cache  [layers, num_pages, page_size, Hkv, D], strides (layer,
 *                     page, slot, head) in elements, the last dimension contiguous
 *   copies            device int32 [3, n]
 * elem_size 2 or 4 bytes, any D >= 1; base addresses aligned to the element;
 * page_size * Hkv * D up to 2^30.  One kernel on `stream`.
 */
typedef struct spec_pages_copy_args {
    void *k_cache, *v_cache;
    int64_t k_cache_stride[4], v_cache_stride[4];
    const int32_t *copies;
    int32_t n, layers, Hkv, D, page_size, num_pages, elem_size;
} spec_pages_copy_args;

int32_t spec_pages_copy(const spec_pages_copy_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_PAGES_H */
