/*
 * kda_pages.h -- the pages of a cache (kda_attn.h) on MI355X (gfx950): which
 * request holds which, kept on the device, so that a serving step needs no
 * host round trip and can be captured into a graph.  Same library and
 * conventions as kda.h.
 *
 * State, all int32 on the device:
 *   table   [n_slots, max_pages]  the pages of each slot (request), in order
 *   lengths [n_slots]             tokens of each slot, in [0, max_pages * page_size]
 *   refs    [n_pages]             how many slots hold each page; 0 (or less): free
 * A slot holds the first ceil(lengths / page_size) entries of its row; the
 * calls set entries that a slot gives up to -1 and never read the others.
 * Several slots may hold one page (kda_kv_fork).  The calls keep refs equal
 * to the number of holders if it was so before; entries outside [0, n_pages)
 * are passed over.  Lengths out of range are clamped.  page_size as in
 * kda_attn.h.  Free pages are given out lowest number first.
 *
 * Sizes: n_slots * max_pages < 2^30, n_pages < 2^29, max_pages * page_size <
 * 2^30 (else KDA_ERR_TOO_LARGE).  Tensors 4-byte aligned, workspaces 16.
 * Results are deterministic: the counts are changed by integer atomics, whose
 * order does not matter.
 */
#ifndef KDA_PAGES_H_
#define KDA_PAGES_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_PAGES_MAX_TENSORS 16
#define KDA_PAGES_MAX_SLOTS 65536   /* slots, and pairs of a fork */

/*
 * Sets the length of every slot to want[slot] (clamped into [0, max_pages *
 * page_size]): grows it with free pages, or gives up the pages behind its new
 * end, as for drafts that were rejected; 0 frees the slot.  Pages are given up
 * first, then given out in the order of the slots.  ok[slot] is 1, or 0 for a
 * slot that wanted more pages than were left after those before it (the ones
 * that were refused included): it keeps its length and pages.
 *   A slot that is cut back into a page that others hold, too, still shares it,
 * and appending would write into theirs.  Fork it to another slot then: the
 * branch has its own copy of such an open page.
 *   want, ok int32 [n_slots]; ok may be NULL.
 */
int kda_kv_resize(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* want,
                  int32_t* ok, int32_t n_slots, int32_t max_pages, int32_t n_pages,
                  int32_t page_size, hipStream_t stream);

/*
 * Makes slot dst[i] a branch of slot src[i], for all i < n at once (every
 * source as it was before the call, so that slots may change places): dst
 * gives up its own pages and holds src's, except that a last page that is
 * not full is copied, so that both can be appended to.  Copies go to pages
 * that were free before the call, in the order of i.  ok[i] is 1, or 0 where
 * src[i] or dst[i] is no slot, an earlier i has the same dst, or no free page
 * was left for the copy: dst then stays as it is.  A pair without a copy (its
 * source ends with a full page or holds nothing) needs no free page.  src[i] ==
 * dst[i] changes nothing.
 *   src, dst, ok int32 [n]; ok may be NULL.  n <= KDA_PAGES_MAX_SLOTS.
 *   pages[t], page_bytes[t], page_stride_bytes[t], t < n_tensors <=
 *   KDA_PAGES_MAX_TENSORS: host arrays of the tensors that hold the pages'
 *   data (16-byte aligned, sizes and strides multiples of 16; page p of
 *   tensor t starts at pages[t] + p * page_stride_bytes[t]).
 *   workspace: kda_kv_fork_workspace_bytes(...).
 */
size_t kda_kv_fork_workspace_bytes(int32_t n, int32_t n_slots, int32_t max_pages);
int kda_kv_fork(int32_t* table, int32_t* lengths, int32_t* refs, const int32_t* src,
                const int32_t* dst, int32_t* ok, int32_t n, int32_t n_slots, int32_t max_pages,
                int32_t n_pages, int32_t page_size, void* const* pages, const int64_t* page_bytes,
                const int64_t* page_stride_bytes, int32_t n_tensors, void* workspace,
                size_t workspace_bytes, hipStream_t stream);

/*
 * Moves the pages in use to the numbers 0 .. n_live - 1: the k-th lowest page
 * in use from n_live on goes to the k-th lowest free one below.  Writes the
 * new table (entries behind a slot's pages: -1), the new refs and n_live int32
 * [1], and copies the pages' data.  table_out may be table itself and
 * refs_out refs itself.  The data of pages that are free afterwards stays.
 *   pages, page_bytes, page_stride_bytes, n_tensors as for kda_kv_fork.
 *   workspace: kda_kv_compact_workspace_bytes(...).
 */
size_t kda_kv_compact_workspace_bytes(int32_t n_pages);
int kda_kv_compact(const int32_t* table, const int32_t* lengths, const int32_t* refs,
                   int32_t* table_out, int32_t* refs_out, int32_t* n_live, int32_t n_slots,
                   int32_t max_pages, int32_t n_pages, int32_t page_size, void* const* pages,
                   const int64_t* page_bytes, const int64_t* page_stride_bytes, int32_t n_tensors,
                   void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_PAGES_H_ */
