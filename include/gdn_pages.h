/*
 * gdn_pages.h: C ABI of the operators on the pages of a pool, a cache of recurrent states (one page
 * per sequence, for instance [H, d, d] fp32) or of anything else of a fixed size.  Conventions of
 * gdn.h.  No passage of the pages applies; the fork is the cache's side of "Musings on long-context
 * fine-tuning", section "Isolating the recurrent layers" (one prefix state, many continuations).
 *
 * A pool is [num_pages, page_bytes] (page_bytes a multiple of 16, 16-byte aligned) and its `live`
 * flags are device int32 [num_pages], 0 for a free page.  Page numbers are device int32, read on
 * the device: nothing waits for the host, so the calls can be captured into a graph.  A page number
 * that a call cannot take sets a fault flag (gdn_device_faults: 2 a page outside its pool or a
 * parent that is not live, 4 a page that one call would write twice or both read and write, 8 no
 * free page; debug mode returns GDN_ERR_DEVICE_CHECK) and its entry is left out; the others are
 * done.  Lists and flags of one call do not overlap.  Calls on one pool are ordered by their stream.
 */
#ifndef GDN_PAGES_H_
#define GDN_PAGES_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace that any call below needs for a pool of num_pages pages (of pages_copy:
 * dst's) and lists of `count` entries.  Host only. */
gdn_status gdn_pages_workspace_size(int32_t num_pages, int32_t count, size_t *bytes);

/* dst[dst_pages[i]] = src[src_pages[i]] for i < count.  src_pages[i] = -1 writes zeros,
 * dst_pages[i] = -1 skips the pair.  dst and src are one pool (the same address; the page counts may
 * differ) or do not overlap.  Of pairs with the same destination (and pages in range) the first is
 * done; in one pool a pair whose source is another pair's destination is left out. */
gdn_status gdn_pages_copy(void *dst, int32_t dst_num_pages, const void *src, int32_t src_num_pages,
                          int64_t page_bytes, const int32_t *dst_pages, const int32_t *src_pages,
                          int32_t count, void *workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* Takes a free page for each parent, in order, the lowest free page first, copies the parent's page
 * to it (zeros for a parent of -1: a new sequence) and marks it live.  children[i] is the page taken,
 * or -1 when no page was free or parents[i] is not a live page.  A parent may be named many times. */
gdn_status gdn_pages_fork(void *pool, int32_t *live, int32_t num_pages, int64_t page_bytes,
                          const int32_t *parents, int32_t count, int32_t *children,
                          void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Marks pages free (-1 entries are skipped; freeing a free page does nothing). */
gdn_status gdn_pages_free(int32_t *live, int32_t num_pages, const int32_t *pages, int32_t count,
                          hipStream_t stream);

/* Moves the live pages into pages 0 .. L - 1 (L of them live) with the fewest copies: the live pages
 * at or past L go, in order, into the free pages before L.  remap[p] is where page p went (p if it
 * stayed), -1 if it was free.  Pages from L on keep their old bytes. */
gdn_status gdn_pages_compact(void *pool, int32_t *live, int32_t num_pages, int64_t page_bytes,
                             int32_t *remap, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_PAGES_H_ */
