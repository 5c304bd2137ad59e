/*
 * kda_pages.h -- C ABI of the pages of a paged key-value cache (kda_layers.h):
 * handing them out, taking them back, sharing them between rows that go on from
 * the same tokens, and moving them together.
 *
 * All of it happens on the device, in the order of the stream, so that a captured
 * decoding loop can take pages as its rows grow.  The state is three arrays of the
 * caller's:
 *   page_table  [num_rows, max_pages] int32: token p of row i lives in page
 *               page_table[i][p / page_size], as for kda_paged_append; a row's
 *               pages are its first held[i] entries, and what the calls below
 *               give up becomes -1
 *   held        [num_rows] int32: pages that each row holds
 *   refs        [num_pages] int32: how many table entries (and other holders, which
 *               the caller may add) hold each page.  A page is free where it is 0;
 *               a negative count keeps it from ever being handed out, and no call
 *               changes the count (pages of the caller's own, which rows may share
 *               for good); kda_pages_compact moves such a page as any other in use,
 *               and its count with it, so that an id held outside the table has to
 *               follow page_map
 * All start as -1, 0 and 0.  Free pages are handed out lowest first, rows and
 * pairs served in order: results depend on the arguments alone.
 *
 * A page that several rows hold is only read: kda_pages_fork shares full pages
 * and copies the last one where it is partly filled.  A row that is cut back into
 * a page that it shares would write to it with its next token: cut it back to a
 * whole page, or fork it first.
 *
 * The conventions of kda_layers.h hold.  What these calls update is theirs alone
 * while they run: two calls on the same state go one after the other in a stream.
 * page_size is a power of two up to 1024, as the cache's.
 */
#ifndef KDA_GB300_PAGES_H
#define KDA_GB300_PAGES_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of kda_pages_resize: 0 (and the workspace may be NULL) for pools of up to 65536 pages, and for sizes
 * that it refuses. */
size_t kda_pages_resize_workspace_size(int num_rows, int max_pages, int num_pages);

/*
 * kda_pages_resize -- row i gets or gives back pages so that it holds those of
 * tokens[i] tokens, ceil(tokens[i] / page_size); 0 ends the row, a negative
 * number leaves it as it is.
 *   tokens      [num_rows] int32, device
 *   workspace   16-byte aligned, kda_pages_resize_workspace_size() bytes
 * Pages given back in a call are free for the rows that grow in it.  Where the
 * free pages run out, the rows that come too late get what is left or nothing:
 * held[i] says how many pages they have, and KDA_ERR_NO_PAGES is recorded.
 * Recorded as KDA_ERR_INVALID_ARG: more tokens than max_pages pages take, or
 * held[i] outside the table (the row is left as it is); an entry given back that
 * is no page, or one without holders (its count is left; a negative entry is
 * passed over).  num_rows * max_pages below 2^31.
 */
kda_status_t kda_pages_resize(int32_t *page_table, int num_rows, int max_pages, int32_t *held,
                              int32_t *refs, int num_pages, const int32_t *tokens, int page_size,
                              void *workspace, size_t workspace_bytes, uint32_t *status,
                              kda_stream_t stream);

/* Workspace bytes of kda_pages_fork; 0 for sizes that it refuses. */
size_t kda_pages_fork_workspace_size(int num_rows, int max_pages, int num_forks);

/*
 * kda_pages_fork -- row dst[i] goes on from the tokens of row src[i]: it shares
 * that row's full pages, and where the last page is partly filled gets a free
 * page with a copy of it in every pool.
 *   pools       num_pools device pointers (an array on the host, read before the
 *               call returns): tensors of num_pages pages each, such as keys,
 *               values and scales of all layers, no two of them overlapping
 *   page_bytes  num_pools sizes of a page in them (on the host), any >= 0; what is
 *               a multiple of 16, with the pool's address, is copied fastest
 *   lens        [num_rows] int32: tokens of each row; lens[dst[i]] becomes lens[src[i]]
 *   src, dst    [num_forks] int32, device; a pair with a negative row is padding
 *   workspace   16-byte aligned, kda_pages_fork_workspace_size() bytes
 * A row can be the source of many pairs and the destination of one, but not both
 * a source and a destination; a destination holds no pages before (kda_pages_resize
 * to 0).  Pairs that break this (of several with one destination, all but the
 * first), rows outside the table, lengths of more than the pages held, and a last
 * page that is none in use are recorded as KDA_ERR_INVALID_ARG and the pair left
 * out.  A pair for whose copy no page is free is left out and recorded as
 * KDA_ERR_NO_PAGES.  num_rows * max_pages below 2^31.
 */
kda_status_t kda_pages_fork(void *const *pools, const int64_t *page_bytes, int num_pools,
                            int32_t *page_table, int num_rows, int max_pages, int32_t *held,
                            int32_t *refs, int num_pages, int32_t *lens, const int32_t *src,
                            const int32_t *dst, int num_forks, int page_size, void *workspace,
                            size_t workspace_bytes, uint32_t *status, kda_stream_t stream);

/* Workspace bytes of kda_pages_compact; 0 for sizes that it refuses. */
size_t kda_pages_compact_workspace_size(int num_pages);

/*
 * kda_pages_compact -- moves the pages in use (refs not 0, negative ones among them)
 * to the front of all pools: of L of them, those with ids of L and more go, in order, to
 * the free ones below L; the others stay.  Table and counts follow.
 *   pools, page_bytes: as for kda_pages_fork
 *   page_map    [num_pages] int32 (written): the new id of each page, -1 for one
 *               that was free
 *   live        [1] int32 (written): L
 *   workspace   16-byte aligned, kda_pages_compact_workspace_size() bytes
 * Entries of the table that are negative stay; one that is no page in use becomes
 * -1 and is recorded as KDA_ERR_INVALID_ARG.  The table may be NULL where num_rows
 * or max_pages is 0 (page_map then serves the caller's own).
 */
kda_status_t kda_pages_compact(void *const *pools, const int64_t *page_bytes, int num_pools,
                               int32_t *page_table, int num_rows, int max_pages, int32_t *refs,
                               int num_pages, int32_t *page_map, int32_t *live, void *workspace,
                               size_t workspace_bytes, uint32_t *status, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_PAGES_H */
