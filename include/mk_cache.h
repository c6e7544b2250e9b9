/*
 * mk_cache.h -- C ABI for the paged KV cache around the decode step: who holds
 * which page (fork, resize, compact, copy) and attention that reads the pages
 * several sequences share once for all of them.
 *
 * The pools, page tables and lengths are those of mk.h: per layer and for K
 * and V a pool [num_pages][n_kv_heads][page_size][head_dim] in bf16, one table
 * row of page ids per sequence, post-RoPE keys.  Here the tables and lengths
 * live on the DEVICE, so that a batch can change without the host waiting;
 * copy them back for mk_build_schedule.
 *
 * Conventions as in mk.h: mk_status results, nothing throws, caller-owned
 * device memory, library-owned workspace, work enqueued on the stream given at
 * creation, asynchronous unless stated.  A handle's calls belong to one stream:
 * two calls of one handle that overlap on the GPU (from two streams, or two
 * captured graphs replayed side by side) race on its workspace; use one handle
 * for each.  Calls other than create, sync and destroy can be captured into a
 * CUDA graph (make the handle with the capturing stream).
 */
#ifndef MK_CACHE_H
#define MK_CACHE_H

#include "mk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- page ownership --------------------------------------------------------
 *
 * page_refs[p] is the number of table rows (or other holders the caller counts
 * there, such as a prefix kept for later) that hold page p; 0 means free.  A
 * sequence of length L uses the first ceil(L / page_size) entries of its row;
 * entries behind them are -1 and not read.  Calls keep one invariant of their
 * own: pages are handed out lowest id first, so results do not depend on timing.
 *
 * Every call is all or nothing.  A call whose DEVICE arguments are wrong (an id
 * or length out of range, the same destination twice, a used table entry that
 * names no held page) or that runs out of pages changes nothing; its status is
 * kept, the calls behind it change nothing either, and mk_kv_sync returns the
 * status and clears it. */

typedef struct {
  int32_t n_pools;            /* K and V pools of every layer: 2 * n_layers (at most 512) */
  int32_t num_pages;          /* pages in each pool (at most 2^21) */
  int32_t page_size;          /* tokens per page */
  int32_t n_seqs;             /* table rows (at most 65536) */
  int32_t max_pages_per_seq;  /* entries per row */
  int64_t page_bytes;         /* bytes of a page in one pool: n_kv_heads * page_size * head_dim * 2 */
  void *const *pools;         /* HOST array [n_pools] of DEVICE pointers, 16-byte aligned */
  int32_t *page_tables;       /* DEVICE [n_seqs][max_pages_per_seq] */
  int32_t *seq_lens;          /* DEVICE [n_seqs] */
  int32_t *page_refs;         /* DEVICE [num_pages] */
} mk_kv_desc;

typedef struct mk_kv mk_kv;

/* Checks the description (it is copied) and allocates the workspace.
 * MK_ERR_INVALID_ARG / MK_ERR_UNSUPPORTED / MK_ERR_NO_DEVICE / MK_ERR_CUDA. */
mk_status mk_kv_create(const mk_kv_desc *desc, void *stream, mk_kv **out);
void mk_kv_destroy(mk_kv *kv);

/* Copies page src_pages[i] over page dst_pages[i] in every pool (DEVICE int32
 * [n], n <= num_pages).  Tables and holders are not looked at.  Destinations
 * are distinct, and none is the source of another pair; src == dst does
 * nothing. */
mk_status mk_kv_copy_pages(mk_kv *kv, int32_t n, const int32_t *src_pages,
                           const int32_t *dst_pages);

/* Makes sequence dst_seqs[i] a copy of src_seqs[i] (DEVICE int32 [n], n <=
 * n_seqs), every source as it was before the call, so a permutation of beams is
 * one call.  Destinations are distinct; what they held is released first;
 * src == dst does nothing.  Full pages are shared; a last page that is partly
 * filled is copied into a free page of its own (one that was free or is
 * released by this call, and is no source of it), so that both sequences can be
 * appended to.  MK_ERR_NO_PAGES when there are too few. */
mk_status mk_kv_fork(mk_kv *kv, int32_t n, const int32_t *src_seqs, const int32_t *dst_seqs);

/* Sets the length of sequences seqs[i] (distinct) to new_lens[i] (DEVICE int32
 * [n], n <= n_seqs), the releases of all of them first.  Growing takes free
 * pages, and replaces a partly filled last page that has other holders by a
 * copy; their new positions hold whatever the pages held.  Shrinking releases
 * the pages behind the new length; 0 frees the sequence.  MK_ERR_NO_PAGES when
 * there are too few, MK_ERR_PAGE_OOB for a length behind the table row. */
mk_status mk_kv_resize(mk_kv *kv, int32_t n, const int32_t *seqs, const int32_t *new_lens);

/* Moves the held pages to the lowest ids: with H pages held, the k-th held page
 * with an id >= H goes to the k-th free id < H, in every pool; tables and
 * holders follow.  page_map: DEVICE int32 [num_pages] or NULL; receives each
 * page's new id, or -1 for a free page (what other holders need). */
mk_status mk_kv_compact(mk_kv *kv, int32_t *page_map);

/* Waits for the stream and returns the status of the first call that was
 * refused since the last mk_kv_sync (MK_OK if none was); clears it.
 * MK_ERR_INVALID_ARG while the stream is being captured. */
mk_status mk_kv_sync(mk_kv *kv);

#ifdef __cplusplus
}
#endif

#endif /* MK_CACHE_H */
