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
 * status and clears it.  Where several arguments of a call are wrong, a page or
 * length out of range (MK_ERR_PAGE_OOB) is reported before anything else
 * (MK_ERR_INVALID_ARG), and both before MK_ERR_NO_PAGES. */

typedef struct {
  int32_t n_pools;            /* K and V pools of every layer: 2 * n_layers (at most 512) */
  int32_t num_pages;          /* pages in each pool (at most 2^20) */
  int32_t page_size;          /* tokens per page */
  int32_t n_seqs;             /* table rows (at most 65536) */
  int32_t max_pages_per_seq;  /* entries per row; n_seqs rows have at most 2^30 */
  int64_t page_bytes;         /* bytes of a page in one pool: n_kv_heads * page_size * head_dim * 2 */
  void *const *pools;         /* HOST array [n_pools] of DEVICE pointers, 16-byte aligned */
  int32_t *page_tables;       /* DEVICE [n_seqs][max_pages_per_seq] */
  int32_t *seq_lens;          /* DEVICE [n_seqs] */
  int32_t *page_refs;         /* DEVICE [num_pages] */
} mk_kv_desc;

typedef struct mk_kv mk_kv;

/* Checks the description (it is copied) and allocates the workspace: 4 bytes for
 * each table entry, 20 for each page (or 16, and 4 for each row where there are more
 * rows), 16 for each row.
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
 * [n], n <= n_seqs), the releases of all of them first: what shrinking rows hold
 * alone, growing ones can take.  Growing takes free pages, and replaces a partly
 * filled last page that had other holders before the call by a copy; the new
 * positions hold whatever the pages held.  Every row that grows out of such a page
 * takes a copy, also where the others leave the page in the same call, and the page
 * is free behind the call if nobody is left: to keep it for the last one, resize the
 * others in a call before.  Shrinking releases the pages behind the new length; 0
 * frees the sequence.  MK_ERR_NO_PAGES when
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

/* ---- attention over shared pages -------------------------------------------
 *
 * A batch of sequences, each with one or more query tokens, attends to its paged
 * K and V.  Consecutive sequences form groups; the first prefix_lens[g] tokens
 * of a group's sequences lie in the same pages, and those pages are read once
 * for all of the group's query tokens and heads (single tokens of 64 samples of
 * one prompt read the prompt once instead of 64 times). */

typedef struct {
  int32_t n_q_heads, n_kv_heads, head_dim;   /* as mk_create; n_q_heads / n_kv_heads <= 64 */
  int32_t page_size, num_pages;              /* page_size a multiple of 16, at most 256 */
  int32_t max_tokens;                        /* query tokens of a call, at most 2^20 */
  int32_t max_seqs, max_groups;              /* of a call, at most 1024 and 512 */
  int32_t n_layers;
  const void *const *k_caches;               /* HOST arrays [n_layers] of DEVICE pools */
  const void *const *v_caches;
  float scale;                               /* of the scores, below 2^127; 0: 1 / sqrt(head_dim) */
} mk_attn_desc;

/* A call's batch.  The arrays are DEVICE memory and are read by the call on the
 * GPU, so they can be updated between replays of a captured call. */
typedef struct {
  int32_t n_seqs, n_tokens;
  int32_t n_groups;                 /* 0: no sequence shares pages */
  int32_t max_pages_per_seq;        /* entries of a table row */
  const int32_t *page_tables;       /* [n_seqs][max_pages_per_seq] */
  const int32_t *seq_lens;          /* [n_seqs] cached tokens, the query tokens among them */
  const int32_t *q_offsets;         /* [n_seqs + 1] from 0, not decreasing, the last one <=
                                     * n_tokens: sequence b's query tokens; or NULL: one
                                     * token each, n_tokens == n_seqs */
  const int32_t *group_starts;      /* [n_groups + 1] from 0 to n_seqs, not decreasing */
  const int32_t *prefix_lens;       /* [n_groups] */
} mk_attn_batch;

typedef struct mk_attn mk_attn;

/* Allocates the workspace: two fp32 partial results of every query token and head and
 * 512 rows of them an SM, 4 * head_dim + 8 bytes each, and 32 bytes for each token and
 * kv head.  With 32 heads of 128 on 152 SMs that is 43 MB for 64 tokens, 201 MB for
 * 4800, 588 MB for 16384.
 * MK_ERR_INVALID_ARG / MK_ERR_UNSUPPORTED / MK_ERR_NO_DEVICE / MK_ERR_CUDA. */
mk_status mk_attn_create(const mk_attn_desc *desc, void *stream, mk_attn **out);
void mk_attn_destroy(mk_attn *attn);

/* Attention of the batch's query tokens over layer `layer`'s pools.  With T
 * query tokens and length L, query t of a sequence sits at position L - T + t
 * and sees the keys at positions <= its own (K and V of the query tokens are in
 * the cache already).  q: bf16 [n_tokens][n_q_heads][head_dim], q_token_stride
 * elements from a token to the next (a multiple of 8; heads are contiguous);
 * out: bf16 [n_tokens][n_q_heads][head_dim], contiguous; lse: fp32
 * [n_tokens][n_q_heads] or NULL, the natural logarithm of the softmax sum.  Both
 * q and out 16-byte aligned; q, out and lse do not overlap.  A token that sees no key (T > L) gets zeros and
 * lse -inf; rows behind the last sequence's tokens are not written.
 *
 * Only positions below a sequence's length are read, and their K and V have to
 * be finite; page entries and contents behind it do not matter.  A sequence of
 * length 0 or without query tokens reads nothing.  What the others of a group
 * share is read through the first one's table row: the whole pages of the
 * prefix, as far as the shortest of them fills them.  Their rows have to name
 * the same pages there.  Softmax in fp32;
 * the probabilities enter the product with V as two bf16 parts, good to 2^-17,
 * and the result is rounded to bf16.  The same call gives the same bits.  A call whose query tokens times
 * table width are beyond what 32 bits of work items hold (2^20 tokens over
 * millions of keys) is MK_ERR_UNSUPPORTED.
 *
 * A wrong DEVICE argument (offsets, lengths or starts that are out of order or
 * out of range: nothing is written; a page id out of range: that page's keys
 * are undefined) is reported by mk_attn_sync, once. */
mk_status mk_prefix_attention(mk_attn *attn, int32_t layer, const mk_attn_batch *batch,
                              const void *q, int64_t q_token_stride, void *out, float *lse);

/* Waits for the stream and returns the first device error since the last
 * mk_attn_sync (MK_OK if none); clears it.  MK_ERR_INVALID_ARG while the stream
 * is being captured.  Besides the errors of mk_prefix_attention there is
 * MK_ERR_DEVICE_TIMEOUT: a wait inside a kernel ran out of time, and that call's
 * results are undefined; later calls are not touched by it. */
mk_status mk_attn_sync(mk_attn *attn);

/* How long a wait inside a kernel lasts before the call is given up
 * (MK_ERR_DEVICE_TIMEOUT), in nanoseconds; 2e9 unless set.  For the calls behind
 * this one; a captured call keeps the limit that it was captured with. */
mk_status mk_attn_set_wait_limit_ns(mk_attn *attn, uint64_t ns);

/* Test only: in the next call every SM waits for something that never comes, so
 * that the way out of such a wait can be tested without a hang. */
mk_status mk_attn_debug_poison_wait(mk_attn *attn);

#ifdef __cplusplus
}
#endif

#endif /* MK_CACHE_H */
