/*
 * mk_rules.h -- C ABI for what stands between the logits of a step and the next
 * tokens: penalties for tokens that were there already, biases, grammar masks,
 * and the greedy token under them.
 *
 * The logits are those of mk_decode_step, or of the tokens of drafted trees.
 * Conventions as in mk_cache.h: mk_status results, nothing throws, caller-owned
 * device memory, work enqueued on the stream given at creation, asynchronous
 * unless stated; a handle's calls belong to one stream, calls that overlap on
 * the GPU take a handle each.  mk_rules_apply can be captured into a CUDA graph.
 */
#ifndef MK_RULES_H
#define MK_RULES_H

#include "mk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What holds for the rows of a call.  The arrays are DEVICE memory, 4-byte aligned, and
 * are read by the call on the GPU, so they can be updated between replays of a captured
 * call.  NULL leaves a rule out (ranges and tokens, path_offsets and path_tokens, and the
 * three of the bias come together). */
typedef struct {
  int32_t n_rows;
  int32_t n_tokens, n_path, n_bias, n_masks; /* entries of the arrays below; the first two at most 2^29 - 1 */
  const int32_t *tokens;       /* [n_tokens] the sequences' tokens */
  const int32_t *ranges;       /* [n_rows][2]: a row's history is tokens[begin .. end - 1]; the
                                * rows of a tree share their sequence's */
  const int32_t *prompt_lens;  /* [n_rows]: the history's first tokens that were not generated, or NULL: 0 */
  const int32_t *path_offsets; /* [n_rows + 1] from 0, not decreasing, into path_tokens: drafted tokens */
  const int32_t *path_tokens;  /* [n_path]  between the history and the row; generated ones */
  const float *repetition, *presence, *frequency; /* [n_rows] each, or NULL: 1, 0, 0 */
  const int32_t *bias_offsets; /* [n_rows + 1] from 0, not decreasing */
  const int32_t *bias_tokens;  /* [n_bias], rising within a row */
  const float *bias;           /* [n_bias] */
  const uint32_t *allowed;     /* [n_masks][(vocab + 31) / 32]: bit t % 32 of word t / 32: token t may follow */
  const int32_t *allowed_rows; /* [n_rows]: a row's mask, negative: all may follow (those of all rows where
                                * n_masks is 0, allowed NULL or not); NULL: mask i of row i */
} mk_rules_batch;

typedef struct mk_rules mk_rules;

/* Allocates the workspace: 8 bytes a row.  vocab and max_rows from 1 to 2^24.
 * MK_ERR_INVALID_ARG / MK_ERR_UNSUPPORTED / MK_ERR_NO_DEVICE / MK_ERR_CUDA. */
mk_status mk_rules_create(int32_t vocab, int32_t max_rows, void *stream, mk_rules **out);
void mk_rules_destroy(mk_rules *rules);

/* For each row and token t, with c times t among the row's generated tokens (history behind
 * the prompt, and path), in this order, each step in fp32 and rounded by itself:
 *   t anywhere in history or path:  x <- x > 0 ? x / repetition : x * repetition
 *   c > 0:                          x <- x - frequency * c, then x <- x - presence
 *   t has a bias:                   x <- x + bias
 *   t may not follow:               x <- -inf
 * logits: DEVICE [n_rows][vocab], fp32 or (is_bf16) bf16, row_stride elements from a row to
 * the next; out: fp32 [n_rows][vocab], contiguous, or NULL; it may be logits itself (fp32,
 * row_stride == vocab) and overlaps them in no other way, nor anything else that the call reads.  out_tokens: int32 [n_rows] or NULL:
 * each row's largest x, ties to the lowest t, NaN never; -1 where none is above -inf.  One of
 * the two is given.  The same call gives the same bits.
 *
 * Ids outside [0, vocab) in histories and paths (padding) count for nothing.  A row with a wrong
 * DEVICE argument (a range, offset or mask out of range, a negative prompt length, a repetition
 * not above 0, bias tokens out of range or not rising) is not written, and reported by
 * mk_rules_sync, once. */
mk_status mk_rules_apply(mk_rules *rules, const mk_rules_batch *batch, const void *logits,
                         int32_t is_bf16, int64_t row_stride, float *out, int32_t *out_tokens);

/* mk_rules_apply behind mk_decode_step on the same stream, in place on its logits; out_tokens is the
 * step's out_next_tokens, in which a row that is refused gets -1 instead of keeping the step's token
 * (its logits stay the step's). */
mk_status mk_rules_follow(mk_rules *rules, const mk_rules_batch *batch, float *logits, int32_t *out_tokens);

/* What mk_rules_apply returns for these arguments before it looks at the device; enqueues nothing.
 * MK_ERR_BATCH for more than max_rows rows, MK_ERR_UNSUPPORTED for more tokens than above. */
mk_status mk_rules_check(const mk_rules *rules, const mk_rules_batch *batch, const void *logits,
                         int32_t is_bf16, int64_t row_stride, const float *out, const int32_t *out_tokens);

/* Waits for the stream and returns the first device error since the last mk_rules_sync
 * (MK_OK if none); clears it.  MK_ERR_INVALID_ARG while the stream is being captured. */
mk_status mk_rules_sync(mk_rules *rules);

#ifdef __cplusplus
}
#endif

#endif /* MK_RULES_H */
