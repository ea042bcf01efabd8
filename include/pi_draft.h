/*
 * pi_draft.h — C ABI of the operators of libpi.so that a decode loop needs to
 * check several drafted tokens per slot in one step, and to draw tokens.  With
 * the cache of pi_serve.h:
 *
 *   pi_cache_fork      the slots grow by their drafts
 *   per layer: pi_tree_attention (the drafts' keys and values in, attention
 *              out), pi_layer_decode (pi.h)
 *   pi_token_sample    every draft's logits -> the token that follows it (or
 *                      pi_token_logprobs: the most likely one)
 *   pi_tree_accept     the drafts that those confirm stay in the cache
 *
 * pi_token_sample serves a loop of single tokens too.  The conventions, the
 * cache and its limits are those of pi_serve.h.
 */
#ifndef PI_DRAFT_H
#define PI_DRAFT_H

#include "pi_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PI_TREE_MAX 64

/* Bytes of workspace of pi_tree_attention; 0 for invalid sizes.  Host-only.  The
 * size goes by head_dim alone: a workspace serves any slots, heads and drafts.  One
 * buffer of the largest size may serve every call of pi_serve.h and of this header
 * on its stream. */
size_t pi_tree_workspace_size(const pi_cache_desc* cache, int32_t slots, int32_t heads,
                              int32_t drafts);

/* Attention of several drafted tokens per slot over its cache, in one pass over
 * it.  The drafts of a slot form trees: parent[s][i] is -1 (it follows the
 * tokens before the drafts) or an earlier draft; parent NULL means a chain
 * (i - 1), such as a piece of a prompt.  Slot s has count[s] drafts (count NULL:
 * all `drafts`, 1..PI_TREE_MAX), 0 <= count[s] <= min(drafts, len[s]).  Its
 * length counts them: with base = len[s] - count[s], draft i is stored as token
 * base + i.  Its depth is the number of its ancestors among the drafts, its
 * position base + depth.  With g = h / (heads / kv_heads), draft i sees
 *     V = the tokens before base, its ancestors among the drafts and itself,
 *         of these the ones at a position p with window == 0, or
 *         p > position - window, or p < sinks;
 *     a_t = scale q[s][i][h] . K[t][g]
 *     y[s][i][h] = sum_V exp(a_t) V[t][g] / sum_V exp(a_t),
 *     lse[s][i][h] = log sum_V exp(a_t).
 *   q [slots][drafts][heads][head_dim] fp32; y the same shape, fp32, in another
 *   buffer; lse NULL or [slots][drafts][heads] fp32.  Rows of drafts from count[s]
 *   on are neither read nor written.
 *   k_new, v_new: NULL (the drafts' rows are in the cache already), or both
 *   [slots][drafts][kv_heads][head_dim] fp32: rows are rounded to the cache's
 *   type, stored at the drafts' places in `layer`, and attended to as stored.
 *   The pages of those places must be the slot's alone (pi_cache_fork sees to it).
 * Precision, infinite operands, rows that are not visible and timeouts are as
 * in pi_paged_attention (PI_BF16: rows of q whose elements are all below 2^-110 keep
 * fewer bits).  A page number out of range hides its tokens (drafts given by k_new
 * are seen, but not stored), a parent out of range counts as -1, a
 * length or count out of range as no drafts; all write PI_ERR_INDEX to
 * *dev_status.  For the same lengths, counts and sizes results are the same bit
 * for bit. */
pi_status pi_tree_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                            int32_t heads, int32_t max_pages, int32_t drafts,
                            const int32_t* parent, const int32_t* count, const float* q,
                            const float* k_new, const float* v_new, const int32_t* table,
                            const int32_t* len, void* pool, float scale, int32_t window,
                            int32_t sinks, float* y, float* lse, int32_t* dev_status, void* ws,
                            size_t ws_bytes, pi_stream stream);

/* Diagnostic of that call's failure path: pi_tree_attention (scale 1, chains, no
 * window, no new rows) on a cache with head_dim >= 64 and page_tokens a multiple
 * of 8, except that one more copy of keys is awaited, never ordered, so the waits for it
 * run out after limit_ns nanoseconds (1e3 .. 5e9).  The block lets its copies and
 * products under way end (2 s at most) and leaves, and PI_ERR_TIMEOUT lands in
 * *dev_status; y is not meaningful.  Slot 0 must have a token before its drafts.
 * Returns PI_OK when the launch was issued. */
pi_status pi_selftest_tree_timeout(const pi_cache_desc* cache, int32_t slots, int32_t heads,
                                   int32_t max_pages, int32_t drafts, const float* q,
                                   const int32_t* table, const int32_t* len, void* pool, float* y,
                                   int32_t* dev_status, void* ws, size_t ws_bytes,
                                   int64_t limit_ns, pi_stream stream);

/* Keeps the drafts that the chosen tokens confirm.  tokens[s][i] is draft i's
 * token, choice[s][i] the token chosen to follow it (from its logits; negative:
 * none).  Draft 0 is the tree's root, itself chosen before: it is taken.  From a
 * draft that is taken, its child whose token is the one chosen there is taken
 * next (the lowest of several), until there is none.  parent and count as in
 * pi_tree_attention; trees of other drafts without a parent are not taken.
 *   path [slots][drafts]: the drafts taken, in order, then -1
 *   accepted [slots]: their number; 0 for a slot without drafts
 *   next [slots]: the token chosen at the last of them, -1 without drafts
 *   len_out [slots]: len[s] - count[s] + accepted[s]
 * The j-th draft taken moves to token base + j of its slot in all layers of
 * `pool` (NULL: nothing moves); rows past len_out are left as they are.
 * pi_cache_fork then trims the slots and grows them for the next drafts.  The
 * outputs must be other buffers than the inputs.  A page out of range is not
 * followed (the row does not move), a parent out of range counts as -1, a slot
 * whose length or count is out of range has no drafts and the length 0; all write
 * PI_ERR_INDEX to *dev_status. */
pi_status pi_tree_accept(const pi_cache_desc* cache, int32_t slots, int32_t max_pages,
                         int32_t drafts, const int32_t* parent, const int32_t* count,
                         const int32_t* tokens, const int32_t* choice, const int32_t* table,
                         const int32_t* len, void* pool, int32_t* len_out, int32_t* path,
                         int32_t* accepted, int32_t* next, int32_t* dev_status, pi_stream stream);

/* Bytes of workspace of pi_token_sample; 0 for invalid sizes.  Host-only.  The call
 * checks its workspace but does not write it at present: a row's sums stay on the
 * SMs. */
size_t pi_sample_workspace_size(int32_t rows, int32_t vocab);

/* Draws a token per row of logits x (layout, dtype and alignment as in
 * pi_token_logprobs) with the random number u[r] in [0, 1).  Tokens are ordered
 * by descending logit, equal ones by ascending index, and the filters keep the
 * first ones of that order:
 *     w_i = exp((x_i - max x) / temperature[r])
 *     1. at most top_k[r] tokens (<= 0: no limit) of those with w_i > 0 and
 *        w_i >= min_p[r],
 *     2. of these the fewest whose w sum to top_p[r] times the sum of all of
 *        these or more (top_p >= 1: all); never less than one;
 *     token[r] = the first whose running sum of w exceeds u[r] times the sum of
 *        those kept;  logprob[r] = log(w / that sum).
 * temperature 0 takes the largest (logprob 0).  temperature [rows] fp32 or NULL
 * (1), top_k [rows] int32 or NULL, top_p and min_p [rows] fp32 or NULL (off), u
 * [rows] fp32; logprob may be NULL.  Sums are exact to 2^-35 of each weight, whatever
 * the vocabulary: the token is that of exact sums where the draw and the end of what
 * top-p keeps are further than 2^-34 of the sum from the next one's border.  A row
 * whose logits are all -infinity, or hold a NaN or +infinity, gives token -1 and
 * logprob NaN; so does one whose temperature is negative, infinite or NaN, whose u is
 * outside [0, 1), or whose top_p or min_p is NaN or negative or min_p above 1; all
 * write PI_ERR_RANGE to *dev_status.  Weights below 2^-64 count as 0, temperatures
 * below 1e-30 as 1e-30.  rows >= 0, vocab 1..1 << 24. */
pi_status pi_token_sample(const void* logits, int32_t dtype, int32_t rows, int32_t vocab,
                          int64_t stride, const float* temperature, const int32_t* top_k,
                          const float* top_p, const float* min_p, const float* u, int32_t* token,
                          float* logprob, int32_t* dev_status, void* ws, size_t ws_bytes,
                          pi_stream stream);

#ifdef __cplusplus
}
#endif
#endif
