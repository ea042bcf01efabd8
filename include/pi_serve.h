/*
 * pi_serve.h — C ABI of the serving operators of libpi.so: a paged key-value
 * cache with the attention of one new token over it, the page bookkeeping of
 * parallel sampling and beam search, and the scoring of tokens.  They are
 * what a decode loop runs around the sparse FFN of pi.h:
 *
 *   pi_token_logprobs  logits -> log probabilities, entropy, alternatives
 *   pi_cache_fork      the chosen continuations -> tables, lengths, pages
 *   per layer: pi_paged_attention (new keys and values in, attention out),
 *              pi_layer_decode (pi.h)
 *
 * The conventions of pi.h hold: device pointers owned by the caller, 16-byte
 * aligned; no allocation, no host synchronisation; counts stay on the device
 * (a step can be captured in a CUDA graph); host-detected errors are returned
 * before anything is launched; device-detected errors go to *dev_status (an
 * int32 the caller zeroes; the first error wins).  A workspace is zero-filled
 * before its first use, serves one stream at a time, and is left ready for
 * the next call.  Results do not depend on the order in which blocks run.
 *
 * The cache
 * ---------
 *   pool   [layers][pages][2][kv_heads][page_tokens][head_dim]  (dtype)
 *          a page holds page_tokens tokens' keys (0), then values (1), of
 *          every kv head; page p has the same number in every layer
 *   table  [slots][max_pages] int32: table[s][j] is the page of slot s's
 *          tokens [j page_tokens, (j + 1) page_tokens); entries past a
 *          slot's length are not read
 *   len    [slots] int32: tokens in the slot, 0 <= len <= max_pages page_tokens
 * Pages may stand in several slots' tables (shared prompts).
 * Sizes: layers, kv_heads 1..256; head_dim % 8 == 0, 8..256; page_tokens
 * 1..256; pages 1..1 << 26; slots 1..1024; max_pages >= 1 with
 * max_pages page_tokens < 1 << 31.
 */
#ifndef PI_SERVE_H
#define PI_SERVE_H

#include "pi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Logits may also be fp32 (weights and caches are PI_F16 / PI_BF16 only). */
#define PI_F32 2

#define PI_CACHE_MAX_SLOTS 1024
#define PI_TOPK_MAX 32

/* Shape of a cache pool. */
typedef struct {
  int32_t layers;
  int32_t pages;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_tokens;
  int32_t dtype; /* pi_dtype of the pool */
} pi_cache_desc;

/* Bytes of workspace for the calls below on this cache with this many slots
 * and query heads (0 where no attention is run).  0 for invalid sizes.
 * Host-only; no CUDA call. */
size_t pi_cache_workspace_size(const pi_cache_desc* cache, int32_t slots, int32_t heads);

/* Attention of one new token per slot over its cache.  With n = len[s] (the
 * new token included) and g = h / (heads / kv_heads), over the visible tokens
 *     V = { t < n : window == 0 or t >= n - window or t < sinks }
 *     a_t = scale q[s][h] . K[t][g]
 *     y[s][h] = sum_V exp(a_t) V[t][g] / sum_V exp(a_t),
 *     lse[s][h] = log sum_V exp(a_t).
 * An empty slot (n = 0), and scores that are all -infinity, give y = 0 and
 * lse = -infinity.  Rows of a page that are not visible are not used whatever
 * they hold (NaN and infinities too).  Infinite operands of visible rows count
 * as the formulas say: an infinite key's score is +-infinity (NaN where
 * products of both signs or 0 x infinity meet; beside it, elements of q below
 * 2^-96 may count as 0 in PI_BF16), and a score of -infinity weighs nothing; a
 * score of NaN or +infinity makes the head's y and lse NaN.
 * An infinite value makes its element of y infinite, however small the weight
 * (NaN where both signs meet, or where a value that is not finite has the
 * weight 0 of a score of -infinity).
 *   q [slots][heads][head_dim] fp32; y the same shape, fp32; lse NULL or
 *   [slots][heads] fp32; heads a multiple of kv_heads, at most 1024.
 *   k_new, v_new: NULL (the new token is in the cache already), or both
 *   [slots][kv_heads][head_dim] fp32: row s is rounded to the cache's type,
 *   stored as token n - 1 of slot s in `layer`, and attended to as stored.
 *   The page of that token must be the slot's alone (pi_cache_fork sees to
 *   it).
 * The products take the cache's 16-bit rows exactly and q and the softmax
 * weights as sums of 16-bit parts that together keep at least 22 bits; sums
 * and softmax statistics are fp32.  A length outside [0, max_pages
 * page_tokens] counts as 0 and a page number outside [0, pages) hides its
 * tokens; both write PI_ERR_INDEX to *dev_status.  A wait for a tile's copy
 * that runs out (1 s, or PI_WAIT_LIMIT_NS) writes PI_ERR_TIMEOUT; y is then not
 * meaningful and ws must be zero-filled again.  The split of the work over
 * the GPU follows the lengths of all slots, so a slot's result may differ in
 * rounding between batches; for the same lengths it is the same bit for bit. */
pi_status pi_paged_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                             int32_t heads, int32_t max_pages, const float* q,
                             const float* k_new, const float* v_new, const int32_t* table,
                             const int32_t* len, void* pool, float scale, int32_t window,
                             int32_t sinks, float* y, float* lse, int32_t* dev_status, void* ws,
                             size_t ws_bytes, pi_stream stream);

/* Diagnostic of the attention's failure path: pi_paged_attention (scale 1, no
 * window, no new rows) on a PI_F16 cache with head_dim 64 and page_tokens a
 * multiple of 16, except that the copy of block 0's first tile is never
 * ordered, so the wait for it runs out after limit_ns nanoseconds (1e3 ..
 * 5e9).  The warp then lets the copies under way land (2 s at most, which the
 * missing one takes) and leaves, and PI_ERR_TIMEOUT lands in *dev_status; y is
 * not meaningful and ws must be zero-filled again.  Slot 0 must not be empty.
 * Returns PI_OK when the launch was issued. */
pi_status pi_selftest_attention_timeout(const pi_cache_desc* cache, int32_t slots, int32_t heads,
                                        int32_t max_pages, const float* q, const int32_t* table,
                                        const int32_t* len, void* pool, float* y,
                                        int32_t* dev_status, void* ws, size_t ws_bytes,
                                        int64_t limit_ns, pi_stream stream);

/* Stores keys and values of `tokens` tokens (prompts, or one step): token i
 * of k, v [tokens][kv_heads][head_dim] fp32 goes, rounded to the cache's
 * type, to position pos[i] of slot slot[i] in `layer`.  slot[i] = -1 skips
 * the token.  A slot, position or page number out of range is not followed:
 * the token is skipped and PI_ERR_INDEX written to *dev_status.  No two
 * tokens may name the same place.  tokens >= 0. */
pi_status pi_cache_append(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                          int32_t max_pages, int32_t tokens, const int32_t* slot,
                          const int32_t* pos, const float* k, const float* v,
                          const int32_t* table, void* pool, int32_t* dev_status,
                          pi_stream stream);

/* One step of the slots' bookkeeping: reorders, forks, frees, trims and grows
 * them, in one call.  For slot s, p = parent[s]:
 *   p = -1: the slot begins empty; else it continues slot p of table_in /
 *   len_in (several slots may continue one p; slots nobody continues are
 *   freed).  With b = len_in[p] (0 for p = -1):
 *     len[s] = max(0, b + grow[s]);  keep = min(b, len[s]).
 *   The keep / page_tokens full pages are shared with p.  A partly filled
 *   last page stays with the lowest such slot if nothing else refers to it;
 *   every other slot gets a fresh page with its contents in all layers.  The
 *   rest of ceil(len[s] / page_tokens) pages are fresh, contents undefined;
 *   table entries past them are -1.
 * Fresh pages are the pages that nothing refers to after the sharing, lowest
 * number first, handed out in slot order.  If they run out, PI_ERR_CAPACITY
 * is written to *dev_status and the slots that got fewer end at the last
 * token that has a page; so does a slot whose length would pass max_pages
 * page_tokens.
 *   held: NULL or [pages] int32 >= 0, references from outside the slots
 *   (prompts kept for later); ref [pages]: held + the references of `table`.
 *   pool: NULL (tables only) or the pool whose pages are copied.
 *   pairs [slots][2]: (from, to) of each copied page, in slot order;
 *   counts[0] their number, counts[1] the pages with ref > 0.
 * table_in and len_in are read only; table and len must be other buffers.
 * A parent, length or page number out of range is not followed and writes
 * PI_ERR_INDEX: the slot begins empty; a full page's entry becomes -1; a
 * partly filled page is replaced by a fresh one, contents undefined. */
pi_status pi_cache_fork(const pi_cache_desc* cache, int32_t slots, int32_t max_pages,
                        const int32_t* parent, const int32_t* grow, const int32_t* held,
                        const int32_t* table_in, const int32_t* len_in, int32_t* table,
                        int32_t* len, int32_t* ref, void* pool, int32_t* pairs, int32_t* counts,
                        int32_t* dev_status, void* ws, size_t ws_bytes, pi_stream stream);

/* Moves the live pages (referred to by a used table entry, or held) to the
 * front of the pool, so that its end can be given back: with c live pages,
 * those numbered >= c move, in ascending order, to the unused numbers below
 * c, in ascending order, in all layers; the others stay.
 *   map [pages]: a live page's new number, -1 for the others.
 *   table (may be table_in): the mapped tables, -1 past a slot's pages.
 *   ref [pages]: references by new number (held included).
 *   pairs [pages / 2][2]: (from, to) of the moved pages; counts[0] their
 *   number, counts[1] = c.  held, pool as in pi_cache_fork (the caller
 *   follows `map` for what it holds). */
pi_status pi_cache_compact(const pi_cache_desc* cache, int32_t slots, int32_t max_pages,
                           const int32_t* held, const int32_t* table_in, const int32_t* len,
                           int32_t* table, int32_t* ref, int32_t* map, void* pool,
                           int32_t* pairs, int32_t* counts, int32_t* dev_status, void* ws,
                           size_t ws_bytes, pi_stream stream);

/* Copies page pairs[i][0] to page pairs[i][1] in every layer, i < *count
 * (<= cap; the rest is not copied and PI_ERR_CAPACITY written): for further
 * pools that follow the same tables.  No page may be both a source and a
 * target.  A pair out of range is skipped and writes PI_ERR_INDEX. */
pi_status pi_cache_copy(const pi_cache_desc* cache, const int32_t* pairs, const int32_t* count,
                        int32_t cap, void* pool, int32_t* dev_status, pi_stream stream);

/* Bytes of workspace of pi_token_logprobs; 0 for invalid sizes. */
size_t pi_logprob_workspace_size(int32_t rows, int32_t vocab, int32_t topk);

/* Scores tokens from logits x [rows] of `vocab` values, row r at
 * logits + r stride (elements; stride >= vocab; rows may begin anywhere, the
 * pointers passed are 16-byte aligned like all: a shifted view such as
 * tokens[1:] is copied first), dtype PI_F16, PI_BF16 or PI_F32.  With z = log sum exp(x):
 *     logprob[r] = x[tokens[r]] - z      (0 where tokens[r] = -1)
 *     entropy[r] = z - sum_i p_i x_i,  p_i = exp(x_i - z)  (p_i = 0: nothing)
 *     top_idx[r][j], top_logprob[r][j]: the topk largest logits in descending
 *     order, equal logits by ascending index; topk <= min(vocab, 32).
 * tokens and logprob may both be NULL, entropy may be NULL, top_idx and
 * top_logprob are not touched for topk = 0.  Logits of -infinity (banned
 * tokens) have probability 0.  A row of nothing but -infinity has entropy 0
 * and log probabilities -infinity; a NaN or +infinity in a row makes its
 * figures NaN (its top_idx ranks NaN below everything).  A token outside
 * [-1, vocab) gives NaN and PI_ERR_INDEX on *dev_status.  Sums are fp32.
 * rows >= 0, vocab 1..1 << 24. */
pi_status pi_token_logprobs(const void* logits, int32_t dtype, int32_t rows, int32_t vocab,
                            int64_t stride, const int32_t* tokens, int32_t topk, float* logprob,
                            float* entropy, int32_t* top_idx, float* top_logprob,
                            int32_t* dev_status, void* ws, size_t ws_bytes, pi_stream stream);

#ifdef __cplusplus
}
#endif
#endif
