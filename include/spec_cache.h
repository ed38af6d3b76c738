/*
 * spec_cache.h -- C ABI of the paged key/value cache around the verify step of speculative
 * decoding, on GB300 (sm_103a): the attention whose output becomes the target logits that
 * spec_reject.h verifies, and the cache's bookkeeping before and after it.
 *
 * One step of a serving loop, for the requests 0 .. B-1 of a batch:
 *   spec_cache_reserve   pages for the step's new tokens (a page shared with another request is
 *                        copied before it is written)
 *   per layer: spec_cache_append (the new tokens' keys and values into the pages), then
 *              spec_attention (the new tokens over their cached context)
 *   spec_reject_sample / spec_tree_verify_greedy on the logits
 *   spec_cache_commit    the accepted tokens stay: the length advances by accepted + 1; a tree's
 *                        accepted path, scattered over the step's rows, is moved together
 *   spec_cache_release   (when wanted) pages behind the committed tokens, or of finished requests
 * and spec_cache_fork makes a request that shares another's committed tokens.  In place of the two calls per layer:
 * spec_cache_append_rotated turns keys and queries by their positions on the way; spec_attention_window sees the last
 * positions and the first ones only; spec_attention_shared reads the pages that several requests share once for all
 * (spec_cache_share finds them).
 *
 * The rollback of rejected drafts ("第12章 投机解码：以小博大" §12.3.4: the next step starts
 * accepted + 1 positions further) is the commit: rows of rejected tokens lie behind the committed
 * length and are overwritten by the next step.
 *
 * A request's tokens: lens[r] committed ones at positions 0 .. lens[r] - 1, then the step's
 * n_r = cu_new[r + 1] - cu_new[r] new ones (0 <= n_r; the token that the last step produced and
 * its drafts, the nodes of a draft tree with the root first, or a chunk of a prompt) at positions
 * lens[r] .. lens[r] + n_r - 1.  Row cu_new[r] + i of a step's arrays belongs to new token i of
 * request r: k_r drafts are k_r + 1 new tokens, the target rows of spec_reject_sample, the nodes
 * of spec_tree_verify_greedy.  cu_new[0] = 0, and cu_new[B] may be below the arrays' N rows: rows
 * from cu_new[B] on are padding and are neither used nor written (attention may read queries there, the
 * appends read nothing).
 *
 * Conventions beyond those of spec_reject.h (ownership, asynchrony, host-visible errors, pending
 * CUDA errors):
 *   - The device that owns the cache's memory is current.
 *   - Calls that change a cache (reserve, append, commit, fork, release) are ordered by the
 *     caller: they run on one stream, or behind one another by events (append_rotated and share among
 *     them).  Attention only reads, in each of its three forms; calls
 *     may run at the same time on several streams, each with a workspace of its own; host threads that
 *     call it on one stream share a workspace only behind a lock (a call launches two kernels).
 *     Appends of different layers may run at the same time.
 *   - Every call can be captured into a CUDA graph.  All device data (tables, lengths, cu_new) are
 *     read when the graph runs; sizes, pointers and strides are those of the capture.  Two graphs
 *     that can run at the same time need attention workspaces of their own.
 *   - Errors in device data are collected in the cache's error word (SPEC_DEVERR_* bits, the
 *     lowest request concerned), which stays set until spec_cache_error() clears it.  A request
 *     with an error is skipped by the call that finds it; a cu_new that does not start at 0 or
 *     decreases (or passes N) makes the whole call do nothing.  No kernel traps or asserts.
 *   - Identical inputs give bit-identical outputs.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_reject.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the cache's error word, beside SPEC_DEVERR_LAYOUT (cu_new), _TREE (a parent outside
 * [0, i), a root's parent not -1, more than SPEC_CACHE_MAX_TREE nodes, a path that is not
 * accepted + 1 nodes long) and _TIMEOUT of spec_reject.h. */
#define SPEC_DEVERR_PAGE 32     /* a page id outside [0, num_pages), a page written that is not the
                                   request's alone, a page released more often than it is held */
#define SPEC_DEVERR_CAPACITY 64 /* reserve: the free pages do not suffice */
#define SPEC_DEVERR_LENGTH 128  /* a negative length; more tokens than max_pages pages (reserve, append)
                                   or the pages held (attention, commit, fork) contain, so also a step
                                   whose reserve found no room; an accepted count outside [-1, n_r);
                                   attention: more work than it can number (see there) */
#define SPEC_DEVERR_FORK 256    /* a fork's source or destination out of range, a destination that
                                   holds pages, is named twice or is also a source */

/* Largest draft tree (nodes of one request, the root included). */
#define SPEC_CACHE_MAX_TREE 128
/* Largest head dimension of spec_attention(), spec_attention_window() and spec_attention_shared(). */
#define SPEC_ATTENTION_MAX_HEAD_DIM 128
/* Largest head dimension of spec_cache_append_rotated(). */
#define SPEC_ROTATION_MAX_HEAD_DIM 256

/*
 * A cache.  Keys and values are num_layers x num_pages pages of page_size tokens of num_kv_heads
 * rows of head_dim elements, at the strides given (in elements, the same for k and v; element
 * (layer, page, token, head, i) at layer * layer_stride + page * page_stride + token *
 * token_stride + head * head_stride + i).  k and v are 16-byte aligned and the strides are
 * positive multiples of 8 elements (the stride of a dimension of size 1 is not looked at); max_pages
 * * page_size and page_size * num_kv_heads * head_dim / 8 are below 2^30 (SPEC_ERR_UNSUPPORTED
 * otherwise).  All pointers are device memory of the caller's; the struct itself is read during the call only.
 */
typedef struct spec_cache {
    void *k, *v;
    int32_t dtype;         /* spec_dtype: SPEC_BF16 or SPEC_F16 */
    int32_t num_layers, num_pages, page_size, num_kv_heads;
    int32_t head_dim;      /* a multiple of 8, at most 1024 */
    int64_t layer_stride, page_stride, token_stride, head_stride;
    int32_t *page_table;   /* [num_requests, max_pages], rows table_stride elements apart: the page
                              of tokens i * page_size .. (i + 1) * page_size - 1 in column i;
                              columns from held[r] on are not used (append and fork may read them,
                              the other calls do not) */
    int64_t table_stride;
    int32_t num_requests, max_pages;
    int32_t *lens;         /* [num_requests] committed tokens */
    int32_t *held;         /* [num_requests] pages held */
    int32_t *ref_counts;   /* [num_pages] requests that hold the page */
    int32_t *free_pages;   /* [num_pages] a stack: entries 0 .. *num_free - 1 are free pages */
    int32_t *num_free;     /* [1] */
    int32_t *error;        /* [2] the error word: bits, lowest request (INT32_MAX = none) */
    void *scratch;         /* spec_cache_scratch_size() bytes, 16-byte aligned; zero at the start */
} spec_cache;

/* Bytes of a cache's scratch (0 for invalid sizes). */
size_t spec_cache_scratch_size(int32_t num_requests, int32_t num_pages);

/* Empties a cache: no request holds tokens or pages, every page is free (page 0 on top of the
 * stack's bottom: pages are handed out from the highest), table entries are -1, the error word is
 * clear, the scratch is zero.  Keys and values are left as they are. */
spec_status spec_cache_init(const spec_cache *cache, void *stream);

/* Reads (and clears) the error word; waits for `stream`.  Returns SPEC_OK or
 * SPEC_ERR_DEVICE_INPUT with *error_bits and *first_bad_request (-1 when no single request is
 * concerned); SPEC_ERR_TIMEOUT when a bounded wait inside a kernel gave up. */
spec_status spec_cache_error(const spec_cache *cache, void *stream, int32_t *error_bits,
                             int32_t *first_bad_request);

/*
 * Room for the step's new tokens: every request with n_r > 0 gets the pages that lens[r] + n_r
 * tokens need and it does not hold yet, from the top of the stack of free pages, in the order of
 * requests and columns.  Where the first new token falls into a page that other requests hold too,
 * the request gets a copy first (its committed rows, in every layer) and the old page's count goes
 * down; of several requests that write to one page and are its only holders, the last keeps it.
 * When the free pages do not suffice nothing is changed (SPEC_DEVERR_CAPACITY, with the first
 * request that finds none); a request that would pass max_pages is skipped
 * (SPEC_DEVERR_LENGTH).  Pages reserved and not used (rejected drafts) stay with the request.
 * A step that goes on without its room: append skips the rows (SPEC_DEVERR_PAGE), attention and commit
 * the requests whose pages do not contain the new tokens (SPEC_DEVERR_LENGTH).  Where all that was
 * missing is the copy of a shared page, commit cannot tell: its num_accepted must be -1.
 */
spec_status spec_cache_reserve(const spec_cache *cache, const int32_t *cu_new, int32_t B, void *stream);

/*
 * The keys and values of the new tokens into the pages of one layer.
 *   k_new, v_new  device, [N, num_kv_heads, head_dim] of the cache's type: rows token_stride and
 *                 heads head_stride elements apart, unit stride inside (strides multiples of 8
 *                 elements, pointers 16-byte aligned; k_new and v_new each with their own strides)
 * Rows are written only to pages that their request alone holds (see spec_cache_reserve); other
 * rows are skipped (SPEC_DEVERR_PAGE).  lens does not change.
 */
spec_status spec_cache_append(const spec_cache *cache, int32_t layer, const void *k_new, int64_t k_token_stride,
                              int64_t k_head_stride, const void *v_new, int64_t v_token_stride,
                              int64_t v_head_stride, const int32_t *cu_new, int32_t B, int64_t N, void *stream);

/*
 * The rotation of positions: the first `dim` elements of a head form dim / 2 pairs, elements i and dim / 2 + i
 * (neighbours == 0) or 2 i and 2 i + 1; at position p a pair (a, b) becomes
 *   (a cos - b sin, b cos + a sin),  cos = table[p * row_stride + i], sin = table[p * row_stride + dim / 2 + i]
 * and the elements behind stay as they are.
 *   table       device fp32, 16-byte aligned, `positions` rows row_stride elements apart (>= dim and a multiple of
 *               4; not looked at for one row)
 *   dim         even, at most head_dim; a multiple of 16, or of 8 with neighbours (SPEC_ERR_UNSUPPORTED otherwise)
 */
typedef struct spec_rotation {
    const float *table;
    int64_t row_stride;
    int32_t positions, dim, neighbours;
} spec_rotation;

/*
 * spec_cache_append() with the keys turned by their positions on the way, and the queries of the same tokens: new
 * token i of request r stands at position lens[r] + i (parent == NULL) or, as node i of a tree (parent given,
 * spec_tree_verify_greedy's), at lens[r] + its depth, where a commit moves it.  Its key and value are written to
 * place lens[r] + i.  Computed in fp32, rounded to the cache's type once.
 *   q, q_out  device, [N, num_q_heads, head_dim] of the cache's type, strides as for spec_cache_append(); q_out may
 *             be q (with its strides); num_q_heads == 0: keys and values alone
 * The positions lens[r] .. lens[r] + n_r - 1 lie in the table (SPEC_DEVERR_LENGTH otherwise, and the request is
 * skipped, as it is with a malformed tree or one of more than SPEC_CACHE_MAX_TREE nodes, SPEC_DEVERR_TREE).  A row that
 * spec_cache_append() would skip is skipped in q_out too.  head_dim is at most SPEC_ROTATION_MAX_HEAD_DIM
 * (SPEC_ERR_UNSUPPORTED otherwise).  `rotation` is read during the call only.
 */
spec_status spec_cache_append_rotated(const spec_cache *cache, int32_t layer, const void *k_new,
                                      int64_t k_token_stride, int64_t k_head_stride, const void *v_new,
                                      int64_t v_token_stride, int64_t v_head_stride, const void *q,
                                      int64_t q_token_stride, int64_t q_head_stride, int32_t num_q_heads, void *q_out,
                                      int64_t out_token_stride, int64_t out_head_stride, const int32_t *cu_new,
                                      int32_t B, int64_t N, const int32_t *parent, const spec_rotation *rotation,
                                      void *stream);

/*
 * The step's outcome: lens[r] advances by num_accepted[r] + 1 where n_r > 0 and num_accepted[r] >=
 * 0 (-1, a request reported invalid, commits nothing), and where the pages held contain the step's
 * tokens (SPEC_DEVERR_LENGTH otherwise, and the length stays).  With a tree, the accepted path from
 * the root to last_node[r] (num_accepted[r] + 1 nodes) is moved, in every layer, to positions
 * lens[r] + depth; rows that already lie there stay.
 *   parent, last_node  device int32 [N] and [B], as spec_tree_verify_greedy() takes and returns
 *                      them; both NULL for chains
 *   num_accepted       device int32 [B], as the sampler and the tree verification return it
 *   out_lens           device int32 [B] that receives the new lengths; NULL or cache->lens to
 *                      advance the cache's own
 */
spec_status spec_cache_commit(const spec_cache *cache, const int32_t *cu_new, int32_t B, int64_t N,
                              const int32_t *num_accepted, const int32_t *parent, const int32_t *last_node,
                              int32_t *out_lens, void *stream);

/*
 * `num_forks` requests made from others: request dst[f] gets the committed tokens of src[f] by
 * holding the same pages (each page's count goes up by one; nothing is copied before
 * spec_cache_reserve finds a shared page that would be written).  A destination holds no pages
 * before; sources may repeat, destinations may not.
 */
spec_status spec_cache_fork(const spec_cache *cache, const int32_t *src, const int32_t *dst, int32_t num_forks,
                            void *stream);

/*
 * Truncates the requests 0 .. B-1 to keep_lens[r] tokens (device int32 [B]; NULL keeps the
 * committed ones; a longer value changes no length) and gives back the pages behind them: counts
 * go down, table entries become -1, and pages that no request holds any more are put on the stack
 * of free pages in ascending order.  keep_lens[r] = 0 frees a request.
 */
spec_status spec_cache_release(const spec_cache *cache, const int32_t *keep_lens, int32_t B, void *stream);

/*
 * Attention of the new tokens over the cache.  Row cu_new[r] + i of q, head h, sees the keys of kv
 * head h / (num_q_heads / num_kv_heads) at the committed positions 0 .. lens[r] - 1 and at those
 * of the new tokens j <= i (parent == NULL), or of node i and its ancestors (parent given):
 *   out = sum_t p_t v_t,  p = softmax over the visible t of scale * (q . k_t)
 *   lse = log sum_t exp(scale * (q . k_t))
 * Products of the cache's 16-bit values are summed in fp32; the maximum, the sum and the output's
 * accumulator are fp32; p is rounded to the cache's type once before its product with v (its sum
 * is not; fp16 holds p / p_max * 2^7 or more: in full from 2^-21 of the largest on, in multiples of
 * 2^-31 of it below), the output once at the end.
 *   q, out        device, [N, num_q_heads, head_dim] of the cache's type, strides as for
 *                 spec_cache_append; num_q_heads a multiple of num_kv_heads, at most 128 times
 *   parent        device int32 [N] (spec_tree_verify_greedy's), or NULL
 *   scale         finite, > 0
 *   lse           device fp32 [N, num_q_heads], or NULL
 *   workspace     spec_attention_workspace_size() bytes; contents need no initialisation
 * Scores scale * (q . k_t) are held in fp32; finite results are certain for scores below 1.8e8 (fp16)
 * and 1.4e9 (bf16) in size, where a step of fp32 is a factor of 2^16 and 2^128 between weights.
 * page_size is a multiple of 8, head_dim at most SPEC_ATTENTION_MAX_HEAD_DIM and N * num_q_heads
 * below 2^30 (SPEC_ERR_UNSUPPORTED otherwise).  The keys and values of all lens[r] + n_r tokens are
 * read, from the pages held (SPEC_DEVERR_LENGTH where those contain fewer); rows behind them are not
 * used whatever they hold.  A key or value that is not finite reaches the rows that see it and no
 * others.  A page id out of range reads as zeros (SPEC_DEVERR_PAGE); the rows of other requests with
 * errors are not written.  A request whose work for one kv head is past counting is an error too
 * (SPEC_DEVERR_LENGTH): with R blocks of 256 query rows and K = lens[r] + n_r keys, where
 * R (4 + K / 128) reaches 2^31.
 */
size_t spec_attention_workspace_size(const spec_cache *cache, int32_t num_q_heads, int32_t B, int64_t N);
spec_status spec_attention(const spec_cache *cache, int32_t layer, const void *q, int64_t q_token_stride,
                           int64_t q_head_stride, int32_t num_q_heads, const int32_t *cu_new, int32_t B, int64_t N,
                           const int32_t *parent, float scale, void *out, int64_t out_token_stride,
                           int64_t out_head_stride, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * spec_attention() of which a row at position p sees only the keys at positions above p - window (its own among
 * them) and those of the first `sinks` positions.  New token i of a chain stands at position lens[r] + i, node i of
 * a tree at lens[r] + its depth.  Keys that no row of a request sees are not read, nor are their table entries.
 *   window  >= 1;  sinks  >= 0
 * Everything else, the workspace too, is as for spec_attention(): all lens[r] + n_r tokens lie in the pages held.
 * Work is past counting where R (19 + 5 (K / 128)) reaches 2^31, of the K keys that a block of query rows can see: at
 * most window + sinks, its own tokens and 256 more.
 */
spec_status spec_attention_window(const spec_cache *cache, int32_t layer, const void *q, int64_t q_token_stride,
                                  int64_t q_head_stride, int32_t num_q_heads, const int32_t *cu_new, int32_t B,
                                  int64_t N, const int32_t *parent, float scale, int32_t window, int32_t sinks,
                                  void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * The plan of spec_attention_shared(): for each of the requests 0 .. B-1 four numbers, the first request of its group
 * and the end (one more than the last), the tokens that all of the group share, and 0.  Two neighbouring requests
 * are linked when their committed tokens begin with the same pages, whole ones, of min_tokens tokens or more (>= 0,
 * and at least one page); a group is a run of links, and shares the tokens of its shortest link.  A request of no link
 * is a group of its own that shares 0 tokens, and so is, with SPEC_DEVERR_LENGTH, one whose pages held do not contain
 * its tokens.
 *   shared  device int32 [B, 4], 16-byte aligned
 * The plan holds for the steps that follow, in every layer, as long as the requests keep their first pages: committed
 * tokens may be added, and a request is planned anew when it was released or truncated.  It may also be written by the
 * caller: groups that do not overlap, `tokens` a multiple of page_size, the same three numbers for every request of a
 * group.
 * Uses the cache's scratch: ordered by the caller like the calls that change a cache.
 */
spec_status spec_cache_share(const spec_cache *cache, int32_t B, int32_t min_tokens, int32_t *shared, void *stream);

/*
 * spec_attention() that reads the tokens which the requests of a group share once for all of them, from the pages of
 * its first request: same results, but for the order of sums.  Entries of the plan that the requests do not fit (a
 * group out of range or of one request, fewer committed tokens than it shares, another entry for its first request)
 * count as no group; whether the pages are in fact the same is not looked at.
 * Work is past counting where R (19 + 5 (K / 128)) reaches 2^31, of the K keys that a request does not share; a group
 * whose own reaches 2^30 shares nothing.
 *   shared     device int32 [B, 4], 16-byte aligned, as spec_cache_share() writes it
 *   workspace  spec_attention_shared_workspace_size() bytes; contents need no initialisation (two sums of every row
 *              and query head beside spec_attention()'s: 553 MB for 16384 rows of 32 heads of 128)
 * After a wait that gave up (SPEC_DEVERR_TIMEOUT) the results count for nothing, as those of the other calls do.
 */
size_t spec_attention_shared_workspace_size(const spec_cache *cache, int32_t num_q_heads, int32_t B, int64_t N);
spec_status spec_attention_shared(const spec_cache *cache, int32_t layer, const void *q, int64_t q_token_stride,
                                  int64_t q_head_stride, int32_t num_q_heads, const int32_t *cu_new, int32_t B,
                                  int64_t N, const int32_t *parent, float scale, const int32_t *shared, void *out,
                                  int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
