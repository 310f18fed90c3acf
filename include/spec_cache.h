/*
 * spec_cache.h -- C ABI of the paged key/value cache and of the attention that
 * reads it, part of libspecverify.so: what stands between a drafted chain or
 * tree and the logits that spec_verify / spec_verify_tree check, and what
 * follows their verdict.
 *
 * One decoding step of a model with L layers:
 *   spec_cache_resize    pages for the drafted tokens;
 *   spec_cache_append    per layer: the keys and values of the tree's nodes,
 *                        node n of request b at position cache_len[b] + n;
 *   spec_tree_attention  per layer: every node attends to the committed
 *                        positions, its ancestors and itself;
 *   spec_verify(_tree)   on the logits: the accepted path;
 *   spec_cache_commit    the accepted nodes moved to follow the root, all layers
 *                        in one launch, and the lengths advanced;
 *   spec_cache_resize    the pages past the new lengths returned.
 *
 * Layout.  The keys and the values of one layer lie in a pool of num_pages
 * pages of page_size tokens, element (page, token, head, d) at
 *   page * page_stride + token * token_stride + head * head_stride + d
 * (strides in elements, multiples of 8; the last dimension is contiguous, so
 * both orders of tokens and heads inside a page are strides).  Position j of
 * slot (request) b lies in page page_table[b, j / page_size] at token
 * j % page_size.  The slots of a batch share the pool; page_ref counts the
 * slots that hold a page, and a page is free when its count is 0.
 *
 * Conventions are those of spec_verify.h: device pointers unless stated
 * otherwise, nothing allocated, nothing synchronised, all work on `stream`;
 * host-detectable errors are returned before anything is launched;
 * data-dependent problems are clamped or skipped and reported in *dev_status.
 * Every call gives bit-identical results for identical inputs.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bits beyond those of spec_verify.h (SPEC_DEV_BAD_LEN: a length
   outside what the slot's pages hold; SPEC_DEV_BAD_TREE: a parent or a path
   that is none). */
#define SPEC_DEV_BAD_PAGE 16u /* a page number outside the pool where one is needed */
#define SPEC_DEV_NO_PAGES 32u /* too few free pages: the requests not served keep what they had */
#define SPEC_DEV_BAD_SLOT 64u /* a fork whose slots are out of range or in use twice */

#define SPEC_DEV_BAD_VALUE 128u /* a key or value that is not finite was written to a 4-bit cache */

#define SPEC_MAX_SLOTS 8192   /* largest number of slots (rows of the page table) */
#define SPEC_MAX_HEAD_DIM 128 /* largest head dimension of spec_tree_attention */

/* A pool of pages: read on the host during the call. */
typedef struct {
    void *k, *v;            /* keys and values, same layout, 16-byte aligned */
    spec_dtype_t dtype;     /* spec_tree_attention: SPEC_DTYPE_BF16 or SPEC_DTYPE_F16 */
    int layers;             /* layers the call works on (1: one layer's pool) */
    int num_pages;
    int page_size;          /* tokens per page: a power of two of at least 8 */
    int heads;              /* key/value heads */
    int head_dim;           /* a multiple of 8 */
    long long layer_stride; /* strides in elements: multiples of 8; where the extent is above 1 a stride steps over
                               head_dim and all that the smaller strides reach, so no two elements share a place */
    long long page_stride;
    long long token_stride;
    long long head_stride;
} spec_pages_t;

/*
 * spec_cache_resize -- pages for the wanted lengths.  Slot b comes to hold
 * ceil((want_len[b] + extra) / page_size) pages, at most max_pages (want_len[b]
 * < 0: the slot keeps what it has).  First every page past that number is given
 * back: its count in page_ref falls by one and its entry becomes -1.  Then the
 * slots that need more take free pages, the lowest-numbered free page first,
 * in the order of the slots.  A slot whose needs, added to those of the
 * slots before it, exceed the free pages takes none (SPEC_DEV_NO_PAGES).
 *   page_table [B, max_pages] int32, page_count [B] int32 (pages held, in front
 *   of the row), page_ref [num_pages] int32: updated.  want_len [B] int32.
 *   want_len = cache_len, extra = 0 trims every slot to its length; extra = N
 *   makes room for N drafted tokens; want_len[b] = 0 frees slot b.
 *   1 <= B <= SPEC_MAX_SLOTS, 1 <= num_pages, 1 <= max_pages, extra >= 0.
 * One launch.
 */
spec_status_t spec_cache_resize(int32_t *page_table, int32_t *page_count, int32_t *page_ref,
                                const int32_t *want_len, int extra, int page_size, int B,
                                int max_pages, int num_pages, uint32_t *dev_status, void *stream);

/*
 * spec_cache_fork -- requests continued in other slots.  Fork f makes slot
 * dst[f] a copy of slot src[f]: the pages dst[f] held are given back, the full
 * pages of src[f] are shared (their counts rise by one), and the last partial
 * page, which both will go on writing, is copied into a page of its own: the
 * tokens it holds, in every layer.  Free pages are taken as by
 * spec_cache_resize, in the order of the forks; a fork that finds none leaves
 * dst[f] empty (SPEC_DEV_NO_PAGES).  Pages that src[f] holds past its length
 * are not shared.  Shared pages are not to be written again: neither slot's length
 * may be taken back behind the fork while the other holds them.
 *   page_table [slots, max_pages], page_count [slots], page_ref [num_pages],
 *   cache_len [slots] int32: updated.  src, dst [F] int32: a slot may be the
 *   source of many forks; a dst that is also a source, or another fork's dst
 *   with a lower index, or a src whose length its pages do not hold, makes the
 *   fork void (SPEC_DEV_BAD_SLOT / SPEC_DEV_BAD_LEN): nothing of it is done.
 *   1 <= F <= SPEC_MAX_SLOTS, 1 <= slots <= SPEC_MAX_SLOTS.  workspace:
 *   spec_cache_fork_workspace_bytes(F) bytes, 256-byte aligned.  Two launches.
 */
size_t spec_cache_fork_workspace_bytes(int F);
spec_status_t spec_cache_fork(const spec_pages_t *pages, int32_t *page_table, int32_t *page_count,
                              int32_t *page_ref, int32_t *cache_len, const int32_t *src,
                              const int32_t *dst, int F, int slots, int max_pages, void *workspace,
                              size_t workspace_bytes, uint32_t *dev_status, void *stream);

/*
 * spec_cache_copy -- whole pages copied in every layer: page dst_pages[i]
 * becomes a copy of page src_pages[i].  No page may be both source and
 * destination, or the destination of two copies.  A pair with a page outside
 * the pool is skipped (SPEC_DEV_BAD_PAGE).  1 <= n.  One launch.
 */
spec_status_t spec_cache_copy(const spec_pages_t *pages, const int32_t *src_pages,
                              const int32_t *dst_pages, int n, uint32_t *dev_status, void *stream);

/*
 * spec_cache_append -- new keys and values written behind the committed
 * positions of one layer (pages->layers = 1): token n of request b, n <
 * count[b], at position cache_len[b] + n.
 *   k_new, v_new  [B, N, heads, head_dim] of the pool's dtype, 16-byte aligned,
 *                 element (b, n, h, d) at b * new_stride_b + n * new_stride_n +
 *                 h * new_stride_h + d (multiples of 8): slices of a fused
 *                 projection need no copy.
 *   count         [B] int32, clamped to [0, N]; NULL: N tokens each.
 * cache_len is not changed.  A position that the slot's row of the table does
 * not reach, or whose page is outside the pool, is skipped (SPEC_DEV_BAD_LEN /
 * SPEC_DEV_BAD_PAGE).  1 <= N, 1 <= B < 2^16.  One launch.
 */
spec_status_t spec_cache_append(const spec_pages_t *pages, const int32_t *page_table,
                                const int32_t *cache_len, const void *k_new, const void *v_new,
                                long long new_stride_b, long long new_stride_n,
                                long long new_stride_h, const int32_t *count, int B, int N,
                                int max_pages, uint32_t *dev_status, void *stream);

/*
 * spec_cache_commit -- the verdict of a step applied to the cache: node
 * out_nodes[b, i] of request b, i < accept_len[b], moves from position
 * cache_len[b] + out_nodes[b, i] to cache_len[b] + 1 + i in every layer (the
 * root, node 0, stays at cache_len[b]), and the length becomes
 *   new_len[b] = cache_len[b] + 1 + accept_len[b].
 *   out_nodes  [B, N] int32, accept_len [B] int32: as spec_verify_tree writes
 *              them.  out_nodes NULL: linear drafts, whose accepted tokens
 *              are in place already: only the lengths change.
 *   new_len    [B] int32: cache_len itself, or a buffer apart from it.
 * accept_len is clamped to [0, N - 1].  A path is cut, the length too, at the
 * first place without a page (SPEC_DEV_BAD_PAGE) and at an out_nodes[b, i]
 * outside [i + 1, N) (SPEC_DEV_BAD_TREE); where the root's place has no page, or
 * cache_len[b] < 0 (SPEC_DEV_BAD_LEN), the length stays as it is.  So a slot
 * that got no pages for its step does not come to count tokens that were never
 * written.  Linear drafts past the end of the table's row, for which no page
 * can ever stand, are counted and reported (SPEC_DEV_BAD_LEN), as every later
 * call on such a length reports them.
 * 1 <= N <= SPEC_MAX_TREE, 1 <= B < 2^16.  One launch, two when new_len is
 * cache_len.
 */
spec_status_t spec_cache_commit(const spec_pages_t *pages, const int32_t *page_table,
                                const int32_t *cache_len, const int32_t *out_nodes,
                                const int32_t *accept_len, int32_t *new_len, int B, int N,
                                int max_pages, uint32_t *dev_status, void *stream);

/*
 * spec_tree_attention -- attention of the nodes of drafted trees over a paged
 * cache (one layer), the target's pass that scores a tree for
 * spec_verify_tree: "speculative decoding от черновика до проверки"
 * (braintools.ru), the Medusa and EAGLE-2 passages: a tree of candidates is
 * checked in one pass with tree attention.
 *   out[b, n, h] = sum_j p_j v_j,  p = softmax_j(scale * q[b, n, h] . k_j)
 * over the positions j that node n sees, k and v of the head h / (Hq / heads):
 *   - the committed positions [0, cache_len[b]);
 *   - the position cache_len[b] + m of every node m on the path from the root
 *     to n, n included (parent[b, n] < n; parent NULL: a chain, every node
 *     under the one before it: the linear drafts of spec_verify, and with
 *     N = 1 plain decoding of one token);
 *   - with window > 0 only those of them less than `window` tokens back along
 *     the path (node n stands at place cache_len[b] + its depth; window = 1
 *     leaves the node itself), or at one of the first `sinks` places.
 *   lse[b, n, h] = log sum_j exp(scale * q . k_j), nullable float32 [B, N, Hq].
 * Rows n >= node_count[b] (node_count [B] int32, nullable: N each) see nothing:
 * out 0, lse -inf.
 *   q    [B, N, Hq, head_dim] of the pool's dtype, 16-byte aligned, element
 *        (b, n, h, d) at b * q_stride_b + n * q_stride_n + h * q_stride_h + d
 *        (multiples of 8, at least head_dim where the extent is above 1).
 *        out [B, N, Hq, head_dim] contiguous, same dtype.
 *   page_table [B, max_pages], cache_len [B]: entries of pages that no node of
 *        the request sees are not looked at.  What the pool holds at positions
 *        that no node sees (past the end, before a window) may be anything,
 *        infinities and NaN included.  At a position that only some nodes see (a
 *        node of another branch, the low end of a window) a key or value that is
 *        not finite shows in the rows of those nodes and in no others.
 *   A parent that is not an earlier node ends the path there (SPEC_DEV_BAD_TREE);
 *   cache_len[b] + node_count[b] beyond what the row of the table reaches, or
 *   beyond 2^31 - 256, is cut (SPEC_DEV_BAD_LEN); a page outside the pool is
 *   read as page 0 (SPEC_DEV_BAD_PAGE; the request's outputs are then
 *   undefined).  A wait inside the kernel that is in vain for about 2 s gives
 *   the call up (SPEC_DEV_TIMEOUT; outputs undefined).
 *   1 <= B < 2^16, 1 <= N <= SPEC_MAX_TREE, head_dim a multiple of 8 up to
 *   SPEC_MAX_HEAD_DIM, Hq a multiple of heads, heads <= 1024, Hq / heads <= 64,
 *   window >= 0, sinks >= 0.  scale > 0, and scale * log2(e) a float32.
 *   workspace: spec_tree_attention_workspace_bytes, 256-byte aligned; nothing
 *   in it is read that the call has not written.  Two launches.
 * Scores, softmax statistics and sums are float32; the softmax weights are
 * rounded to the dtype for the product with v (their sum is not).  A score of
 * -inf beside finite ones has the weight 0.  A row that sees a NaN score or one
 * of +inf, or whose scores are all -inf, comes out NaN, lse included.
 */
size_t spec_tree_attention_workspace_bytes(int B, int N, int Hq, int heads, int head_dim);
spec_status_t spec_tree_attention(const void *q, long long q_stride_b, long long q_stride_n,
                                  long long q_stride_h, const spec_pages_t *pages,
                                  const int32_t *page_table, const int32_t *cache_len,
                                  const int32_t *parent, const int32_t *node_count, int B, int N,
                                  int Hq, int max_pages, float scale, int window, int sinks,
                                  void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  uint32_t *dev_status, void *stream);

/*
 * The 4-bit cache.  Keys and values in 17/64 of their 16-bit size, for a drafter
 * or any model that reads a long cache once per token.  Its pages are taken,
 * returned and listed as those above (spec_cache_resize); every call below is
 * the 4-bit form of the one above it is named after.
 *
 * 32 channels of one token and key head share a scale s = (1 + m/8) 2^(e - 19),
 * kept as the byte 8 e + m (every byte is a finite scale): a seventh of their
 * largest magnitude, rounded to the nearest such number, ties to even.  A
 * number x is kept as the code clamp(rint(x / s), -8, 7) + 8 and stands for
 * (code - 8) s, which bfloat16 and float16 hold exactly.  Whatever bytes a pool
 * holds, the numbers they stand for are finite: a NaN is kept as 0 and an infinity
 * as the largest number of its sign, both reported (SPEC_DEV_BAD_VALUE); magnitudes
 * above 7 * 7680 (8 * 7680 below 0) are kept as that.
 *
 * Layout.  C = head_dim rounded up to 32.  The bytes of one page and head are
 * page_size / T blocks of T = min(page_size, 128) tokens, one after the other,
 * each (t: token of the block)
 *   keys' codes    [T / 8][C / 32][8 tokens][16 bytes]   32 channels of a token
 *   values' codes  [T / 8][C][4 bytes]                   8 tokens of a channel
 *   keys' scales   [C / 32][T]
 *   values' scales [C / 32][T]
 * The eight codes of a 4-byte word (channels or tokens 0 .. 7) lie at its bits
 * 0, 16, 4, 20, 8, 24, 12, 28.
 */
typedef struct {
    void *data; /* 16-byte aligned */
    int layers; /* layers the call works on */
    int num_pages;
    int page_size; /* tokens per page: a power of two of at least 8 */
    int heads;     /* key/value heads */
    int head_dim;  /* a multiple of 8, at most SPEC_MAX_HEAD_DIM */
    long long layer_stride; /* strides in bytes: multiples of 16; where the extent is above 1 a stride steps over */
    long long page_stride;  /* spec_cache4_page_bytes and all that the smaller strides reach */
    long long head_stride;
} spec_pages4_t;

/* Bytes of one page and head: page_size * C * 17 / 16; 0 for sizes that are refused. */
size_t spec_cache4_page_bytes(int page_size, int head_dim);

/*
 * spec_cache4_append -- as spec_cache_append, k_new and v_new of `dtype`
 * (SPEC_DTYPE_BF16 or SPEC_DTYPE_F16) quantised on the way.  Rows of the table
 * must not share the pages that are written.
 */
spec_status_t spec_cache4_append(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *cache_len,
                                 const void *k_new, const void *v_new, spec_dtype_t dtype, long long new_stride_b,
                                 long long new_stride_n, long long new_stride_h, const int32_t *count, int B, int N,
                                 int max_pages, uint32_t *dev_status, void *stream);

/*
 * spec_cache4_read -- the numbers that a 4-bit cache stands for: positions
 * start[b] + n, n < count[b] (NULL: N each), of request b in every layer of the
 * pool, written to k and v [layers, B, N, heads, head_dim] contiguous, 16-byte
 * aligned, of `dtype`.  Rows from count[b] on, positions that the table does
 * not reach (SPEC_DEV_BAD_LEN) and pages outside the pool (SPEC_DEV_BAD_PAGE)
 * give 0.  1 <= B < 2^16, 1 <= N.  One launch.
 */
spec_status_t spec_cache4_read(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *start,
                               const int32_t *count, void *k, void *v, spec_dtype_t dtype, int B, int N,
                               int max_pages, uint32_t *dev_status, void *stream);

/* spec_cache4_commit, spec_cache4_copy, spec_cache4_fork -- as spec_cache_commit,
   spec_cache_copy and spec_cache_fork.  (A fork copies the last partial page whole.) */
spec_status_t spec_cache4_commit(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *cache_len,
                                 const int32_t *out_nodes, const int32_t *accept_len, int32_t *new_len, int B, int N,
                                 int max_pages, uint32_t *dev_status, void *stream);
spec_status_t spec_cache4_copy(const spec_pages4_t *pages, const int32_t *src_pages, const int32_t *dst_pages, int n,
                               uint32_t *dev_status, void *stream);
spec_status_t spec_cache4_fork(const spec_pages4_t *pages, int32_t *page_table, int32_t *page_count,
                               int32_t *page_ref, int32_t *cache_len, const int32_t *src, const int32_t *dst, int F,
                               int slots, int max_pages, void *workspace, size_t workspace_bytes,
                               uint32_t *dev_status, void *stream);

/*
 * spec_tree_attention4 -- spec_tree_attention over a 4-bit cache: q and out of
 * `dtype`, the keys and values the numbers that the codes stand for.
 *   per_head   0: page_table [B, max_pages]; 1: [B, heads, max_pages], a list of
 *              pages for every key head, as spec_page_select writes them.
 *   workspace: spec_tree_attention4_workspace_bytes, 256-byte aligned.
 * In SPEC_DTYPE_F16 four times scale * log2(e) has to be a float32.  The softmax
 * weights are rounded to float16 for the product with v, in either dtype.
 * All else, rows that are empty or not finite included, is as there.
 */
size_t spec_tree_attention4_workspace_bytes(int B, int N, int Hq, int heads, int head_dim);
spec_status_t spec_tree_attention4(const void *q, spec_dtype_t dtype, long long q_stride_b, long long q_stride_n,
                                   long long q_stride_h, const spec_pages4_t *pages, const int32_t *page_table,
                                   int per_head, const int32_t *cache_len, const int32_t *parent,
                                   const int32_t *node_count, int B, int N, int Hq, int max_pages, float scale,
                                   int window, int sinks, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, uint32_t *dev_status, void *stream);

/*
 * Attention over selected pages.  A page's bounds are the smallest and the
 * largest key of each channel over its committed tokens; sum_d max(q_d lo_d, q_d
 * hi_d) is above every q . k of the page, and a score cheap enough to be formed
 * for all pages.  One step of a layer:
 *   spec_cache_bounds     bounds of the pages written since the last step;
 *   spec_page_scores      a score for every page, request and key head;
 *   spec_page_select      the best pages of each, as lists of pages;
 *   spec_sparse_attention (or spec_tree_attention4) over those lists.
 * The drafted nodes' own keys are attended to as always: their pages follow the
 * selected ones.
 */

/*
 * spec_cache_bounds -- for every page that holds one of the positions [start[b],
 * cache_len[b]) (start NULL: 0): over the page's positions before cache_len[b]
 *   bounds[page, h, 0, d] = min k_d,  bounds[page, h, 1, d] = max k_d
 * (a NaN makes both NaN).  pages->layers = 1; its v is not read.
 *   bounds  [num_pages, heads, 2, head_dim] of the pool's dtype (`dtype` for a
 *           4-bit pool), 16-byte aligned.  Other pages keep theirs.
 * start[b] < 0 counts as 0.  Rows that share a page have to agree on its
 * committed positions, as forked requests do on all but their last page; the
 * copied last page of a fork has bounds once a position of it is summarised.
 * Positions that the table does not reach, and pages outside the pool,
 * are skipped (SPEC_DEV_BAD_LEN, SPEC_DEV_BAD_PAGE).  1 <= B < 2^16.
 * SPEC_DTYPE_BF16 and SPEC_DTYPE_F16.  One launch.
 */
spec_status_t spec_cache_bounds(const spec_pages_t *pages, const int32_t *page_table, const int32_t *start,
                                const int32_t *cache_len, void *bounds, int B, int max_pages, uint32_t *dev_status,
                                void *stream);
spec_status_t spec_cache4_bounds(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *start,
                                 const int32_t *cache_len, void *bounds, spec_dtype_t dtype, int B, int max_pages,
                                 uint32_t *dev_status, void *stream);

/*
 * spec_page_scores -- scores[b, h, i], the score of the page at place i of
 * request b's row for key head h: the largest over the nodes n < node_count[b]
 * (NULL: N each) and the query heads of h of
 *   sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d
 * in float32; -inf at places that hold no committed position, or without nodes.  A
 * score that is not a number is written as NaN.
 *   q       [B, N, Hq, head_dim] of `dtype`, strides as for spec_tree_attention.
 *   bounds  [num_pages, heads, 2, head_dim] of `dtype`.
 *   scores  [B, heads, max_pages] float32.
 * A page outside the pool scores -inf (SPEC_DEV_BAD_PAGE).  1 <= B < 2^16, 1 <= N <= SPEC_MAX_TREE, Hq a multiple of
 * heads, Hq / heads <= 64, heads <= 1024, head_dim a multiple of 8 up to SPEC_MAX_HEAD_DIM.
 * One launch.
 */
spec_status_t spec_page_scores(const void *q, spec_dtype_t dtype, long long q_stride_b, long long q_stride_n,
                               long long q_stride_h, const void *bounds, const int32_t *page_table,
                               const int32_t *cache_len, const int32_t *node_count, float *scores, int B, int N,
                               int Hq, int heads, int head_dim, int max_pages, int num_pages, int page_size,
                               uint32_t *dev_status, void *stream);

/*
 * spec_page_select -- for each request and key head, of the n =
 * ceil(cache_len[b] / page_size) pages that hold committed positions, the min(n, keep) that
 * rank highest, in the order of their places: the first `first` and the last
 * `recent` ones before all others, then by score (a NaN before all numbers),
 * equal scores by place, the earlier one first.
 *   scores     [B, heads, max_pages] float32.
 *   out_table  [B, heads, keep + tail] int32, tail = ceil(extra / page_size):
 *              the selected pages, then the `tail` entries that follow the
 *              committed pages in the request's row (those of `extra` drafted tokens; -1 past
 *              its end), then -1.
 *   out_len    [B] int32: the committed positions that the selected pages hold.
 * So a position p >= cache_len[b] of the cache is position p - cache_len[b] +
 * out_len[b] of the lists.  extra is at least the nodes N of the attention over the lists,
 * which finds their keys there; what the lists do not reach it reports (SPEC_DEV_BAD_PAGE, SPEC_DEV_BAD_LEN) and
 * answers as for any such row of a page table.  cache_len[b] outside [0, max_pages * page_size] is
 * cut (SPEC_DEV_BAD_LEN).  1 <= B < 2^16, 1 <= heads <= 1024, first >= 0, recent >= 1,
 * first + recent <= keep, extra >= 0, max_pages <= SPEC_MAX_SELECT.  One launch.
 */
#define SPEC_MAX_SELECT 131072 /* largest row of the page table that spec_page_select takes */
spec_status_t spec_page_select(const float *scores, const int32_t *page_table, const int32_t *cache_len,
                               int32_t *out_table, int32_t *out_len, int B, int heads, int max_pages, int page_size,
                               int keep, int first, int recent, int extra, uint32_t *dev_status, void *stream);

/* spec_sparse_attention -- spec_tree_attention with a list of pages for every key
   head: page_table [B, heads, max_pages], cache_len the positions that each
   list of the request holds.  `window` and `sinks` count positions of the list, as do those of
   spec_tree_attention4 with per_head = 1: neighbours there may lie far apart in the
   sequence, so a window over a selection is not the window's part of it. */
spec_status_t spec_sparse_attention(const void *q, long long q_stride_b, long long q_stride_n, long long q_stride_h,
                                    const spec_pages_t *pages, const int32_t *page_table, const int32_t *cache_len,
                                    const int32_t *parent, const int32_t *node_count, int B, int N, int Hq,
                                    int max_pages, float scale, int window, int sinks, void *out, float *lse,
                                    void *workspace, size_t workspace_bytes, uint32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
