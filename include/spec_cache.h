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
 *   window >= 0, sinks >= 0.  scale > 0.
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

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
