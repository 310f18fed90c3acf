// spec_cache.cu -- the pages of the paged key/value cache: taking and returning
// them, forking requests, copying pages, writing new keys and values, and
// compacting accepted paths.
//
// Page bookkeeping runs in one thread-block cluster (sv_pages): the free pages
// are those whose count is 0, so the state is the counts alone, returning a
// page is one atomic decrement, and "the lowest free pages first" makes the
// result independent of the order in which the atomics land.  The data movers
// treat keys and values as 16-byte vectors: a thread owns one vector column
// (head, part of the head) of a token and walks tokens, so its address
// arithmetic is one multiply-add per vector.
#include <cooperative_groups.h>

#include <climits>

#include "spec_cache.h"
#include "sv_cache.cuh"

namespace sv {

namespace cg = cooperative_groups;

constexpr int kPgCtas = 8;       // CTAs of the bookkeeping cluster
constexpr int kPgThreads = 1024; // threads of each
constexpr int kPgWarps = kPgThreads / 32;

// Saturating sum of page counts: anything above the pool's size is as good as
// cap = num_pages + 1 (nothing that large is ever served), and sums capped this
// way stay associative and within 32 bits.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap) {
    return min(a + b, cap);
}

__device__ __forceinline__ int pages_for(long long tokens, int shift, int max_pages) {
    const long long p = (tokens + (1ll << shift) - 1) >> shift;
    return (int)(p < max_pages ? p : max_pages);
}

// Gives back page p (one holder less).
__device__ __forceinline__ void drop_page(const PagesArgs &A, int p) {
    if ((unsigned)p >= (unsigned)A.num_pages) {
        flag(A.status, SPEC_DEV_BAD_PAGE);
    } else if (atomicSub(A.ref + p, 1) <= 0) {  // nobody held it: undo
        atomicAdd(A.ref + p, 1);
        flag(A.status, SPEC_DEV_BAD_PAGE);
    }
}

// What the bookkeeping knows of an item, kept in shared memory by every CTA.
template <bool FORK> struct PagesItem;
template <> struct PagesItem<false> {
    int held, need;          // pages held and wanted
};
template <> struct PagesItem<true> {
    int src, dst, len, kind; // kind: 0 void, 1 valid without a partial page, 2 with one
};

// The bookkeeping of spec_cache_resize (FORK false: item i is slot i) and of
// spec_cache_fork (FORK true: item i is fork i).  Bound by latency: a few
// dependent loads, one cluster barrier (two where pages are taken), and a scan
// of the counts split over the cluster's 256 warps.  8 CTAs of one cluster
// instead of one CTA: 2^16 pages are one load round per warp; instead of a
// whole grid: no launch between the phases.  Two resizes and an append of 72
// tokens: 9.9 us (12.3 with three barriers each and the counts read again).  Two
// resizes of 8, 256 and 1024 slots: 8.3, 9.7 and 16.8 us (one CTA: 8.0, 17.1 and 48.1).
template <bool FORK>
__global__ void __cluster_dims__(kPgCtas, 1, 1) __launch_bounds__(kPgThreads, 1) sv_pages(PagesArgs A) {
    constexpr int kWarps = kPgCtas * kPgWarps;
    extern __shared__ uint4 pg_smem[];
    using Item = PagesItem<FORK>;
    Item *items = reinterpret_cast<Item *>(pg_smem);             // [n]
    uint32_t *incl = reinterpret_cast<uint32_t *>(items + A.n);  // [n] running sum of the pages wanted
    int *owner = reinterpret_cast<int *>(incl + A.n);            // FORK: [slots] first fork into a slot
    __shared__ uint32_t warp_sum[kPgWarps], cta_free[kPgCtas], is_src[SPEC_MAX_SLOTS / 32];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gwarp = rank * kPgWarps + warp;
    const uint32_t cap = (uint32_t)A.num_pages + 1u;
    const int page = 1 << A.page_shift;
    pdl_trigger();
    pdl_wait();

    // ---- what every item wants (each CTA forms all of them)
    if constexpr (FORK) {
        for (int i = tid; i < A.slots; i += kPgThreads) owner[i] = INT_MAX;
        for (int i = tid; i < (A.slots + 31) / 32; i += kPgThreads) is_src[i] = 0;
        __syncthreads();
        for (int f = tid; f < A.n; f += kPgThreads) {
            const int s = A.src[f], d = A.dst[f];
            items[f].src = s;
            items[f].dst = d;
            if ((unsigned)s < (unsigned)A.slots) atomicOr(&is_src[s >> 5], 1u << (s & 31));
            if ((unsigned)d < (unsigned)A.slots) atomicMin(&owner[d], f);
        }
        __syncthreads();
        for (int f = tid; f < A.n; f += kPgThreads) {
            const int s = items[f].src, d = items[f].dst;
            int n = 0, kind = 0;
            if ((unsigned)s >= (unsigned)A.slots || (unsigned)d >= (unsigned)A.slots || owner[d] != f ||
                ((is_src[d >> 5] >> (d & 31)) & 1u)) {
                if (rank == 0) flag(A.status, SPEC_DEV_BAD_SLOT);
            } else {
                n = A.len[s];
                if (n < 0 || (n + (long long)page - 1) >> A.page_shift > min(A.count[s], A.max_pages)) {
                    if (rank == 0) flag(A.status, SPEC_DEV_BAD_LEN);
                } else {
                    kind = (n & (page - 1)) ? 2 : 1;
                }
            }
            items[f].len = n;
            items[f].kind = kind;
            incl[f] = kind == 2 ? 1u : 0u;
        }
    } else {
        for (int i = tid; i < A.n; i += kPgThreads) {
            const int w = A.want[i], c = max(0, min(A.count[i], A.max_pages));
            const int need = w < 0 ? c : pages_for((long long)w + A.extra, A.page_shift, A.max_pages);
            items[i].held = c;
            items[i].need = need;
            incl[i] = min((uint32_t)max(0, need - c), cap);
        }
    }
    __syncthreads();
    {  // inclusive scan: each thread a run of consecutive items
        const int per = (A.n + kPgThreads - 1) / kPgThreads;
        const int i0 = min(A.n, tid * per), i1 = min(A.n, i0 + per);
        uint32_t sum = 0;
        for (int i = i0; i < i1; ++i) {
            sum = sat_add(sum, incl[i], cap);
            incl[i] = sum;
        }
        uint32_t x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x = sat_add(x, y, cap);
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        uint32_t before = lane < warp ? warp_sum[lane] : 0u;  // the warps before this one
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before = sat_add(before, __shfl_xor_sync(0xFFFFFFFFu, before, o), cap);
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, 1);
        if (lane > 0) before = sat_add(before, y, cap);
        for (int i = i0; i < i1; ++i) incl[i] = sat_add(incl[i], before, cap);
        __syncthreads();
    }
    const uint32_t total = incl[A.n - 1];

    // ---- pages given back, and full pages shared: `ways` warps to an item
    const int ways = max(1, kWarps / A.n);
    for (int i = gwarp / ways; i < A.n; i += kWarps / ways) {
        const int first = (gwarp % ways) * 32 + lane;
        if constexpr (FORK) {
            const PagesItem<true> it = items[i];
            if (it.kind == 0) continue;
            const int held = max(0, min(A.count[it.dst], A.max_pages)), full = it.len >> A.page_shift;
            const int *from = A.table + (long long)it.src * A.max_pages;
            int *to = A.table + (long long)it.dst * A.max_pages;
            for (int j = first; j < max(held, full); j += ways * 32) {
                const int old = j < held ? to[j] : 0, p = j < full ? from[j] : -1;
                if (j < full) {  // its source holds it too: sharing it frees and takes nothing
                    if ((unsigned)p < (unsigned)A.num_pages) atomicAdd(A.ref + p, 1);
                    else flag(A.status, SPEC_DEV_BAD_PAGE);
                }
                to[j] = p;
                if (j < held) drop_page(A, old);
            }
        } else {
            const int held = items[i].held;
            int *row = A.table + (long long)i * A.max_pages;
            for (int j = items[i].need + first; j < held; j += ways * 32) {
                drop_page(A, row[j]);
                row[j] = -1;
            }
        }
    }
    __threadfence();
    cluster.sync();  // the old counts have been read, and what is free is known

    uint32_t free_total = 0;
    if (total > 0) {
        // ---- free pages counted, each warp a run of the pool
        const int per_warp = (int)(((long long)A.num_pages + kWarps * 32 - 1) / (kWarps * 32)) * 32;
        const long long p0 = (long long)gwarp * per_warp;
        const int run = (int)max(0ll, min((long long)per_warp, (long long)A.num_pages - p0));
        uint32_t mine = 0, mask[8];  // of 256 pages, each lane the same
        auto look = [&](int i) {
            int r[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int j = i + u * 32 + lane;
                r[u] = j < run ? __ldcg(A.ref + p0 + j) : 1;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) mask[u] = __ballot_sync(0xFFFFFFFFu, r[u] == 0);
        };
        for (int i = 0; i < run; i += 256) {
            look(i);
#pragma unroll
            for (int u = 0; u < 8; ++u) mine += (uint32_t)__popc(mask[u]);
        }
        if (lane == 0) warp_sum[warp] = mine;
        __syncthreads();
        const uint32_t w = warp_sum[lane], all = __reduce_add_sync(0xFFFFFFFFu, w);
        uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u);
        if (tid < kPgCtas) *cluster.map_shared_rank(&cta_free[rank], tid) = all;
        cluster.sync();
#pragma unroll
        for (int c = 0; c < kPgCtas; ++c) {
            if (c < rank) before += cta_free[c];
            free_total += cta_free[c];
        }
        // items are served while their running sum is within the free pages
        uint32_t served = total;
        if (total > free_total) {
            int lo = 0, hi = A.n;  // first item past the free pages
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (incl[mid] > free_total) hi = mid;
                else lo = mid + 1;
            }
            served = lo > 0 ? incl[lo - 1] : 0u;
            if (rank == 0 && tid == 0) flag(A.status, SPEC_DEV_NO_PAGES);
        }

        // ---- the lowest free pages handed out in item order
        if (before < served && mine > 0) {
            uint32_t at = before;
            for (int i = 0; i < run && at < served; i += 256) {
                if (run > 256) look(i);  // else the masks are still there
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t r = at + (uint32_t)__popc(mask[u] & ((1u << lane) - 1u));
                    if (((mask[u] >> lane) & 1u) && r < served) {
                        int lo = 0, hi = A.n - 1;  // first item whose running sum exceeds r
                        while (lo < hi) {
                            const int mid = (lo + hi) >> 1;
                            if (incl[mid] > r) hi = mid;
                            else lo = mid + 1;
                        }
                        const int first = lo > 0 ? (int)incl[lo - 1] : 0;
                        const int p = (int)p0 + i + u * 32 + lane;
                        A.ref[p] = 1;
                        if constexpr (FORK) {
                            A.table[(long long)items[lo].dst * A.max_pages + (items[lo].len >> A.page_shift)] = p;
                            A.copies[3 * lo + 1] = p;
                        } else {
                            A.table[(long long)lo * A.max_pages + items[lo].held + (int)r - first] = p;
                        }
                    }
                    at += (uint32_t)__popc(mask[u]);
                }
            }
        }
        if constexpr (FORK) {
            if (total > free_total) {  // forks that found no page share none either
                for (int i = gwarp / ways; i < A.n; i += kWarps / ways) {
                    const PagesItem<true> it = items[i];
                    if (it.kind != 2 || incl[i] <= free_total) continue;
                    int *to = A.table + (long long)it.dst * A.max_pages;
                    for (int j = (gwarp % ways) * 32 + lane; j < it.len >> A.page_shift; j += ways * 32) {
                        drop_page(A, to[j]);
                        to[j] = -1;
                    }
                }
            }
        }
    }

    for (int i = rank * kPgThreads + tid; i < A.n; i += kPgCtas * kPgThreads) {
        if constexpr (FORK) {
            const PagesItem<true> it = items[i];
            const bool ok = it.kind != 2 || incl[i] <= free_total;
            A.copies[3 * i + 2] = it.kind == 2 && ok ? (A.whole ? A.whole : it.len & (page - 1)) : 0;
            if (it.kind == 0) continue;
            if (it.kind == 2 && ok)
                A.copies[3 * i] = A.table[(long long)it.src * A.max_pages + (it.len >> A.page_shift)];
            A.count[it.dst] = ok ? pages_for(it.len, A.page_shift, A.max_pages) : 0;
            A.len[it.dst] = ok ? it.len : 0;
        } else {
            const int held = items[i].held, need = items[i].need;
            const uint32_t excl = i > 0 ? incl[i - 1] : 0u;
            A.count[i] = need < held ? need : held + (incl[i] <= free_total ? (int)(incl[i] - excl) : 0);
        }
    }
}

// ------------------------------------------------------------------ data movers

// One page to another in every layer: whole pages (copies NULL: src[i] to
// dst[i]), or the first tokens of a page as the bookkeeping of a fork listed
// them.  Grid (pairs, layers, token blocks), block (vector columns, tokens).
// Eight loads, four of keys and four of values, are in flight per thread before the
// first store.  64 forks of 16 slots, 24 layers: 31 us for the call, 8 of them the
// bookkeeping, and 124 MB that have to move.  The copy reads a source anew for each of its
// four forks, three times from L2, and by its counters (DRAM 31%, issue 33%) its 12288
// blocks are bound by their chains of dependent loads, not by HBM; blocks of
// keys or values alone took 35 us.
__global__ void __launch_bounds__(256) sv_copy_pages(Pool P, const int *src, const int *dst,
                                                     const int *copies, uint32_t *status) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x;
    int from, to, used = P.page;
    if (copies) {
        used = copies[3 * i + 2];
        if (used == 0) return;
        from = copies[3 * i];
        to = copies[3 * i + 1];
    } else {
        from = src[i];
        to = dst[i];
    }
    if ((unsigned)from >= (unsigned)P.num_pages || (unsigned)to >= (unsigned)P.num_pages) {
        if (threadIdx.x == 0 && threadIdx.y == 0) flag(status, SPEC_DEV_BAD_PAGE);
        return;
    }
    const long long base = (long long)blockIdx.y * P.layer, a = base + (long long)from * P.page_st,
                    b = base + (long long)to * P.page_st;
    const int step = blockDim.y * gridDim.z;
    for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
        const int h = c / P.vecs;
        const long long off = (long long)h * P.head + (c - h * P.vecs);
        for (int t = blockIdx.z * blockDim.y + threadIdx.y; t < used; t += 4 * step) {
            uint4 x[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long at = a + off + (long long)(t + u * step) * P.token;
                if (t + u * step < used) x[u] = ld_stream_v4(P.k + at), y[u] = ld_stream_v4(P.v + at);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long at = b + off + (long long)(t + u * step) * P.token;
                if (t + u * step < used) P.k[at] = x[u], P.v[at] = y[u];
            }
        }
    }
}

// New keys and values into the pages.  Grid (token blocks, requests), block
// (vector columns, tokens), a token per thread row: the grid's many small
// blocks keep enough loads in flight.  Bound by HBM: 16 requests of 2047 tokens,
// 268 MB, 38 us; a few tokens are bound by latency (two dependent loads).
__global__ void __launch_bounds__(256) sv_append(Pool P, const int *table,
                                                 const int *len,
                                                 const uint4 *k_new,
                                                 const uint4 *v_new, long long sb,
                                                 long long sn, long long sh,
                                                 const int *count, int N, int max_pages,
                                                 uint32_t *status) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y;
    const int n0 = len[b], m = count ? max(0, min(count[b], N)) : N;
    if (n0 < 0) {
        if (threadIdx.x == 0 && threadIdx.y == 0) flag(status, SPEC_DEV_BAD_LEN);
        return;
    }
    const int *row = table + (long long)b * max_pages;
    for (int n = blockIdx.x * blockDim.y + threadIdx.y; n < m; n += gridDim.x * blockDim.y) {
        const long long pos = (long long)n0 + n, place = pos >> P.page_shift;
        if (place >= max_pages) {
            if (threadIdx.x == 0) flag(status, SPEC_DEV_BAD_LEN);
            return;
        }
        const int p = row[place];
        if ((unsigned)p >= (unsigned)P.num_pages) {
            if (threadIdx.x == 0) flag(status, SPEC_DEV_BAD_PAGE);
            continue;
        }
        const long long to = (long long)p * P.page_st + (pos & (P.page - 1)) * P.token;
        const long long from = (long long)b * sb + (long long)n * sn;
        for (int c = threadIdx.x; c < P.cols; c += blockDim.x) {
            const int h = c / P.vecs, d = c - h * P.vecs;
            const uint4 x = ld_stream_v4(k_new + from + (long long)h * sh + d);
            const uint4 y = ld_stream_v4(v_new + from + (long long)h * sh + d);
            P.k[to + (long long)h * P.head + d] = x;
            P.v[to + (long long)h * P.head + d] = y;
        }
    }
}

// Accepted nodes moved behind their root.  Grid (requests, layers x {k, v}),
// block (vector columns, rows of the path).  Node i of the path lies at or past
// its place (out_nodes[i] >= i + 1), so a later node is never overwritten by an
// earlier move: all loads of a batch of moves, a barrier, then its stores.
// Nodes already in place are not touched.  Bound by latency at small batches
// (a chain of four dependent loads; 3.0 us at 4 requests of 8 nodes).  128 requests of 64
// nodes, 36 layers: 34 to 36 us for the 180 MB of the nodes that do not lie in place already, a
// floor of 27; DRAM is 48% busy inside the kernel and issue 41% (the same chain, then
// one batch of moves between two barriers).
constexpr int kMoveUnroll = 4;
__global__ void __launch_bounds__(256) sv_commit(Pool P, const int *table, const int *len,
                                                 const int *nodes,
                                                 const int *accept, int *new_len, int N,
                                                 int max_pages, uint32_t *status) {
    __shared__ long long s_src[SPEC_MAX_TREE], s_dst[SPEC_MAX_TREE];
    __shared__ int s_n;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x;
    const bool first = blockIdx.y == 0;
    const int a = commit_path(P, table, len, nodes, accept, b, N, max_pages, s_src, s_dst, &s_n,
                              status, first);
    if (first && new_len && threadIdx.x == 0 && threadIdx.y == 0) new_len[b] = commit_len(len[b], a);
    if (!nodes) return;
    uint4 *pool = ((blockIdx.y & 1) ? P.v : P.k) + (long long)(blockIdx.y >> 1) * P.layer;
    for (int c0 = 0; c0 < P.cols; c0 += blockDim.x) {
        const int c = c0 + threadIdx.x;
        const int h = c / P.vecs;
        const long long off = (long long)h * P.head + (c - h * P.vecs);
        for (int i0 = 0; i0 < a; i0 += kMoveUnroll * blockDim.y) {
            uint4 x[kMoveUnroll];
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u) {
                const int i = i0 + u * blockDim.y + threadIdx.y;
                if (c < P.cols && i < a && s_src[i] != s_dst[i]) x[u] = pool[s_src[i] + off];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u) {
                const int i = i0 + u * blockDim.y + threadIdx.y;
                if (c < P.cols && i < a && s_src[i] != s_dst[i]) pool[s_dst[i] + off] = x[u];
            }
        }
    }
}

// The lengths of spec_cache_commit where they are updated in place: after
// every mover has read the old ones (and reported what it found).
__global__ void __launch_bounds__(64) sv_commit_len(Pool P, const int *table, int *len,
                                                    const int *nodes, const int *accept, int N,
                                                    int max_pages, uint32_t *status) {
    __shared__ long long s_src[SPEC_MAX_TREE], s_dst[SPEC_MAX_TREE];
    __shared__ int s_n;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x;
    const int a = commit_path(P, table, len, nodes, accept, b, N, max_pages, s_src, s_dst, &s_n,
                              status, !nodes);
    if (threadIdx.x == 0) len[b] = commit_len(len[b], a);
}

// ------------------------------------------------------------------ host

spec_status_t make_pool(const spec_pages_t *p, Pool &P) {
    if (!p || !p->k || !p->v) return SPEC_ERR_INVALID_ARG;
    if (p->dtype != SPEC_DTYPE_F32 && p->dtype != SPEC_DTYPE_BF16 && p->dtype != SPEC_DTYPE_F16)
        return SPEC_ERR_UNSUPPORTED;
    if (p->layers < 1 || p->layers > 65535 || p->num_pages < 1 || p->num_pages == INT_MAX ||
        p->page_size < 8 || p->page_size > (1 << 20) || (p->page_size & (p->page_size - 1)) ||
        p->heads < 1 || p->heads > 1024 || p->head_dim < 8 || p->head_dim % 8 || p->head_dim > 1024)
        return SPEC_ERR_INVALID_ARG;
    if (((uintptr_t)p->k & 15) || ((uintptr_t)p->v & 15)) return SPEC_ERR_INVALID_ARG;
    const long long st[4] = {p->layer_stride, p->page_stride, p->token_stride, p->head_stride};
    const int extent[4] = {p->layers, p->num_pages, p->page_size, p->heads};
    for (int i = 0; i < 4; ++i) {
        if (st[i] < 0 || st[i] % 8) return SPEC_ERR_INVALID_ARG;
        if (extent[i] == 1) continue;
        // no two elements may share a place: a stride steps over all that the smaller
        // strides reach (of equal ones the other reaches as far as it steps)
        __int128 reach = p->head_dim;
        for (int j = 0; j < 4; ++j)
            if (j != i && st[j] <= st[i]) reach += (__int128)(extent[j] - 1) * st[j];
        if (st[i] < reach) return SPEC_ERR_INVALID_ARG;
    }
    const int per = p->dtype == SPEC_DTYPE_F32 ? 4 : 8;  // elements of a 16-byte vector
    P.k = static_cast<uint4 *>(p->k);
    P.v = static_cast<uint4 *>(p->v);
    P.layers = p->layers;
    P.num_pages = p->num_pages;
    P.page = p->page_size;
    P.page_shift = 0;
    while ((1 << P.page_shift) < P.page) ++P.page_shift;
    P.vecs = p->head_dim / per;
    P.cols = p->heads * P.vecs;
    P.layer = p->layer_stride / per;
    P.page_st = p->page_stride / per;
    P.token = p->token_stride / per;
    P.head = p->head_stride / per;
    return SPEC_OK;
}

bool current_device(int &dev, int &sms) {
    static int known[kMaxDevices] = {};
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    if (known[dev] == 0 && cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    sms = known[dev];
    return true;
}

// Threads over the vector columns of a token, and over tokens.
static dim3 column_block(int cols) {
    const int x = cols < 256 ? cols : 256;
    return dim3((unsigned)x, (unsigned)(256 / x));
}

// Token blocks of a page copy: four tokens per thread.
static int copy_blocks(const Pool &P, dim3 block) {
    const int n = (P.page + 4 * (int)block.y - 1) / (4 * (int)block.y);
    return n < 64 ? n : 64;
}

template <bool FORK>
static spec_status_t launch_pages(const PagesArgs &A, cudaStream_t s) {
    constexpr size_t item = sizeof(PagesItem<FORK>) + sizeof(uint32_t);
    constexpr size_t most = (item + (FORK ? sizeof(int) : 0)) * SPEC_MAX_SLOTS;
    static_assert(most + 2048 <= 232448, "shared memory of a CTA");
    const size_t smem = item * A.n + (FORK ? sizeof(int) * (size_t)A.slots : 0);
    static bool ready[kMaxDevices] = {};
    int dev = 0, sms = 0;
    if (!current_device(dev, sms)) return SPEC_ERR_CUDA;
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(sv_pages<FORK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)most) != cudaSuccess)
            return SPEC_ERR_CUDA;
        ready[dev] = true;
    }
    return launch_pdl(sv_pages<FORK>, dim3(kPgCtas), dim3(kPgThreads), smem, s, A);
}

spec_status_t launch_fork(const PagesArgs &A, const Pool &P, cudaStream_t s) {
    const spec_status_t sp = launch_pages<true>(A, s);
    if (sp != SPEC_OK) return sp;
    return launch_copy(P, nullptr, nullptr, A.copies, A.n, A.status, s);
}

spec_status_t launch_copy(const Pool &P, const int *src, const int *dst, const int *copies, int n, uint32_t *status,
                          cudaStream_t s) {
    const dim3 block = column_block(P.cols);
    return launch_pdl(sv_copy_pages, dim3((unsigned)n, (unsigned)P.layers, (unsigned)copy_blocks(P, block)), block, 0,
                      s, P, src, dst, copies, status);
}

spec_status_t launch_commit_len(const Pool &P, const int *table, int *len, const int *nodes, const int *accept, int B,
                                int N, int max_pages, uint32_t *status, cudaStream_t s) {
    return launch_pdl(sv_commit_len, dim3((unsigned)B), dim3(64), 0, s, P, table, len, nodes, accept, N, max_pages,
                      status);
}

} // namespace sv

extern "C" {

spec_status_t spec_cache_resize(int32_t *page_table, int32_t *page_count, int32_t *page_ref,
                                const int32_t *want_len, int extra, int page_size, int B,
                                int max_pages, int num_pages, uint32_t *dev_status, void *stream) {
    if (!page_table || !page_count || !page_ref || !want_len || extra < 0 || page_size < 8 ||
        page_size > (1 << 20) || (page_size & (page_size - 1)) || B < 1 || B > SPEC_MAX_SLOTS ||
        max_pages < 1 || num_pages < 1 || num_pages == INT_MAX)
        return SPEC_ERR_INVALID_ARG;
    sv::PagesArgs A = {};
    A.table = page_table;
    A.count = page_count;
    A.ref = page_ref;
    A.want = want_len;
    A.extra = extra;
    while ((1 << A.page_shift) < page_size) ++A.page_shift;
    A.n = A.slots = B;
    A.max_pages = max_pages;
    A.num_pages = num_pages;
    A.status = dev_status;
    return sv::launch_pages<false>(A, static_cast<cudaStream_t>(stream));
}

size_t spec_cache_fork_workspace_bytes(int F) {
    return F < 1 || F > SPEC_MAX_SLOTS ? 0 : ((size_t)F * 3 * sizeof(int32_t) + 255) & ~(size_t)255;
}

spec_status_t spec_cache_fork(const spec_pages_t *pages, int32_t *page_table, int32_t *page_count,
                              int32_t *page_ref, int32_t *cache_len, const int32_t *src,
                              const int32_t *dst, int F, int slots, int max_pages,
                              void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                              void *stream) {
    sv::Pool P;
    const spec_status_t st = sv::make_pool(pages, P);
    if (st != SPEC_OK) return st;
    if (!page_table || !page_count || !page_ref || !cache_len || !src || !dst || F < 1 ||
        F > SPEC_MAX_SLOTS || slots < 1 || slots > SPEC_MAX_SLOTS || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < spec_cache_fork_workspace_bytes(F))
        return SPEC_ERR_WORKSPACE;
    sv::PagesArgs A = {};
    A.table = page_table;
    A.count = page_count;
    A.ref = page_ref;
    A.len = cache_len;
    A.src = src;
    A.dst = dst;
    A.copies = static_cast<int *>(workspace);
    A.page_shift = P.page_shift;
    A.n = F;
    A.slots = slots;
    A.max_pages = max_pages;
    A.num_pages = P.num_pages;
    A.status = dev_status;
    return sv::launch_fork(A, P, static_cast<cudaStream_t>(stream));
}

spec_status_t spec_cache_copy(const spec_pages_t *pages, const int32_t *src_pages,
                              const int32_t *dst_pages, int n, uint32_t *dev_status, void *stream) {
    sv::Pool P;
    const spec_status_t st = sv::make_pool(pages, P);
    if (st != SPEC_OK) return st;
    if (!src_pages || !dst_pages || n < 1) return SPEC_ERR_INVALID_ARG;
    return sv::launch_copy(P, src_pages, dst_pages, nullptr, n, dev_status, static_cast<cudaStream_t>(stream));
}

spec_status_t spec_cache_append(const spec_pages_t *pages, const int32_t *page_table,
                                const int32_t *cache_len, const void *k_new, const void *v_new,
                                long long new_stride_b, long long new_stride_n,
                                long long new_stride_h, const int32_t *count, int B, int N,
                                int max_pages, uint32_t *dev_status, void *stream) {
    sv::Pool P;
    const spec_status_t st = sv::make_pool(pages, P);
    if (st != SPEC_OK) return st;
    if (P.layers != 1 || !page_table || !cache_len || !k_new || !v_new || ((uintptr_t)k_new & 15) ||
        ((uintptr_t)v_new & 15) || new_stride_b < 0 || new_stride_n < 0 || new_stride_h < 0 ||
        new_stride_b % 8 || new_stride_n % 8 || new_stride_h % 8 || B < 1 || B >= (1 << 16) || N < 1 ||
        max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    const int per = pages->dtype == SPEC_DTYPE_F32 ? 4 : 8;
    const dim3 block = sv::column_block(P.cols);
    const unsigned gx = ((unsigned)N + block.y - 1) / block.y;
    return sv::launch_pdl(sv::sv_append, dim3(gx, (unsigned)B), block, 0, static_cast<cudaStream_t>(stream), P,
                          page_table, cache_len, static_cast<const uint4 *>(k_new),
                          static_cast<const uint4 *>(v_new), new_stride_b / per, new_stride_n / per,
                          new_stride_h / per, count, N, max_pages, dev_status);
}

spec_status_t spec_cache_commit(const spec_pages_t *pages, const int32_t *page_table,
                                const int32_t *cache_len, const int32_t *out_nodes,
                                const int32_t *accept_len, int32_t *new_len, int B, int N,
                                int max_pages, uint32_t *dev_status, void *stream) {
    sv::Pool P;
    const spec_status_t st = sv::make_pool(pages, P);
    if (st != SPEC_OK) return st;
    if (!page_table || !cache_len || !accept_len || !new_len || B < 1 || B >= (1 << 16) || N < 1 ||
        N > SPEC_MAX_TREE || max_pages < 1 || P.layers > 32767)
        return SPEC_ERR_INVALID_ARG;
    const bool in_place = new_len == cache_len;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (out_nodes || !in_place) {
        const dim3 block = sv::column_block(P.cols);
        const spec_status_t r =
            sv::launch_pdl(sv::sv_commit, dim3((unsigned)B, out_nodes ? 2u * P.layers : 1u), block, 0, s, P,
                           page_table, cache_len, out_nodes, accept_len,
                           in_place ? (int *)nullptr : new_len, N, max_pages, dev_status);
        if (r != SPEC_OK || !in_place) return r;
    }
    return sv::launch_commit_len(P, page_table, new_len, out_nodes, accept_len, B, N, max_pages, dev_status, s);
}

} // extern "C"
