// sv_cache.cuh -- what the kernels of the paged cache share: the pool of pages
// as 16-byte vectors, status flags, and launches that overlap the end of the
// kernel before them.
#pragma once
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "spec_cache.h"
#include "sv_common.cuh"

namespace sv {

// A pool of pages in units of 16-byte vectors.
struct Pool {
    uint4 *k, *v;
    long long layer, page_st, token, head;  // strides
    int layers, num_pages, page, page_shift;
    int vecs, cols;                         // vectors of a head, of a token
};

spec_status_t make_pool(const spec_pages_t *p, Pool &P);

// What the bookkeeping of pages works on.
struct PagesArgs {
    int *table, *count, *ref, *len;  // len: forks only
    const int *want;                 // resize only
    const int *src, *dst;            // forks only
    int *copies;                     // forks only: [n, 3] page to copy, its copy, tokens (0: none)
    int extra, page_shift, n, slots, max_pages, num_pages;  // n: items (slots or forks)
    int whole;                       // forks only: listed for every page to copy instead of its tokens (0: those)
    uint32_t *status;
};

// The launches of spec_cache.cu that other pools of pages take too: a fork (its bookkeeping and the
// copies it lists), copies of whole pages (src to dst, or as listed), lengths of a commit in place.
spec_status_t launch_fork(const PagesArgs &A, const Pool &P, cudaStream_t s);
spec_status_t launch_copy(const Pool &P, const int *src, const int *dst, const int *copies, int n, uint32_t *status,
                          cudaStream_t s);
spec_status_t launch_commit_len(const Pool &P, const int *table, int *len, const int *nodes, const int *accept, int B,
                                int N, int max_pages, uint32_t *status, cudaStream_t s);

__device__ __forceinline__ void flag(uint32_t *status, uint32_t bits) {
    if (status) atomicOr(status, bits);
}

// The accepted path of one request: place 0 is the root's, place 1 + i that of node i.
// Returns how many nodes after the root are kept, those before the first place without a
// page (nodes: or the first that is no path), and -1 when the root has none: the length
// grows by one more.  s_src / s_dst [N]: the nodes' vector offsets inside a layer, before
// and after.  Called by a whole CTA; warp 0 works.
__device__ __forceinline__ int commit_path(const Pool &P, const int *table, const int *len,
                                           const int *nodes, const int *accept, int b, int N,
                                           int max_pages, long long *s_src, long long *s_dst,
                                           int *s_n, uint32_t *status, bool report) {
    const int lane = threadIdx.y * blockDim.x + threadIdx.x;
    if (lane < 32) {
        const int a = max(0, min(accept[b], N - 1));
        const long long n0 = len[b];
        const int *row = table + (long long)b * max_pages;
        uint32_t bits = 0;
        int places = 0;  // the root's and the nodes' that are kept
        auto offset = [&](long long pos, long long &off) -> bool {  // whether the position has a page
            const long long place = pos >> P.page_shift;
            const int p = place < max_pages ? row[place] : -1;
            off = (long long)p * P.page_st + (pos & (P.page - 1)) * P.token;
            return (unsigned)p < (unsigned)P.num_pages;
        };
        if (n0 < 0) bits = SPEC_DEV_BAD_LEN;
        else places = a + 1;
        for (int i0 = 0; i0 < places; i0 += 32) {
            const int i = i0 + lane;
            bool bad = false;
            if (i < places) {
                long long src, dst;
                if (!nodes && (n0 + i) >> P.page_shift >= max_pages) {
                    bits |= SPEC_DEV_BAD_LEN;  // counted: no page will ever stand for it
                } else if (!offset(n0 + i, dst)) {
                    bad = true;
                    bits |= SPEC_DEV_BAD_PAGE;
                } else if (nodes && i > 0) {
                    const int n = nodes[(long long)b * N + i - 1];
                    if (n < i || n >= N) {
                        bad = true;
                        bits |= SPEC_DEV_BAD_TREE;
                    } else if (!offset(n0 + n, src)) {
                        bad = true;
                        bits |= SPEC_DEV_BAD_PAGE;
                    } else {
                        s_src[i - 1] = src;
                        s_dst[i - 1] = dst;
                    }
                }
            }
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, bad);
            if (mask) places = i0 + __ffs(mask) - 1;
        }
        if (report && bits) flag(status, bits);
        if (lane == 0) *s_n = places - 1;
    }
    __syncthreads();
    return *s_n;
}
// The length after the root and `kept` nodes (linear drafts may leave 32 bits).
__device__ __forceinline__ int commit_len(int len, int kept) {
    return (int)min((long long)len + 1 + kept, (long long)INT_MAX);
}

// The current device, and how many SMs it has; false if that fails or there are more devices than kMaxDevices.
constexpr int kMaxDevices = 64;
bool current_device(int &dev, int &sms);

// Launch that may begin while the kernel before it on the stream is still
// running: every kernel launched this way waits (pdl_wait) before it touches
// memory, so the order of the stream holds.
template <class... P, class... A>
spec_status_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? SPEC_OK
                                                                                      : SPEC_ERR_CUDA;
}

} // namespace sv
