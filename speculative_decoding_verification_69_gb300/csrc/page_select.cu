// page_select.cu -- what chooses the pages that attention reads: the bounds of
// a page's keys, a score for every page, and the best pages as lists.
#include "cache4.cuh"

namespace sv {

// ------------------------------------------------------------------ bounds

struct BoundsArgs {
    Pool P;             // 16-bit pool (vectors)
    Pool4 P4;           // or 4-bit pool
    const int *table, *start, *len;
    uint4 *bounds;      // [page][head][2][vecs]
    int heads, vecs, page, page_shift, num_pages, max_pages;
    uint32_t *status;
};

template <int DT> __device__ __forceinline__ uint32_t min16(uint32_t a, uint32_t b);
template <int DT> __device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b);
#define SV_PAIR(name, dt, type, fn)                                                                  \
    template <> __device__ __forceinline__ uint32_t name<dt>(uint32_t a, uint32_t b) {               \
        const type r = fn(*reinterpret_cast<const type *>(&a), *reinterpret_cast<const type *>(&b)); \
        return *reinterpret_cast<const uint32_t *>(&r);                                              \
    }
SV_PAIR(min16, SPEC_DTYPE_BF16, __nv_bfloat162, __hmin2_nan)
SV_PAIR(max16, SPEC_DTYPE_BF16, __nv_bfloat162, __hmax2_nan)
SV_PAIR(min16, SPEC_DTYPE_F16, __half2, __hmin2_nan)
SV_PAIR(max16, SPEC_DTYPE_F16, __half2, __hmax2_nan)
#undef SV_PAIR

template <int DT> __device__ __forceinline__ void take_bounds(uint4 &lo, uint4 &hi, uint4 a, uint4 b) {
    lo.x = min16<DT>(lo.x, a.x), lo.y = min16<DT>(lo.y, a.y), lo.z = min16<DT>(lo.z, a.z), lo.w = min16<DT>(lo.w, a.w);
    hi.x = max16<DT>(hi.x, b.x), hi.y = max16<DT>(hi.y, b.y), hi.z = max16<DT>(hi.z, b.z), hi.w = max16<DT>(hi.w, b.w);
}

// The smallest and largest of every channel of a page's keys, which any order of the keys gives alike.  Grid (runs of
// pages, requests), block (vector columns, tokens): the columns' threads take every blockDim.y-th token and join in
// shared memory.  18.4 us for 32768 tokens of 8 heads of 128 (67 MB and 8 MB of bounds, 4 TB/s, launch included; HBM busy
// for 41 % of the time, 25 warps waiting for loads at an issue: latency, of a page at a time and its join), 18.5 from 4 bits
// (23.5 with pages of 64); after a step only the pages that grew are read, 4 to 5 us, a launch.
template <int DT, bool FOUR>
__global__ void __launch_bounds__(256) sv_bounds(const __grid_constant__ BoundsArgs A) {
    __shared__ uint4 part[2][256];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y, from = A.start ? max(A.start[b], 0) : 0;
    long long end = A.len[b];
    const bool lead = blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0;
    if (end < 0 || end > (long long)A.max_pages << A.page_shift) {
        if (lead) flag(A.status, SPEC_DEV_BAD_LEN);
        end = end < 0 ? 0 : (long long)A.max_pages << A.page_shift;
    }
    if (from >= end) return;
    const int last = (int)((end - 1) >> A.page_shift);
    const int cols = A.heads * A.vecs;
    const int *row = A.table + (long long)b * A.max_pages;
    int i = (from >> A.page_shift) + blockIdx.x, next = i <= last ? row[i] : 0;
    for (; i <= last; i += gridDim.x) {
        const int p = next;
        if (i + (int)gridDim.x <= last) next = row[i + gridDim.x];
        if ((unsigned)p >= (unsigned)A.num_pages) {
            if (threadIdx.x == 0 && threadIdx.y == 0) flag(A.status, SPEC_DEV_BAD_PAGE);
            continue;
        }
        const int used = (int)min((long long)A.page, end - ((long long)i << A.page_shift));
        for (int c0 = 0; c0 < cols; c0 += blockDim.x) {
            const int c = c0 + threadIdx.x, h = c / A.vecs, d8 = c - h * A.vecs;
            const uint32_t pinf = DT == SPEC_DTYPE_BF16 ? 0x7F807F80u : 0x7C007C00u, ninf = pinf | 0x80008000u;
            uint4 lo = make_uint4(pinf, pinf, pinf, pinf), hi = make_uint4(ninf, ninf, ninf, ninf);
            if (c < cols) {
                if constexpr (!FOUR) {
                    const uint4 *k = A.P.k + (long long)p * A.P.page_st + (long long)h * A.P.head + d8;
#pragma unroll 8
                    for (int t = threadIdx.y; t < used; t += blockDim.y) {
                        const uint4 x = ld_stream_v4(k + (long long)t * A.P.token);
                        take_bounds<DT>(lo, hi, x, x);
                    }
                } else {
                    const uint8_t *k = A.P4.data + p * A.P4.page_st + h * A.P4.head;
#pragma unroll 4
                    for (int t = threadIdx.y; t < used; t += blockDim.y) {
                        const uint32_t w = *reinterpret_cast<const uint32_t *>(k + key4(A.P4, t, d8 >> 2) + (d8 & 3) * 4);
                        const float s = scale_of(k[scale4(A.P4, t, d8 >> 2, false)]);
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 8; e += 2)
                            y[e / 2] = pack16<DT>(((float)((w >> bit4(e)) & 15u) - 8.f) * s,
                                                  ((float)((w >> bit4(e + 1)) & 15u) - 8.f) * s);
                        const uint4 x = make_uint4(y[0], y[1], y[2], y[3]);
                        take_bounds<DT>(lo, hi, x, x);
                    }
                }
            }
            if (blockDim.y > 1) {
                const int at = threadIdx.y * blockDim.x + threadIdx.x;
                __syncthreads();
                part[0][at] = lo, part[1][at] = hi;
                __syncthreads();
                if (threadIdx.y == 0)
                    for (int y = 1; y < blockDim.y; ++y)
                        take_bounds<DT>(lo, hi, part[0][y * blockDim.x + threadIdx.x], part[1][y * blockDim.x + threadIdx.x]);
            }
            if (threadIdx.y == 0 && c < cols) {
                uint4 *to = A.bounds + ((long long)p * A.heads + h) * 2 * A.vecs + d8;
                to[0] = lo;
                to[A.vecs] = hi;
            }
        }
    }
}

// ------------------------------------------------------------------ scores

struct ScoreArgs {
    const uint4 *q, *bounds;
    long long qb, qn, qh;  // strides of q in 16-byte vectors
    const int *table, *len, *node_count;
    float *scores;
    int B, N, G, heads, vecs, max_pages, num_pages, page, page_shift, tiles;
    uint32_t *status;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// c += A (16 pages x 16 channels) B (16 channels x 8 rows)
template <int DT>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if (DT == SPEC_DTYPE_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp scores 16 pages for one key head: the product of the pages' bounds [hi | lo] with the
// rows' [max(q, 0) | min(q, 0)], 16 pages by 8 rows at a time.  Bound by reading the bounds once
// (4 bytes per channel), which the warps' mma.sync keeps up with to about 64 rows: the operands
// go from HBM to registers in the product's own layout (a thread's share of the channels is
// contiguous, since any order of them gives the same sum) and pass no shared memory.
// The grid is as many CTAs as run at once; a warp's next page numbers come while it
// multiplies, so that each unit waits for memory once.  14 us for 4 requests of 4096 pages of 8 heads of 128 (67 MB, 4.8
// TB/s, launch included; 25 with a CTA for every 8 units), 18.4 for 64 requests of up to 512 pages of 8 heads of 64 and
// 20 rows (50 MB in pieces of 256 bytes of a page and head; three CTAs to an SM, q fetched
// ahead or 32 pages to a warp gain nothing).
template <int DT, int BLOCKS>  // BLOCKS of 32 channels
__global__ void __launch_bounds__(256, 2) sv_scores(const __grid_constant__ ScoreArgs A) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    // unit (b, tile, h), the heads of a tile side by side; a step of the grid as such a triple
    long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long step = (long long)gridDim.x * 8;
    int h = (int)(unit % A.heads), tile = (int)(unit / A.heads % A.tiles);
    long long b = unit / A.heads / A.tiles;
    const int step_h = (int)(step % A.heads), step_t = (int)(step / A.heads % A.tiles);
    const long long step_b = step / A.heads / A.tiles;
    int n = 0, rows = 0, page[2] = {-1, -1};
    auto fetch = [&]() {  // the unit's pages and sizes
        if (b >= A.B) return;
        long long len = A.len[b];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = tile * 16 + g + 8 * u;
            page[u] = i < A.max_pages ? A.table[b * A.max_pages + i] : -1;
        }
        rows = (A.node_count ? max(0, min(A.node_count[b], A.N)) : A.N) * A.G;
        if (len < 0 || len > (long long)A.max_pages << A.page_shift) {
            if (tile == 0 && h == 0 && lane == 0) flag(A.status, SPEC_DEV_BAD_LEN);
            len = len < 0 ? 0 : (long long)A.max_pages << A.page_shift;
        }
        n = (int)((len + A.page - 1) >> A.page_shift);
    };
    fetch();
    while (b < A.B) {
        const int i0 = tile * 16, rows_now = rows, h_now = h;
        const long long b_now = b;
        uint4 lo[2][BLOCKS], hi[2][BLOCKS];
        bool there[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + g + 8 * u;
            there[u] = i < n && (unsigned)page[u] < (unsigned)A.num_pages;
            if (i < n && !there[u] && t == 0) flag(A.status, SPEC_DEV_BAD_PAGE);
            const uint4 *x = A.bounds + ((long long)(there[u] ? page[u] : 0) * A.heads + h) * 2 * A.vecs;
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k) {
                const bool real = there[u] && rows > 0 && k * 4 + t < A.vecs;
                lo[u][k] = real ? ld_stream_v4(x + k * 4 + t) : none;
                hi[u][k] = real ? ld_stream_v4(x + A.vecs + k * 4 + t) : none;
            }
        }
        h += step_h;
        tile += step_t;
        b += step_b;
        if (h >= A.heads) h -= A.heads, ++tile;
        if (tile >= A.tiles) tile -= A.tiles, ++b;
        fetch();
        float best[2] = {-INFINITY, -INFINITY};
        const bool any = __any_sync(0xFFFFFFFFu, there[0] || there[1]);
        for (int r0 = 0; r0 < rows_now && any; r0 += 8) {
            const int r = r0 + g, node = r / A.G;
            const uint4 *q = A.q + b_now * A.qb + node * A.qn + (long long)(h_now * A.G + r - node * A.G) * A.qh;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k) {
                // (a plain load: one of data declared constant may be moved before the wait for who writes q)
                const uint4 y = r < rows_now && k * 4 + t < A.vecs ? q[k * 4 + t] : none;
                mma16<DT>(c, hi[0][k].x, hi[1][k].x, hi[0][k].y, hi[1][k].y, max16<DT>(y.x, 0u), max16<DT>(y.y, 0u));
                mma16<DT>(c, hi[0][k].z, hi[1][k].z, hi[0][k].w, hi[1][k].w, max16<DT>(y.z, 0u), max16<DT>(y.w, 0u));
                mma16<DT>(c, lo[0][k].x, lo[1][k].x, lo[0][k].y, lo[1][k].y, min16<DT>(y.x, 0u), min16<DT>(y.y, 0u));
                mma16<DT>(c, lo[0][k].z, lo[1][k].z, lo[0][k].w, lo[1][k].w, min16<DT>(y.z, 0u), min16<DT>(y.w, 0u));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (r0 + 2 * t + e < rows_now) {
                    best[0] = max_nan(best[0], c[e]);
                    best[1] = max_nan(best[1], c[2 + e]);
                }
        }
        float *out = A.scores + (b_now * A.heads + h_now) * A.max_pages;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            best[u] = max_nan(best[u], __shfl_xor_sync(0xFFFFFFFFu, best[u], 1));
            best[u] = max_nan(best[u], __shfl_xor_sync(0xFFFFFFFFu, best[u], 2));
            const int i = i0 + g + 8 * u;
            if (t == 0 && i < A.max_pages) out[i] = there[u] ? best[u] : -INFINITY;
        }
    }
}

// ------------------------------------------------------------------ selection

struct SelectArgs {
    const float *scores;
    const int *table, *len;
    int *out_table, *out_len;
    int heads, max_pages, page, page_shift, keep, first, recent, tail;
    uint32_t *status;
};

// A score as a whole number that orders alike, NaN before all others.  (-inf gives 0x007FFFFF: 0 stands for
// no page, and 0xFFFFFFFF for one that has to be taken.)
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // (-0 is 0)
    if (x != x) return 0xFFFFFFFEu;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A CTA selects for one request and key head.  The threads own runs of consecutive places, in
// registers where they fit.  The rank of the last page taken is found digit by digit: the ranks
// in question span [lo, lo + 2^bits), are counted in up to 2^11 equal parts of that, and the part in
// which the keep-th largest lies is the next span.  (Parts of the span that occurs, not digits of the whole
// number: scores of one sign and size share their upper digits, which all threads would count
// in one place.  Three rounds at most, most often two, instead of sixteen of a search by bits, which
// took 13 us for 8 heads of 4096 pages and 22 for 256 of 1024; this takes 6.4 for 32 heads of 4096 and 7 for
// 256 of 1024, both mostly latency.)  Then a scan gives every page its place.
constexpr int kSelBits = 11, kSelBins = 1 << kSelBits;
template <int THREADS, int ITEMS>  // ITEMS 0: any number, read anew in every round
__global__ void __launch_bounds__(THREADS) sv_select(const __grid_constant__ SelectArgs A) {
    constexpr int kWarps = THREADS / 32, kEach = kSelBins / THREADS;
    __shared__ __align__(16) int bins[kSelBins];
    __shared__ int scan[2][kWarps];
    __shared__ uint32_t ends[2][kWarps];
    __shared__ int found[2];
    pdl_trigger();
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kSelBins; i += THREADS) bins[i] = 0;
    pdl_wait();
    long long len = A.len[b];
    if (len < 0 || len > (long long)A.max_pages << A.page_shift) {
        if (h == 0 && tid == 0) flag(A.status, SPEC_DEV_BAD_LEN);
        len = len < 0 ? 0 : (long long)A.max_pages << A.page_shift;
    }
    const int n = (int)((len + A.page - 1) >> A.page_shift), kept = min(n, A.keep);
    if (h == 0 && tid == 0) A.out_len[b] = (int)(len - ((long long)(n - kept) << A.page_shift));
    const float *scores = A.scores + ((long long)b * A.heads + h) * A.max_pages;
    const int *row = A.table + (long long)b * A.max_pages;
    const int width = A.keep + A.tail;
    int *out = A.out_table + ((long long)b * A.heads + h) * width;
    for (int i = tid; i < width - kept; i += THREADS)  // the drafted tokens' pages, and none
        out[kept + i] = i < A.tail && n + i < A.max_pages ? row[n + i] : -1;
    if (n <= A.keep) {
        for (int i = tid; i < n; i += THREADS) out[i] = row[i];
        return;
    }
    const int per = ITEMS ? ITEMS : (n + THREADS - 1) / THREADS, i0 = tid * per;
    auto rank_at = [&](int i) -> uint32_t {
        if (i >= n) return 0u;
        if (i < A.first || i >= n - A.recent) return 0xFFFFFFFFu;
        return rank_of(scores[i]);
    };
    uint32_t mine[ITEMS ? ITEMS : 1];
    if (ITEMS) {
#pragma unroll
        for (int e = 0; e < ITEMS; ++e) mine[e] = rank_at(i0 + e);
    }
    auto each = [&](auto &&f) {
        if constexpr (ITEMS > 0) {
#pragma unroll
            for (int e = 0; e < ITEMS; ++e) f(i0 + e, mine[e]);
        } else {
            for (int e = 0; e < per; ++e) f(i0 + e, rank_at(i0 + e));
        }
    };
    // the span of the ranks that are up for choice
    uint32_t low = 0xFFFFFFFFu, high = 0u;
    each([&](int, uint32_t r) {
        if (r - 1u < 0xFFFFFFFEu) low = min(low, r), high = max(high, r);
    });
    low = __reduce_min_sync(0xFFFFFFFFu, low), high = __reduce_max_sync(0xFFFFFFFFu, high);
    if (lane == 0) ends[0][warp] = low, ends[1][warp] = high;
    __syncthreads();
    low = __reduce_min_sync(0xFFFFFFFFu, lane < kWarps ? ends[0][lane] : 0xFFFFFFFFu);
    high = __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? ends[1][lane] : 0u);
    // the largest rank that at least `keep` pages reach; of those in the span `want` are to be taken
    uint32_t lo = low;
    int bits = high > low ? 32 - __clz(high - low) : 0, want = A.keep - min(n, A.first + A.recent);
    while (want > 0 && bits > 0) {
        const int shift = max(0, bits - kSelBits);
        const uint32_t span = bits >= 32 ? 0xFFFFFFFFu : (1u << bits) - 1u;
        each([&](int, uint32_t r) {
            if (r - 1u < 0xFFFFFFFEu && r - lo <= span) atomicAdd(&bins[(r - lo) >> shift], 1);
        });
        __syncthreads();
        int c[kEach], sum = 0;  // from the top: the thread's bins, and those above them
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int at = kSelBins - 1 - (tid * kEach + e);
            c[e] = bins[at];
            bins[at] = 0;
            sum += c[e];
        }
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += u;
        }
        if (lane == 31) scan[0][warp] = x;
        __syncthreads();
        const int w = lane < kWarps ? scan[0][lane] : 0;
        int above = x - sum + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0);
        if (above < want && above + sum >= want) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (above < want && above + c[e] >= want) found[0] = kSelBins - 1 - (tid * kEach + e), found[1] = above;
                above += c[e];
            }
        }
        __syncthreads();
        lo += (uint32_t)found[0] << shift;
        want -= found[1];
        bits = shift;
    }
    // pages above the bar are all taken, of those at it the first ones.  (With nothing up for choice, only those
    // that have to be; of those, too many, the first.)
    const uint32_t bar = A.keep > min(n, A.first + A.recent) ? lo : 0xFFFFFFFFu;
    int above = 0, at = 0;
    each([&](int, uint32_t r) { above += r > bar ? 1 : 0, at += r == bar ? 1 : 0; });
    int x = above, y = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) x += u, y += v;
    }
    __syncthreads();
    if (lane == 31) scan[0][warp] = x, scan[1][warp] = y;
    __syncthreads();
    const int w0 = lane < kWarps ? scan[0][lane] : 0, w1 = lane < kWarps ? scan[1][lane] : 0;
    const int ties = A.keep - __reduce_add_sync(0xFFFFFFFFu, w0);  // taken of those at the bar
    int over = x - above + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w0 : 0);
    int equal = y - at + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w1 : 0);
    each([&](int i, uint32_t r) {
        const bool tie = r == bar;
        if (r > bar || (tie && equal < ties)) out[over + min(equal, ties)] = row[i];
        over += r > bar ? 1 : 0;
        equal += tie ? 1 : 0;
    });
}

template <class K> static spec_status_t launch_bounds(K kernel, const BoundsArgs &A, int B, cudaStream_t s) {
    const int cols = A.heads * A.vecs, x = cols < 256 ? cols : 256;
    int dev = 0, sms = 0;
    if (!current_device(dev, sms)) return SPEC_ERR_CUDA;
    // as many CTAs as run at once (16 to an SM: 0.5 us more for few pages; 3: 26 us instead of the 18.4 above)
    const int want = (5 * sms + B - 1) / B, runs = want < A.max_pages ? want : A.max_pages;
    return launch_pdl(kernel, dim3((unsigned)runs, (unsigned)B), dim3((unsigned)x, (unsigned)(256 / x)), 0, s, A);
}

} // namespace sv

extern "C" {

spec_status_t spec_cache_bounds(const spec_pages_t *pages, const int32_t *page_table, const int32_t *start,
                                const int32_t *cache_len, void *bounds, int B, int max_pages, uint32_t *dev_status,
                                void *stream) {
    sv::BoundsArgs A = {};
    const spec_status_t st = sv::make_pool(pages, A.P);
    if (st != SPEC_OK) return st;
    if (pages->dtype != SPEC_DTYPE_BF16 && pages->dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    if (pages->layers != 1 || !page_table || !cache_len || !bounds || ((uintptr_t)bounds & 15) || B < 1 ||
        B >= (1 << 16) || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    A.table = page_table;
    A.start = start;
    A.len = cache_len;
    A.bounds = static_cast<uint4 *>(bounds);
    A.heads = pages->heads;
    A.vecs = A.P.vecs;
    A.page = A.P.page;
    A.page_shift = A.P.page_shift;
    A.num_pages = A.P.num_pages;
    A.max_pages = max_pages;
    A.status = dev_status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return pages->dtype == SPEC_DTYPE_BF16 ? sv::launch_bounds(sv::sv_bounds<SPEC_DTYPE_BF16, false>, A, B, s)
                                           : sv::launch_bounds(sv::sv_bounds<SPEC_DTYPE_F16, false>, A, B, s);
}

spec_status_t spec_cache4_bounds(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *start,
                                 const int32_t *cache_len, void *bounds, spec_dtype_t dtype, int B, int max_pages,
                                 uint32_t *dev_status, void *stream) {
    sv::BoundsArgs A = {};
    const spec_status_t st = sv::make_pool4(pages, A.P4);
    if (st != SPEC_OK) return st;
    if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    if (pages->layers != 1 || !page_table || !cache_len || !bounds || ((uintptr_t)bounds & 15) || B < 1 ||
        B >= (1 << 16) || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    A.table = page_table;
    A.start = start;
    A.len = cache_len;
    A.bounds = static_cast<uint4 *>(bounds);
    A.heads = pages->heads;
    A.vecs = A.P4.D / 8;
    A.page = A.P4.page;
    A.page_shift = A.P4.page_shift;
    A.num_pages = A.P4.num_pages;
    A.max_pages = max_pages;
    A.status = dev_status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_DTYPE_BF16 ? sv::launch_bounds(sv::sv_bounds<SPEC_DTYPE_BF16, true>, A, B, s)
                                    : sv::launch_bounds(sv::sv_bounds<SPEC_DTYPE_F16, true>, A, B, s);
}

spec_status_t spec_page_scores(const void *q, spec_dtype_t dtype, long long q_stride_b, long long q_stride_n,
                               long long q_stride_h, const void *bounds, const int32_t *page_table,
                               const int32_t *cache_len, const int32_t *node_count, float *scores, int B, int N,
                               int Hq, int heads, int head_dim, int max_pages, int num_pages, int page_size,
                               uint32_t *dev_status, void *stream) {
    if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    if (!q || !bounds || !page_table || !cache_len || !scores || ((uintptr_t)q & 15) || ((uintptr_t)bounds & 15) ||
        B < 1 || B >= (1 << 16) || N < 1 || N > SPEC_MAX_TREE || heads < 1 || heads > 1024 || Hq < heads ||
        Hq % heads || Hq / heads > 64 || head_dim < 8 || head_dim % 8 || head_dim > SPEC_MAX_HEAD_DIM ||
        max_pages < 1 || num_pages < 1 || page_size < 8 || page_size > (1 << 20) || (page_size & (page_size - 1)))
        return SPEC_ERR_INVALID_ARG;
    const long long qst[3] = {q_stride_h, q_stride_n, q_stride_b};
    const int qext[3] = {Hq, N, B};
    for (int i = 0; i < 3; ++i)
        if (qst[i] % 8 || qst[i] < (qext[i] > 1 ? head_dim : 0)) return SPEC_ERR_INVALID_ARG;
    sv::ScoreArgs A = {};
    A.q = static_cast<const uint4 *>(q);
    A.bounds = static_cast<const uint4 *>(bounds);
    A.qb = q_stride_b / 8;
    A.qn = q_stride_n / 8;
    A.qh = q_stride_h / 8;
    A.table = page_table;
    A.len = cache_len;
    A.node_count = node_count;
    A.scores = scores;
    A.B = B;
    A.N = N;
    A.G = Hq / heads;
    A.heads = heads;
    A.vecs = head_dim / 8;
    A.max_pages = max_pages;
    A.num_pages = num_pages;
    A.page = page_size;
    while ((1 << A.page_shift) < page_size) ++A.page_shift;
    A.tiles = (max_pages - 1) / 16 + 1;
    A.status = dev_status;
    const long long ctas = ((long long)B * heads * A.tiles + 7) / 8;
    int dev = 0, sms = 0;
    if (!sv::current_device(dev, sms)) return SPEC_ERR_CUDA;
    const dim3 grid((unsigned)(ctas < 2 * sms ? ctas : 2 * sms)), block(256);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf = dtype == SPEC_DTYPE_BF16;
    if (head_dim <= 64)
        return bf ? sv::launch_pdl(sv::sv_scores<SPEC_DTYPE_BF16, 2>, grid, block, 0, s, A)
                  : sv::launch_pdl(sv::sv_scores<SPEC_DTYPE_F16, 2>, grid, block, 0, s, A);
    return bf ? sv::launch_pdl(sv::sv_scores<SPEC_DTYPE_BF16, 4>, grid, block, 0, s, A)
              : sv::launch_pdl(sv::sv_scores<SPEC_DTYPE_F16, 4>, grid, block, 0, s, A);
}

spec_status_t spec_page_select(const float *scores, const int32_t *page_table, const int32_t *cache_len,
                               int32_t *out_table, int32_t *out_len, int B, int heads, int max_pages, int page_size,
                               int keep, int first, int recent, int extra, uint32_t *dev_status, void *stream) {
    if (!scores || !page_table || !cache_len || !out_table || !out_len || B < 1 || B >= (1 << 16) || heads < 1 ||
        heads > 1024 || max_pages < 1 || max_pages > SPEC_MAX_SELECT || page_size < 8 || page_size > (1 << 20) ||
        (page_size & (page_size - 1)) || keep < 1 || keep > SPEC_MAX_SELECT || first < 0 || recent < 1 ||
        first > keep - recent || extra < 0 || extra > (1 << 20))
        return SPEC_ERR_INVALID_ARG;
    sv::SelectArgs A = {};
    A.scores = scores;
    A.table = page_table;
    A.len = cache_len;
    A.out_table = out_table;
    A.out_len = out_len;
    A.heads = heads;
    A.max_pages = max_pages;
    A.page = page_size;
    while ((1 << A.page_shift) < page_size) ++A.page_shift;
    A.keep = keep;
    A.first = first;
    A.recent = recent;
    A.tail = (extra + page_size - 1) / page_size;
    A.status = dev_status;
    const dim3 grid((unsigned)heads, (unsigned)B);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The fewest threads that keep a row in registers, 16 places each at most: 32 requests of 1025 places and 8 heads take
    // 7 us with 256 threads and 12 with 1024; beyond, every round reads the scores again.
    if (max_pages <= 256 * 4) return sv::launch_pdl(sv::sv_select<256, 4>, grid, dim3(256), 0, s, A);
    if (max_pages <= 256 * 8) return sv::launch_pdl(sv::sv_select<256, 8>, grid, dim3(256), 0, s, A);
    if (max_pages <= 1024 * 8) return sv::launch_pdl(sv::sv_select<1024, 8>, grid, dim3(1024), 0, s, A);
    if (max_pages <= 1024 * 16) return sv::launch_pdl(sv::sv_select<1024, 16>, grid, dim3(1024), 0, s, A);
    return sv::launch_pdl(sv::sv_select<1024, 0>, grid, dim3(1024), 0, s, A);
}

} // extern "C"
