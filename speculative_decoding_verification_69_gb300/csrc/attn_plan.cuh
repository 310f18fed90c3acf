// attn_plan.cuh -- what the attention kernels over paged caches share (tree_attn.cu in 16
// bits, tree_attn4.cu in 4): the list of work units and its cuts, the warp that
// schedules them, the nodes' paths, tensor-core instructions, and the join of the
// parts of an item that a cut fell into.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "lm_gemm.cuh"
#include "spec_cache.h"
#include "sv_cache.cuh"
#include "tmem.cuh"

namespace sv {

constexpr int kTaKeys = 128;        // keys of a tile (MMA N of S, MMA K of O)
constexpr int kTaRows = 128;        // rows of a stream (MMA M, TMEM lanes)
constexpr int kTaSlots = 4;         // segments the scheduler may be ahead
constexpr int kTaMaxCtas = 160;     // CTAs the workspace has room for
constexpr int kTaJoinLanes = 16;    // lanes of a row in the join
constexpr int kTaChunks = 128;      // entries of the running sum over requests
constexpr uint32_t kTaTries = 1u << 19;                  // looks of a wait: 2 s
constexpr unsigned long long kTaWaitNs = 2000000000ull;  // for the waits at the end
constexpr float kTaGrow = 8.f;      // growth of a row's maximum that rescales its O

extern bool g_diag_timeout;  // spec_debug_force_wait_timeout

// What the two streams of a CTA divide between them.
enum { kTaSplitKeys, kTaSplitRows, kTaSplitHeads };

struct TaArgs {
    const int *table, *len, *parent, *node_count;
    long long row_b, row_h;  // from one request's row of the table to the next, from one key head's (0: one for all)
    int B, N, Hq, H, G, D, max_pages, num_pages, page, page_shift;
    int window, sinks;
    int np;              // nodes of one stream's rows
    int box;             // tokens of a TMA box
    float scale_log2;
    uint16_t *out;
    float *lse;
    float *part_o;       // [cta][2][rows][D]
    float2 *part_ml;     // [cta][2][rows]: m, l (see tree_attn_join)
    const uint16_t *v;   // the pool's values and their strides in elements (K and V come through tensor
    long long v_page, v_token, v_head;  // maps: these are for values that are not finite)
    int4 *joins;         // [cta]: request, key head (or pair), first node and parts (0: none), see tree_attn_join
    uint32_t *status;
    uint32_t tries;      // looks of a wait
};

// What one request's tiles cover: positions [0, min(sinks, ...)) in its first
// `st` tiles and [wlo, end) in the tiles from wt0 on.
struct Geo {
    int c, cnt, end;   // committed positions, nodes, positions
    int wlo;           // first position inside the root's window
    int st, wt0, nt;   // sink tiles, first window tile, tiles
    __device__ __forceinline__ int tile(int i) const { return i < st ? i : wt0 + (i - st); }
};

// Committed positions and nodes of request b, clamped to what the table can hold.
__device__ __forceinline__ int2 ta_lens(const TaArgs &A, int b) {
    // (a tile of positions past the last one stays below 2^31)
    const int cap = (int)min((long long)A.max_pages << A.page_shift, (1ll << 31) - 2 * kTaKeys);
    int cnt = A.node_count ? max(0, min(__ldcg(A.node_count + b), A.N)) : A.N;
    int c = __ldcg(A.len + b);
    if (c < 0 || c > cap - cnt) {
        flag(A.status, SPEC_DEV_BAD_LEN);
        c = max(0, min(c, cap));
        cnt = min(cnt, cap - c);
    }
    return make_int2(c, cnt);
}
__device__ __forceinline__ Geo ta_geo(const TaArgs &A, int2 lens) {
    Geo g;
    g.c = lens.x;
    g.cnt = lens.y;
    g.end = g.c + g.cnt;
    g.wlo = A.window ? max(0, g.c - A.window + 1) : 0;
    g.wt0 = g.wlo / kTaKeys;
    g.st = A.window && A.sinks > 0 ? min((A.sinks - 1) / kTaKeys + 1, g.wt0) : 0;
    g.nt = g.cnt > 0 ? g.st + (g.end - 1) / kTaKeys + 1 - g.wt0 : 0;
    return g;
}

// A run of key tiles of one (request, key head, row tile).
struct Seg {
    Geo g;
    int b, hk, node0;   // node0: first node of the row tile
    int i0, n;          // tiles [i0, i0 + n) of the g.nt
};

// A segment as the scheduling warp hands it to the others; n = 0 ends the list.
struct SegSlot {
    Seg s;
    unsigned long long path[SPEC_MAX_TREE];  // the nodes that each node sees
    int low[SPEC_MAX_TREE];                  // the first committed position in its window
};

template <int MODE> __device__ __forceinline__ int ta_nodes(const TaArgs &A) {
    return A.np * (MODE == kTaSplitRows ? 2 : 1);
}
// Row tiles of a request with cnt nodes (the host makes them whole for cnt = N).
template <int MODE> __device__ __forceinline__ int ta_row_tiles(const TaArgs &A, int cnt) {
    const int npt = ta_nodes<MODE>(A);
    return cnt <= npt ? 1 : (cnt + npt - 1) / npt;
}
template <int MODE> __device__ __forceinline__ long long ta_units(const TaArgs &A, const Geo &g) {
    return (long long)g.nt * (A.H * ta_row_tiles<MODE>(A, g.cnt));
}
__device__ __forceinline__ long long ta_div(long long a, long long b) {  // a, b >= 0; 32 bits when they fit
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The scheduling warp's place in the list of units.
template <int MODE> struct Walk {
    int b0;          // the lanes hold the lengths of requests b0 + lane
    int2 lens;
    int b, hk, rt, rts, i0;
    Geo g;

    __device__ __forceinline__ void fetch(const TaArgs &A, int from) {
        const int lane = threadIdx.x & 31;
        b0 = from;
        lens = from + lane < A.B ? ta_lens(A, from + lane) : make_int2(0, 0);
    }
    __device__ __forceinline__ void enter(const TaArgs &A, int request) {
        b = request;
        g = ta_geo(A, make_int2(__shfl_sync(0xFFFFFFFFu, lens.x, b - b0), __shfl_sync(0xFFFFFFFFu, lens.y, b - b0)));
        rts = ta_row_tiles<MODE>(A, g.cnt);
        hk = rt = i0 = 0;
    }
    // To unit u, which exists; the first requests have been fetched.
    __device__ __forceinline__ void find(const TaArgs &A, const long long *incl, long long u) {
        const int lane = threadIdx.x & 31;
        const int per = (A.B + kTaChunks - 1) / kTaChunks;
        int from = 0, k = 0;
        long long base = 0;
#pragma unroll 1
        for (int i = 0; i < kTaChunks; i += 32) {  // the chunks that end at or before u
            const long long x = base + incl[i + lane];
            k = __popc(__ballot_sync(0xFFFFFFFFu, x <= u));
            from = i;
            if (k < 32) {
                if (k > 0) base = __shfl_sync(0xFFFFFFFFu, x, k - 1);
                break;
            }
            base = __shfl_sync(0xFFFFFFFFu, x, 31);
        }
        if (per > 1) {  // the requests of the chunk that end at or before u
#pragma unroll 1
            for (from = (from + k) * per;; from += 32) {
                fetch(A, from);
                long long x = ta_units<MODE>(A, ta_geo(A, lens));
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                    if (lane >= o) x += y;
                }
                k = __popc(__ballot_sync(0xFFFFFFFFu, base + x <= u));
                if (k > 0) base += __shfl_sync(0xFFFFFFFFu, x, k - 1);
                if (k < 32 || from + 32 >= A.B) break;
            }
        } else if (from != b0) {
            fetch(A, from);
        }
        enter(A, min(from + min(k, 31), A.B - 1));
        // (the bounds hold by themselves unless the lengths are written during the call,
        // which then must not lead out of any array)
        const int item = (int)min(ta_div(max(u - base, 0ll), max(g.nt, 1)), (long long)A.H * rts - 1);
        hk = item / rts;
        rt = item - hk * rts;
        i0 = (int)min(max(u - base - (long long)item * g.nt, 0ll), max(g.nt - 1ll, 0ll));
    }
    // Past n tiles, within or to the end of the item.
    __device__ __forceinline__ void advance(const TaArgs &A, int n) {
        i0 += n;
        if (i0 < g.nt) return;
        i0 = 0;
        if (++rt < rts) return;
        rt = 0;
        if (++hk < A.H) return;
        int next = b + 1;  // the next request that has nodes
        for (;;) {
            const int lane = threadIdx.x & 31;
            const uint32_t some = __ballot_sync(0xFFFFFFFFu, lens.y > 0 && b0 + lane >= next);
            if (some) {
                enter(A, b0 + __ffs(some) - 1);
                return;
            }
            if (b0 + 32 >= A.B) return;
            fetch(A, next = b0 + 32);
        }
    }
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *tm, int x, int y, int z, int w,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// True in one lane of a converged warp.  Products and copies are issued under
// this predicate, with operands that are the same in all lanes: the compiler
// then knows them to be uniform and issues them back to back.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one)::"memory");
    return one != 0;
}

// Whether the phase is over, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for a phase, until another role has given up or `tries` looks have been in
// vain; a look sleeps for 3.9 us unless the phase ends.  (A limit by count: the wait is
// inlined in many places, and a timer in each was code to be fetched, 4 us of 105 at a
// window of 128 and 512 requests.)
__device__ __forceinline__ bool ta_wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t tries) {
#pragma unroll 1
    for (uint32_t i = 0; i < tries; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    return false;
}

// D (TMEM) (+)= A (shared) B (shared)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D (TMEM) (+)= A (TMEM, two 16-bit elements per column) B (shared)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f16: float32 accumulator, A and B of the
// cache's dtype, M = 128; b_mn: B is MN-major.
template <int DT> __device__ __forceinline__ constexpr uint32_t ta_idesc(int n, bool b_mn) {
    const uint32_t f = DT == SPEC_DTYPE_BF16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kTaRows >> 4) << 24);
}

template <int DT> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<SPEC_DTYPE_BF16>(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}
template <> __device__ __forceinline__ uint32_t pack2<SPEC_DTYPE_F16>(float lo, float hi) {
    const __half2 x = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// The nodes on the path to every node, as bits, for nodes `lane` and `lane +
// 32` of the warp: the links are followed by doubling (6 rounds reach 64).
__device__ __forceinline__ void ta_paths(const TaArgs &A, int b, int cnt, unsigned long long (&anc)[2]) {
    const int lane = threadIdx.x & 31;
    if (!A.parent) {
        anc[0] = (2ull << lane) - 1ull;
        anc[1] = lane == 31 ? ~0ull : (2ull << (lane + 32)) - 1ull;
        return;
    }
    int up[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int n = lane + 32 * k;
        anc[k] = 1ull << n;
        up[k] = -1;
        if (n > 0 && n < cnt) {
            up[k] = __ldcg(A.parent + (long long)b * A.N + n);
            if ((unsigned)up[k] >= (unsigned)n) {
                flag(A.status, SPEC_DEV_BAD_TREE);
                up[k] = -1;
            }
        }
    }
#pragma unroll 1
    while (__any_sync(0xFFFFFFFFu, up[0] >= 0 || up[1] >= 0)) {  // at most 6 rounds
        unsigned long long na[2];
        int nu[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int p = up[k] & 31;
            const unsigned long long a0 = __shfl_sync(0xFFFFFFFFu, anc[0], p), a1 = __shfl_sync(0xFFFFFFFFu, anc[1], p);
            const int u0 = __shfl_sync(0xFFFFFFFFu, up[0], p), u1 = __shfl_sync(0xFFFFFFFFu, up[1], p);
            na[k] = up[k] < 0 ? anc[k] : anc[k] | (up[k] < 32 ? a0 : a1);
            nu[k] = up[k] < 0 ? -1 : (up[k] < 32 ? u0 : u1);
        }
        anc[0] = na[0], anc[1] = na[1];
        up[0] = nu[0], up[1] = nu[1];
    }
}

// log sum exp of a row from its reference (base 2) and sum, which is 0 or NaN where no
// score is above -inf or one is not a number.
__device__ __forceinline__ float ta_lse(bool exists, float m, float l) {
    if (!exists) return -INFINITY;
    return l > 0.f ? 0.69314718056f * (m + log2f(l)) : __uint_as_float(0x7FFFFFFFu);
}

// The units of all requests, summed up to the end of each chunk of them (kTaChunks threads; every 32nd chunk
// begins anew).  Returns whether some request has fewer than N nodes.
template <int MODE> __device__ __forceinline__ bool ta_sum_units(const TaArgs &A, long long *incl) {
    const int per = (A.B + kTaChunks - 1) / kTaChunks;
    const int lane = threadIdx.x & 31;
    bool fewer = false;  // some request has fewer than N nodes
    const int b0 = threadIdx.x * per, b1 = min(A.B, b0 + per);
    long long x = 0;
#pragma unroll 2
    for (int b = b0; b < b1; ++b) {
        const int2 lens = ta_lens(A, b);
        fewer |= lens.y < A.N;
        x += ta_units<MODE>(A, ta_geo(A, lens));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    incl[threadIdx.x] = x;
    return fewer;
}

// The scheduling warp: the segments of the units [u_first, u_last) handed to the others, runs of `run` units
// being a CTA's.
template <int MODE>
__device__ __forceinline__ void ta_schedule(const TaArgs &A, Walk<MODE> &w, const long long *incl, SegSlot *seg,
                                    uint64_t *seg_full, uint64_t *path_full, uint64_t *seg_free,
                                    long long u_first, long long u_last, long long run,
                                    volatile int *abort) {
    const int lane = threadIdx.x & 31;
    int k = 0, b = -1;
    bool ok = true;
    unsigned long long anc[2] = {0, 0};
    int low[2] = {0, 0};
    if (u_first < u_last) w.find(A, incl, u_first);
    for (long long left = u_last - u_first; ok; ++k) {
        Seg s = {};
        if (left > 0) {
            s.g = w.g;
            s.b = w.b;
            s.hk = w.hk;
            s.node0 = w.rt * ta_nodes<MODE>(A);
            s.i0 = w.i0;
            s.n = (int)min((long long)(w.g.nt - w.i0), left);
            left -= s.n;
        }
        if (k >= kTaSlots)
            ok = __all_sync(0xFFFFFFFFu,
                            ta_wait(&seg_free[k % kTaSlots], (k / kTaSlots - 1) & 1, abort, A.tries));
        if (!ok) break;
        SegSlot &slot = seg[k % kTaSlots];
        if (lane == 0) {
            slot.s = s;
            mbar_arrive(reinterpret_cast<unsigned long long *>(&seg_full[k % kTaSlots]));
        }
        if (k == 0 && lane == 0) {
            // the CTA's first unit lies inside an item: if the item began in the CTA
            // before, this is its first cut, where its parts are joined
            const long long start = u_first - s.i0;
            int parts = 0;
            if (s.i0 > 0 && start >= u_first - run) {
                const long long last = min(ta_div(start + s.g.nt - 1, run), gridDim.x - 1ll);
                parts = (int)(last - (long long)blockIdx.x) + 2;
            }
            A.joins[blockIdx.x] = make_int4(s.b, s.hk, s.node0, parts);
        }
        // the loads and scores go ahead; the softmax warps need the paths too
        if (s.n > 0 && s.b != b) {
            ta_paths(A, b = s.b, s.g.cnt, anc);
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // less the nodes before the window
                if (!A.window) break;
                low[x] = max(0, s.g.c + __popcll(anc[x]) - A.window);
                unsigned long long left = anc[x];
#pragma unroll 1
                for (int place = s.g.c; left && place < low[x]; ++place) {
                    const unsigned long long bit = left & (0ull - left);
                    if (place >= A.sinks) anc[x] &= ~bit;
                    left ^= bit;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            slot.path[lane + 32 * x] = anc[x];
            slot.low[lane + 32 * x] = low[x];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(&path_full[k % kTaSlots]));
        if (s.n == 0) break;
        w.advance(A, s.n);
    }
    __syncwarp();
}

// The parts of an item that cuts fell into, joined in the order of the keys.
// joins[j]: the first cut of an item lies at CTA j's first unit; its parts are
// slot 1 of the CTA before, where it begins, and slot 0 of CTA j and those after.  A part
// holds sums of weights 2^(x - m) of scores x in base 2, or (RAW) 2^((x - m) scale + lift) of scores
// that are not scaled yet, whose differences scaling would round; m is -inf where the row does not exist.
// 16 lanes per row, two vectors of four columns each: bound by the latency of three
// dependent loads at few rows (3.4 us of a call of one token at one request) and
// by instructions at many (10 us at 64 nodes and 64 requests); a warp per row
// took 16.7 us there, 8 lanes 9.5 but 3 us more with 20 parts of 64 rows.
template <int DT, bool RAW>
static __global__ void __launch_bounds__(256) tree_attn_join(TaArgs A, int rows_used, int rows_cta, int mode,
                                                             float scale, float lift) {
    constexpr int L = kTaJoinLanes, kVecs = 32 / L;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % L, prow = blockIdx.y * (256 / L) + threadIdx.x / L;
    const int4 a = A.joins[blockIdx.x];
    const int parts = a.w, first = (int)blockIdx.x - 1;
    auto slot = [&](int i) { return ((first + i) * 2 + (i == 0 ? 1 : 0)) * rows_cta + prow; };
    // the first L parts' m and l, fetched beside the description of the cut
    float2 x0 = make_float2(-INFINITY, 0.f);
    if (first >= 0 && first + lane < (int)gridDim.x && prow < rows_cta) x0 = A.part_ml[slot(lane)];
    const int stream = prow / rows_used, row = prow - stream * rows_used;
    const int local = row / A.G, node = a.z + (mode == kTaSplitRows ? stream * A.np : 0) + local;
    const int hk = mode == kTaSplitHeads ? 2 * a.y + stream : a.y;
    if (parts == 0) return;
    // (of an odd number of heads in pairs the last one is none)
    const bool works = prow < rows_cta && node < A.N && hk * A.G < A.Hq;
    const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, works);
    if (!works) return;
    float m = lane < parts ? x0.x : -INFINITY;
    for (int i = lane + L; i < parts; i += L) m = fmaxf(m, A.part_ml[slot(i)].x);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o, L));
    const bool some = m != -INFINITY;  // the row exists
    float l = 0.f;
    float4 o[kVecs] = {};
    for (int i0 = 0; i0 < parts; i0 += L) {
        float w = 0.f;
        if (some && i0 + lane < parts) {
            const float2 x = i0 == 0 ? x0 : A.part_ml[slot(i0 + lane)];
            w = ex2(RAW ? (x.x - m) * scale : x.x - m);
            l = fmaf(x.y, w, l);
        }
        const int k = min(L, parts - i0);
#pragma unroll 8
        for (int i = 0; i < k; ++i) {
            const float wi = __shfl_sync(lanes, w, i, L);
            const float4 *part = reinterpret_cast<const float4 *>(A.part_o + (long long)slot(i0 + i) * A.D);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                if (4 * (lane + v * L) < A.D) {
                    const float4 x = part[lane + v * L];
                    o[v].x = fmaf(x.x, wi, o[v].x);
                    o[v].y = fmaf(x.y, wi, o[v].y);
                    o[v].z = fmaf(x.z, wi, o[v].z);
                    o[v].w = fmaf(x.w, wi, o[v].w);
                }
            }
        }
    }
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) l += __shfl_xor_sync(lanes, l, d, L);
    const float inv = some ? 1.f / l : 0.f;
    const long long orow = ((long long)a.x * A.N + node) * A.Hq + (long long)hk * A.G + (row - local * A.G);
    uint2 *dst = reinterpret_cast<uint2 *>(A.out + orow * A.D);
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
        if (4 * (lane + v * L) < A.D)
            dst[lane + v * L] = some ? make_uint2(pack2<DT>(o[v].x * inv, o[v].y * inv),
                                                  pack2<DT>(o[v].z * inv, o[v].w * inv))
                                     : make_uint2(0u, 0u);
    if (lane == 0 && A.lse) A.lse[orow] = ta_lse(some, RAW ? fmaxf(m * scale, -FLT_MAX) - lift : m, l);
}

constexpr float kTaLog2e = 1.44269504089f;
// Whether the factor of the scores is a number: an infinite one would make NaN of a score of 0.
static bool ta_scale_ok(float scale, float times) { return scale > 0.f && scale * kTaLog2e * times <= FLT_MAX; }

// A 4D tensor map over 16-bit elements, 64 of them (128 bytes, the swizzle
// span) wide; elements past an extent read as zero.  lines: what lies beside a row is of no use, so L2 fetches
// 128 bytes and not 256.
static bool ta_tmap(CUtensorMap *tm, int dtype, const void *base, const cuuint64_t (&dims)[4],
                    const cuuint64_t (&strides)[3], cuuint32_t box1, cuuint32_t box2, bool lines = false) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn)
            return false;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    const cuuint32_t box[4] = {64, box1, box2, 1}, estr[4] = {1, 1, 1, 1};
    return encode(tm, dtype == SPEC_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B,
                  lines ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

} // namespace sv
