// tree_attn.cu -- attention of drafted trees over a paged key/value cache on the
// sm_103a tensor cores.
//
// Mathematics.  For one request and one key head all N nodes' query heads of
// the group (G = Hq / heads) read the same keys and values, so the N * G rows
// form one matrix: S = Q K^T, softmax over the keys each row sees, O = P V.
// One pass over the keys keeps per row a reference m (near the running maximum
// of the scaled scores, base 2), l = sum 2^(s - m) and O = sum 2^(s - m) v:
// a later, larger maximum rescales l and O by 2^(m - m'), the online softmax of
// M. Milakov and N. Gimelshein, "Online normalizer calculation for softmax" (2018).
// O is rescaled only when the maximum has grown by more than 2^8, a refinement
// published since for accumulators that are dear to rescale: until then the weights
// are merely larger than 1, exactly representable in scale, and O stays untouched
// in the tensor memory.  Partial results over disjoint keys join the same way.
//
// Split.  The work is a list of units, one per (request, key head, row tile,
// 128-key tile) that somebody sees, in that order, cut into equal runs, one per
// CTA of a grid of one CTA per SM.  So one long request spreads over the GPU and
// thousands of short ones balance whatever their lengths; the lengths are
// read on the device.  A (request, head, row tile) that a cut falls into
// leaves float32 partials in the workspace, joined by tree_attn_join.
//
// One CTA: a warp each that schedules, loads K (and Q), loads V and issues the
// products, and two streams of softmax, four warps each (thread = row).  Up to
// 128 rows the streams take the key tiles in turn, each with its own m, l and
// O, joined at the end (kTaSplitKeys), or, with many requests, a key head each
// (kTaSplitHeads: a unit is then a pair of heads).  With more rows they take 128
// rows each of the same key tile (kTaSplitRows), so a row tile is 256 rows for
// one read of K and V.  Either way one stream's exponentials run while the
// tensor cores work for the other.
//
// What bounds it, with device times of a call, join included, on a GPU that copies
// 6.7 TB/s and multiplies bfloat16 matrices at 1937 TFLOP/s (32 query and 8 key heads of
// 128 unless said otherwise):
//   1 request of 131071 tokens, 16 nodes        96 us   5.6 TB/s    HBM, and a join of 20 parts
//   32 requests of up to 4096 tokens, 9 nodes   75 us   5.5 TB/s    HBM
//   64 requests, 64 nodes each (256 rows)      210 us   4.2 TB/s, 1000 TFLOP/s: a stream's chain of
//                scores, two halves of weights and values; the tensor cores are 45% busy
//   512 requests, 9 nodes, window of 128      101 us   2.2 TB/s    64 query heads of 64: short segments,
//                so the softmax warps' latency, half of it in masks, clearing and output
//   1 request of 1000 tokens, 1 node          11.5 us   latency: lengths, pages, a tile, the join
// K, V and P go through 128-key tiles because a product of 64 columns takes 48 cycles where
// one of 128 takes 64; P lies in the tensor memory (head_dim above 64: over its scores, since
// two accumulators leave no other columns), since it would otherwise be written to and read
// from shared memory, the port of which bounds a row tile of 256 rows at about 2050 cycles
// per key tile.
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
constexpr int kTaThreads = 384;     // 8 softmax warps, then K loads, products, scheduling and V loads
constexpr int kTaWarpK = 8, kTaWarpMma = 9, kTaWarpPlan = 10, kTaWarpV = 11;
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
    int B, N, Hq, H, G, D, max_pages, num_pages, page, page_shift;
    int window, sinks;
    int np;              // nodes of one stream's rows
    int box;             // tokens of a TMA box
    float scale_log2;
    uint16_t *out;
    float *lse;
    float *part_o;       // [cta][2][rows][D]
    float2 *part_ml;     // [cta][2][rows]: m (base 2), l
    const uint16_t *v;   // the pool's values and their strides in elements (K and V come through tensor
    long long v_page, v_token, v_head;  // maps: these are for values that are not finite)
    int4 *joins;         // [cta]: request, key head (or pair), first node and parts (0: none), see tree_attn_join
    uint32_t *status;
    uint32_t tries;      // looks of a wait
};

template <int DP, int MODE> struct TaCfg {
    static constexpr bool kOwnP = DP <= 64;  // the weights have tensor-memory columns of their own
    static constexpr int kStreamQ = kTaRows * DP * 2;            // bytes of one stream's Q
    static constexpr int kQ = kStreamQ * (MODE == kTaSplitKeys ? 1 : 2);
    static constexpr int kStage = kTaKeys * DP * 2;              // one K or V tile
    // as many tiles in flight as the shared memory holds beside Q
    static constexpr int kStagesK = DP == 128 ? 2 : (MODE == kTaSplitKeys ? 6 : 5);
    static constexpr int kStagesV = DP == 128 ? (MODE == kTaSplitKeys ? 3 : 2) : 6;
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

template <int DP, int MODE> struct TaShared {
    using C = TaCfg<DP, MODE>;
    uint8_t q[C::kQ];
    uint8_t k[C::kStagesK][C::kStage], v[C::kStagesV][C::kStage];
    long long incl[kTaChunks];  // units of the requests up to the end of each chunk, from every 32nd chunk on
    SegSlot seg[kTaSlots];
    int pages[2][32];           // K's and V's next pages
    uint64_t seg_full[kTaSlots], path_full[kTaSlots], seg_free[kTaSlots];
    uint64_t k_full[C::kStagesK], k_empty[C::kStagesK], v_full[C::kStagesV], v_empty[C::kStagesV];
    uint64_t s_full[2], p_full[2][2], pv_done[2][2];  // [stream][half of a tile]
    uint64_t q_full, q_free, o_free[2], ml_full, done;
    uint32_t tmem_base;
    int abort;
    int bad_v[2][2];            // [stream with kTaSplitHeads, else 0][segment parity]: 1 + the segment that
                                // held values that are not finite where only some rows see them
    float2 ml[MODE == kTaSplitKeys ? 2 : 1][2][MODE == kTaSplitKeys ? kTaRows : 1];  // [segment parity][stream][row]
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

// Shared-memory descriptor of a V tile as the B operand of O += P V: keys are
// the K dimension, the head dimension is contiguous (MN-major).  128-byte
// swizzle atoms of 8 keys x 64 elements: the next 8 keys 1024 bytes on (stride
// byte offset), the next 64 elements kTaKeys * 128 bytes on (leading byte
// offset).
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((uint32_t)(kTaKeys * 128) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
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

// Whether the two 16-bit elements of x are infinities or NaN: bits 15 and 31.  (All bits of
// the exponent are then set, and its lowest one more carries there.)
template <int DT> __device__ __forceinline__ uint32_t not_finite(uint32_t x) {
    constexpr uint32_t kExp = DT == SPEC_DTYPE_BF16 ? 0x7F807F80u : 0x7C007C00u;
    constexpr uint32_t kLow = DT == SPEC_DTYPE_BF16 ? 0x00800080u : 0x04000400u;
    return (x & kExp) + kLow;
}
// The same two with 0 for those.
template <int DT> __device__ __forceinline__ uint32_t finite_part(uint32_t x) {
    const uint32_t bad = not_finite<DT>(x);
    return x & (((bad >> 15) & 1u ? 0u : 0xFFFFu) | (bad >> 31 ? 0u : 0xFFFF0000u));
}
template <int DT> __device__ __forceinline__ float2 unpack2(uint32_t x) {
    if (DT == SPEC_DTYPE_BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// The positions [j, j + 64) that a row sees: committed ones from `low` on and the
// first `sinks`, and the nodes of its path, which lie from position c on.
// (Positions are below 2^31, and so are their differences.)
__device__ __forceinline__ unsigned long long seen_bits(int j, int c, int low, int sinks, unsigned long long path) {
    auto below = [&](int end) -> unsigned long long {  // the positions before `end`
        const int n = end - j;
        return n <= 0 ? 0ull : ~0ull >> max(64 - n, 0);
    };
    const int d = j - c;
    const unsigned long long nodes = d >= 64 || d <= -64 ? 0ull : d >= 0 ? path >> d : path << -d;
    return (below(c) & ~below(low)) | below(min(sinks, c)) | nodes;
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

// Adds to a row's accumulators the elements that were taken out of the values because they are
// not finite and not all rows see them: from the pool, those that the row does see (its weight
// for them is above 0, however small).  Stream `of` of a, a ^ 1 (two) holds the segment's tiles
// whose number from base0 on has its parity (kTaSplitKeys), or all of them.  Rare, and so out
// of line: the kernel's code is fetched anew by every short call.
template <int DT, int DP, int MODE>
__device__ __noinline__ void ta_add_not_finite(const TaArgs &A, Seg s, int hk, uint32_t o_cols, int col0, int a,
                                               bool two, bool valid, int sinks, int edge, int low,
                                               unsigned long long path, uint32_t base0) {
    constexpr int kCols = MODE == kTaSplitKeys ? DP / 2 : DP;
    const Geo &g = s.g;
    const int *table = A.table + (long long)s.b * A.max_pages;
    const uint16_t *v = A.v + hk * A.v_head + col0;
#pragma unroll 1
    for (int x = 0; x < (two ? 2 : 1); ++x) {
        const int of = a ^ x;
#pragma unroll 1
        for (int d = 0; d < kCols; d += 32) {
            uint32_t o[32];
            tmem_load(o_cols + (uint32_t)(of * DP + d), o);
#pragma unroll 1
            for (int i = 0; i < 2 * SPEC_MAX_TREE && valid; ++i) {
                const bool node_at = i >= SPEC_MAX_TREE;
                const int j = node_at ? g.c + (i - SPEC_MAX_TREE) : g.wlo + i;
                if (node_at ? j >= g.end || g.cnt == 1 : j >= edge || j < sinks) continue;
                if (!(node_at ? (path >> (j - g.c)) & 1ull : j >= low)) continue;
                const int t = g.st + j / kTaKeys - g.wt0 - s.i0;  // its tile of the segment
                if (t < 0 || t >= s.n) continue;
                if (MODE == kTaSplitKeys && ((base0 + (uint32_t)t) & 1u) != (uint32_t)of) continue;
                int page = __ldcg(table + (j >> A.page_shift));
                if ((unsigned)page >= (unsigned)A.num_pages) page = 0;
                const uint4 *src =
                    reinterpret_cast<const uint4 *>(v + page * A.v_page + (j & (A.page - 1)) * A.v_token + d);
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    if (col0 + d + e >= A.D) break;
                    const uint4 y = __ldcg(src + e / 8);
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t bad = not_finite<DT>(w[q]);
                        const float2 f = unpack2<DT>(w[q]);
                        uint32_t &lo = o[e + 2 * q], &hi = o[e + 2 * q + 1];
                        if ((bad >> 15) & 1u) lo = __float_as_uint(__uint_as_float(lo) + f.x);
                        if (bad >> 31) hi = __float_as_uint(__uint_as_float(hi) + f.y);
                    }
                }
            }
            __syncwarp();
            tmem_store(o_cols + (uint32_t)(of * DP + d), o);
        }
    }
    tmem_wait_store();
}

// ------------------------------------------------------------------ the kernel

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_attn(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TaArgs A) {
    using C = TaCfg<DP, MODE>;
    using Sh = TaShared<DP, MODE>;
    extern __shared__ uint8_t ta_raw[];
    Sh &sh = *reinterpret_cast<Sh *>((reinterpret_cast<uintptr_t>(ta_raw) + 1023) & ~(uintptr_t)1023);
    // through a shuffle, so that the compiler knows the roles' branches, and what is
    // computed in them, to be the same in all lanes of a warp
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    constexpr int kKS = C::kStagesK, kVS = C::kStagesV;
    constexpr int kHalves = DP / 64;
    constexpr int kPer = MODE == kTaSplitHeads ? 2 : 1;  // K and V tiles of a unit
    // P is scaled up to 2^15 in float16, so that weights 2^-29 below the
    // maximum are still normal numbers; bfloat16 has float32's range
    constexpr float kLift = DT == SPEC_DTYPE_F16 ? 7.f : 0.f;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kKS; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], 1);
        }
        for (int s = 0; s < kVS; ++s) {
            mbar_init(&sh.v_full[s], 1);
            mbar_init(&sh.v_empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh.p_full[i][h], 4);
                mbar_init(&sh.pv_done[i][h], 1);
            }
        }
        for (int i = 0; i < kTaSlots; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.path_full[i], 1);
            mbar_init(&sh.seg_free[i], 8 + 3);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_free, 1);
        mbar_init(&sh.o_free[0], 4);
        mbar_init(&sh.o_free[1], 4);
        mbar_init(&sh.ml_full, 8);
        mbar_init(&sh.done, 1);
        sh.abort = 0;
        for (int i = 0; i < 4; ++i) sh.bad_v[i >> 1][i & 1] = 0;
        fence_mbar_init();
        tma_prefetch_map(&tm_q);
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == kTaWarpMma) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    pdl_trigger();
    pdl_wait();
    Walk<MODE> w;
    if (warp == kTaWarpPlan) w.fetch(A, 0);
    bool fewer = false;  // some request has fewer than N nodes
    // the units of all requests, summed up to the end of each chunk of them
    if (threadIdx.x < kTaChunks) {
        const int per = (A.B + kTaChunks - 1) / kTaChunks;
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
        sh.incl[threadIdx.x] = x;
    }
    tc_fence_before();
    fewer = __syncthreads_or(fewer) != 0;
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
    volatile int *abort = &sh.abort;
    long long total = 0;
    for (int i = 31; i < kTaChunks; i += 32) total += sh.incl[i];
    const long long run = ta_div(total + gridDim.x - 1, gridDim.x);
    const long long u_first = min(total, (long long)blockIdx.x * run), u_last = min(total, u_first + run);

    // segment k, or nothing when the wait for it ran out
    auto take = [&](uint64_t *bars, int k) -> const SegSlot * {
        const bool ok = ta_wait(&bars[k % kTaSlots], (k / kTaSlots) & 1, abort, A.tries);
        return __all_sync(0xFFFFFFFFu, ok) ? &sh.seg[k % kTaSlots] : nullptr;
    };
    auto give = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(&sh.seg_free[k % kTaSlots]));
    };

    if (warp == kTaWarpPlan) {  // ----------------------------------------------- scheduling
        int k = 0, b = -1;
        bool ok = true;
        unsigned long long anc[2] = {0, 0};
        int low[2] = {0, 0};
        if (u_first < u_last) w.find(A, sh.incl, u_first);
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
                                ta_wait(&sh.seg_free[k % kTaSlots], (k / kTaSlots - 1) & 1, abort, A.tries));
            if (!ok) break;
            SegSlot &slot = sh.seg[k % kTaSlots];
            if (lane == 0) {
                slot.s = s;
                mbar_arrive(reinterpret_cast<unsigned long long *>(&sh.seg_full[k % kTaSlots]));
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
            if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(&sh.path_full[k % kTaSlots]));
            if (s.n == 0) break;
            w.advance(A, s.n);
        }
        __syncwarp();
    } else if (warp == kTaWarpK || warp == kTaWarpV) {  // --------------- loads
        const bool is_k = warp == kTaWarpK;
        const CUtensorMap *tm = is_k ? &tm_k : &tm_v;
        uint8_t *tiles = is_k ? sh.k[0] : sh.v[0];
        uint64_t *full = is_k ? sh.k_full : sh.v_full, *empty = is_k ? sh.k_empty : sh.v_empty;
        const uint32_t stages = is_k ? kKS : kVS;
        uint32_t stage = 0, fill = 0;               // next stage, and how often all have been filled
        int seg_no = 0, q_loads = 0;
        const int nb = kTaKeys / A.box;             // boxes of a tile
        const int ahead = 32 / nb;                  // tiles whose pages one load of the warp fetches
        const int box = lane % nb;
        bool ok = true;
        for (; ok; ++seg_no) {
            const SegSlot *sp = take(sh.seg_full, seg_no);
            if (!sp || sp->s.n == 0) break;
            const Seg s = sp->s;
            give(seg_no);
            const int *row = A.table + (long long)s.b * A.max_pages;
            const int i_end = s.i0 + s.n;
            // first position of this lane's box in tile i, and whether some node sees any of it
            auto box_pos = [&](int i) -> int { return s.g.tile(i) * kTaKeys + box * A.box; };
            auto box_seen = [&](int j) -> bool {
                return j < s.g.end && (s.g.wlo - j < A.box || j < A.sinks);
            };
            auto fetch = [&](int i0) -> int {  // page of this lane's box in tile i0 + lane / nb
                const int i = i0 + lane / nb;
                if (i >= i_end) return 0;
                const int j = box_pos(i);
                if (!box_seen(j)) return 0;
                int p = __ldcg(row + (j >> A.page_shift));
                if ((unsigned)p >= (unsigned)A.num_pages) {
                    flag(A.status, SPEC_DEV_BAD_PAGE);
                    p = 0;
                }
                return p;
            };
            // the pages of `ahead` tiles at a time go to shared memory, where the lane that
            // issues the copies reads them in a loop (unrolled over the boxes its code was
            // read anew for every tile, 250 cycles a copy); the next ones are on their way
            int base = s.i0, at = s.i0, nxt = 0;  // first tile of those in shared memory, next to be fetched
            int *pages = sh.pages[is_k ? 0 : 1];
            // Q of this segment once the scores of the last one are done: looked for
            // before every load, so that the tiles need not wait for it
            bool q_due = is_k;
            auto issue_q = [&]() {
                constexpr int kQs = MODE == kTaSplitKeys ? 1 : 2;
                if (elect_one()) {
                    mbar_expect_tx(&sh.q_full, (uint32_t)(kQs * kHalves * A.np * A.G * 128));
#pragma unroll 1
                    for (int q = 0; q < kQs; ++q)
#pragma unroll 1
                        for (int h = 0; h < kHalves; ++h)
                            tma_load_4d(sh.q + q * C::kStreamQ + h * kTaRows * 128, &tm_q, h * 64,
                                        (MODE == kTaSplitHeads ? 2 * s.hk + q : s.hk) * A.G,
                                        MODE == kTaSplitRows ? s.node0 + q * A.np : s.node0, s.b, &sh.q_full);
                }
                __syncwarp();
                q_due = false;
                ++q_loads;
            };
            auto look_q = [&]() {
                if (q_due &&
                    __any_sync(0xFFFFFFFFu, seg_no == 0 || mbar_test_wait(&sh.q_free, (uint32_t)(seg_no - 1) & 1u)))
                    issue_q();
            };
            for (int i = s.i0; i < i_end && ok; ++i) {
                if (i == s.i0 || i == base + ahead) {
                    base = i;
                    int now;
#pragma unroll 1
                    do {  // at first these and the next ones, then one load ahead
                        now = nxt;
                        nxt = fetch(at);
                        at += ahead;
                    } while (at == s.i0 + ahead);
                    __syncwarp();
                    pages[lane] = now;
                    __syncwarp();
                }
                const uint32_t seen = __ballot_sync(0xFFFFFFFFu, lane < nb && box_seen(box_pos(i)));
                const int tok = (s.g.tile(i) * kTaKeys) & (A.page - 1);
#pragma unroll 1
                for (int head = s.hk * kPer; head < (s.hk + 1) * kPer && ok; ++head) {
#pragma unroll 1
                    for (uint32_t tries = 0;; ++tries) {
                        look_q();
                        if (fill == 0 || __any_sync(0xFFFFFFFFu, mbar_try_wait(&empty[stage], (fill - 1) & 1u)))
                            break;
                        if (__any_sync(0xFFFFFFFFu, *abort || tries >= A.tries)) {
                            *abort = 1;
                            ok = false;
                            break;
                        }
                    }
                    if (!ok) break;
                    uint8_t *tile = tiles + stage * C::kStage;
                    if (elect_one()) {
                        mbar_expect_tx(&full[stage], (uint32_t)(__popc(seen) * kHalves * A.box * 128));
                        const int *page = pages + (i - base) * nb;
#pragma unroll 1
                        for (int x = 0; x < nb; ++x, ++page, tile += A.box * 128) {
                            if (!((seen >> x) & 1u)) continue;
                            tma_load_4d(tile, tm, 0, tok, head, *page, &full[stage]);
                            if (kHalves == 2) tma_load_4d(tile + kTaKeys * 128, tm, 64, tok, head, *page, &full[stage]);
                        }
                    }
                    __syncwarp();
                    if (++stage == stages) stage = 0, ++fill;
                }
            }
            if (ok && q_due) {
                ok = __all_sync(0xFFFFFFFFu, ta_wait(&sh.q_free, (uint32_t)(seg_no - 1) & 1u, abort, A.tries));
                if (ok) issue_q();
            }
        }
        // every copy has landed before the CTA may exit
        for (uint32_t x = 0; x < stages; ++x) {
            const uint32_t n = fill + (x < stage ? 1u : 0u);
            if (n > 0) mbar_wait_bounded(&full[x], (n - 1) & 1u, kTaWaitNs);
        }
        if (q_loads > 0) mbar_wait_bounded(&sh.q_full, (uint32_t)(q_loads - 1) & 1u, kTaWaitNs);
        __syncwarp();
    } else if (warp == kTaWarpMma) {  // --------------------------------- products
        uint32_t k_tile = 0, v_tile = 0;   // K and V tiles used
        uint32_t use[2] = {0, 0};          // tiles of each stream whose values are through
        int seg_no = 0;
        bool ok = true;
        constexpr uint32_t kIdS = ta_idesc<DT>(kTaKeys, false), kIdO = ta_idesc<DT>(DP, true);
        const uint64_t q_desc = umma_desc_sw128(smem_u32(sh.q)), k_desc = umma_desc_sw128(smem_u32(sh.k[0])),
                       vt_desc = v_desc(smem_u32(sh.v[0]));
        auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xFFFFFFFFu, ta_wait(bar, parity, abort, A.tries)) != 0;
        };
        // The wait for a phase that ends within a product or two: looked at before it is
        // slept on.
        auto wait_soon = [&](uint64_t *bar, uint32_t parity) -> bool {
#pragma unroll 1
            for (int n = 0; n < 256; ++n)
                if (mbar_test_wait(bar, parity)) return true;
            return wait(bar, parity);
        };
        // Scores of stream i against the next K tile; release: the tile's last use,
        // last: the segment's.  Where they overwrite the columns of the stream's last weights
        // (!kOwnP) the values formed from those have to be through: products of one thread
        // are only sure to execute in the order of issue when they share accumulator and
        // shape.  The wait costs 208 us instead of 196 at 64 requests of 64 nodes, 39.3
        // instead of 38.2 at a window of 4096 and 16 nodes, 0 to 1% elsewhere; scores in two
        // halves of 64 keys, each behind the values of its own columns, took 249 and 42.8.
        auto scores = [&](int i, bool release, bool last) -> bool {
            const uint32_t st = k_tile % kKS;
            if ((MODE != kTaSplitRows || i == 0) && !wait(&sh.k_full[st], (k_tile / kKS) & 1u)) return false;
            if (!C::kOwnP && use[i] > 0 && !wait_soon(&sh.pv_done[i][1], (use[i] - 1) & 1u)) return false;
            tc_fence_after();
            const uint64_t qd = q_desc + (uint64_t)((MODE == kTaSplitKeys ? 0 : i) * (C::kStreamQ / 16));
            const uint64_t kd = k_desc + (uint64_t)(st * (C::kStage / 16));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {  // the columns past D hold zeros
                    const uint64_t off = (uint64_t)((k >> 2) * (kTaRows * 128 / 16) + (k & 3) * 2);
                    mma_ss(tmem + (uint32_t)(i * kTaKeys), qd + off, kd + off, kIdS, k > 0 ? 1u : 0u);
                }
                umma_commit(&sh.s_full[i]);
                if (release) umma_commit(&sh.k_empty[st]);
                if (last) umma_commit(&sh.q_free);
            }
            __syncwarp();
            if (release) ++k_tile;
            return true;
        };
        // O of stream i plus its weights of half h times that half of the next V tile
        // (fresh: the first of the segment)
        auto values = [&](int i, int h, bool fresh, bool release) -> bool {
            const uint32_t st = v_tile % kVS;
            if (!wait(&sh.p_full[i][h], use[i] & 1u)) return false;
            if (h == 0 && (MODE != kTaSplitRows || i == 0) && !wait(&sh.v_full[st], (v_tile / kVS) & 1u)) return false;
            tc_fence_after();
            const uint64_t vd = vt_desc + (uint64_t)(st * (C::kStage / 16) + h * (kTaKeys / 2 * 128 / 16));
            const uint32_t p = tmem + (C::kOwnP ? 384u + (uint32_t)(i * (kTaKeys / 2) + h * (kTaKeys / 4))
                                                : (uint32_t)(i * kTaKeys + h * (kTaKeys / 2) + kTaKeys / 4));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTaKeys / 32; ++k)
                    mma_ts(tmem + 256u + (uint32_t)(i * DP), p + (uint32_t)(k * 8), vd + (uint64_t)(k * 2048 / 16),
                           kIdO, fresh && h == 0 && k == 0 ? 0u : 1u);
                umma_commit(&sh.pv_done[i][h]);
                if (release) umma_commit(&sh.v_empty[st]);
            }
            __syncwarp();
            if (release) ++v_tile;
            if (h == 1) ++use[i];
            return true;
        };
        if (MODE == kTaSplitRows) {
            for (; ok; ++seg_no) {
                const SegSlot *sp = take(sh.seg_full, seg_no);
                if (!sp || sp->s.n == 0) break;
                const int n = __shfl_sync(0xFFFFFFFFu, sp->s.n, 0);
                give(seg_no);
                ok = wait(&sh.q_full, (uint32_t)seg_no & 1u);
                ok = ok && scores(0, false, false) && scores(1, true, n == 1);
                for (int t = 0; t < n && ok; ++t) {
                    const bool more = t + 1 < n;
                    if (t == 0 && seg_no > 0)
                        ok = wait(&sh.o_free[0], (uint32_t)(seg_no - 1) & 1u) &&
                             wait(&sh.o_free[1], (uint32_t)(seg_no - 1) & 1u);
                    ok = ok && values(0, 0, t == 0, false) && values(0, 1, false, false) &&
                         (!more || scores(0, false, false)) && values(1, 0, t == 0, false) &&
                         values(1, 1, false, true) && (!more || scores(1, true, t + 2 == n));
                }
            }
        } else {
            // The streams take the CTA's tiles in turn, whatever segment they belong to;
            // a stream's next scores follow its values at once, also those of the next
            // segment, so that they are there when its results have been written.
            const uint32_t tiles = (uint32_t)(u_last - u_first) * kPer;
            int s_seg = 0, s_left = 0, v_seg = 0, v_left = 0;  // segments begun by scores and values, tiles left
            bool fresh0 = false, fresh1 = false;               // the next values are the stream's first of a segment
            auto next_scores = [&](int i) -> bool {
                if (s_left == 0) {
                    if (!wait(&sh.seg_full[s_seg % kTaSlots], (uint32_t)(s_seg / kTaSlots) & 1u)) return false;
                    s_left = __shfl_sync(0xFFFFFFFFu, sh.seg[s_seg % kTaSlots].s.n, 0) * kPer;
                    if (!wait(&sh.q_full, (uint32_t)s_seg & 1u)) return false;
                    ++s_seg;
                }
                return scores(i, true, --s_left == 0);
            };
            auto next_values = [&](int i) -> bool {
                if (v_left == 0) {
                    v_left = __shfl_sync(0xFFFFFFFFu, sh.seg[v_seg % kTaSlots].s.n, 0) * kPer;
                    ++v_seg;
                    fresh0 = fresh1 = true;
                }
                // both streams' warps read either stream's O, or each its own (kTaSplitHeads)
                if (v_seg > 1 && (i == 0 ? fresh0 : fresh1)) {
                    const uint32_t parity = (uint32_t)(v_seg - 2) & 1u;
                    if (MODE == kTaSplitKeys && !wait(&sh.o_free[i ^ 1], parity)) return false;
                    if (!wait(&sh.o_free[i], parity)) return false;
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h)
                    if (!values(i, h, i == 0 ? fresh0 : fresh1, h == 1)) return false;
                if (i == 0) fresh0 = false;
                else fresh1 = false;
                if (--v_left == 0) give(v_seg - 1);
                return true;
            };
            // Before the last values of a segment no scores are put: its results wait for
            // them (kTaSplitHeads: each stream's for its own).
            int given = 0;  // tiles whose scores have been issued
#pragma unroll 1
            for (int e = -1; e < (int)tiles && ok; ++e) {
                if (e >= 0) ok = next_values(e & 1);
#pragma unroll 1
                while (ok && given < min(e + 3, (int)tiles) && (MODE == kTaSplitHeads || given <= e + 1 || v_left != 1))
                    ok = next_scores(given++ & 1);
            }
        }
        // every MMA has finished before the TMEM is freed
        if (elect_one()) umma_commit(&sh.done);
        mbar_wait_bounded(&sh.done, 0u, kTaWaitNs);
        __syncwarp();
    } else if (warp < 8) {  // ------------------------------------------- softmax
        const int stream = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + (uint32_t)(stream * kTaKeys);   // S
        const uint32_t tp = C::kOwnP ? tmem + lanes + 384u + (uint32_t)(stream * (kTaKeys / 2))
                                     : ts + kTaKeys / 4;                   // P, or over the second half of each half of S
        constexpr int kPHalf = C::kOwnP ? kTaKeys / 4 : kTaKeys / 2;       // columns from P's first half to its second
        const uint32_t to = tmem + lanes + 256u + (uint32_t)(stream * DP);  // O
        const int rows_used = A.np * A.G, local = row / A.G;
        uint32_t base = 0;                     // the CTA's tiles before this segment
        int seg_no = 0;
        bool ok = true;
        for (; ok; ++seg_no) {
            const SegSlot *sp = take(sh.path_full, seg_no);
            if (!sp || sp->s.n == 0) break;
            const Seg s = sp->s;
            const Geo &g = s.g;
            const int node = s.node0 + (MODE == kTaSplitRows ? stream * A.np : 0) + local;
            const bool valid = row < rows_used && node < g.cnt;
            const unsigned long long path = valid ? sp->path[node] : 0ull;
            const int low = valid ? sp->low[node] : 0;
            give(seg_no);
            const int sinks = A.window ? A.sinks : 0;
            // positions that some rows of the request see and others do not: its nodes, and before
            // them [wlo, edge) without the sinks
            const int edge = A.window && g.cnt > 1 ? min(g.c, g.c + g.cnt - A.window) : 0;
            int *bad_v = &sh.bad_v[MODE == kTaSplitHeads ? stream : 0][seg_no & 1];
            const bool warp_works = __any_sync(0xFFFFFFFFu, valid);
            float m = -INFINITY;                       // reference of the weights, less the lift
            float2 l2 = make_float2(0.f, 0.f);
            const int t_step = MODE == kTaSplitKeys ? 2 : 1;
            bool first = true;
            const int t0 = MODE == kTaSplitKeys ? (int)((base + stream) & 1u) : 0;
            for (int t = t0; t < s.n && ok; t += t_step, first = false) {
                const int j0 = g.tile(s.i0 + t) * kTaKeys;
                const uint32_t use = (base + (uint32_t)t) >> (MODE == kTaSplitKeys ? 1 : 0);  // the stream's
                // values that no node sees may be anything: they are cleared, so that their zero
                // weights leave them out (kTaSplitRows: by stream 0, whose weights are used first).
                // So are elements that are not finite where only some rows see them; those rows
                // get them with the result (the check makes 208.9 us of 207.4 at 64 requests of 64
                // nodes, 101.0 of 99.1 at a window of 128, 11.5 of 11.2 at one token).
                // The tile is waited for before its scores, which leaves the time they take, where
                // the stage's parity can be trusted by then (kEarly): not while the fill before
                // this one may be due.  The stream has seen its last tile's scores, which were
                // issued when the values up to one tile before that (kTaSplitRows) or two (the
                // streams in turn, so 4 before this one) had their tiles.  Otherwise the scores
                // come first, which were issued after the values two tiles before.
                constexpr bool kEarly = MODE == kTaSplitRows || kVS >= 4;
                const uint32_t v_tile = (base + (uint32_t)t) * kPer + (MODE == kTaSplitHeads ? stream : 0);
                const uint32_t v_stage = v_tile % kVS, v_parity = (v_tile / kVS) & 1u;
                const bool clear = (MODE != kTaSplitRows || stream == 0) &&
                                   (g.end - j0 < kTaKeys || (j0 < g.wlo && A.sinks - j0 < kTaKeys) ||
                                    (g.cnt > 1 && (g.c - j0 < kTaKeys || (j0 < edge && g.wlo - j0 < kTaKeys))));
                auto clear_v = [&]() -> bool {
                    if (!__all_sync(0xFFFFFFFFu, ta_wait(&sh.v_full[v_stage], v_parity, abort, A.tries))) return false;
                    // positions that only some see, 16 bytes of a value to a thread
                    const int lo0 = max(max(g.wlo, sinks), j0), lo1 = max(g.c, j0);
                    const int n0 = max(0, min(edge, j0 + kTaKeys) - lo0);
                    const int n1 = g.cnt > 1 ? max(0, min(g.end, j0 + kTaKeys) - lo1) : 0;
#pragma unroll 1
                    for (int x = row; x < (n0 + n1) * 8 * kHalves; x += kTaRows) {
                        const int k = x / (8 * kHalves), key = (k < n0 ? lo0 + k : lo1 + (k - n0)) - j0;
                        uint4 *z = reinterpret_cast<uint4 *>(sh.v[v_stage] + (x / 8 % kHalves) * kTaKeys * 128 +
                                                             key * 128 + x % 8 * 16);
                        const uint4 y = *z;
                        const uint32_t bad = not_finite<DT>(y.x) | not_finite<DT>(y.y) | not_finite<DT>(y.z) |
                                             not_finite<DT>(y.w);
                        if (bad & 0x80008000u) {
                            *z = make_uint4(finite_part<DT>(y.x), finite_part<DT>(y.y), finite_part<DT>(y.z),
                                            finite_part<DT>(y.w));
                            *(volatile int *)bad_v = seg_no + 1;
                        }
                    }
                    if (g.end - j0 <= row || (g.wlo - j0 > row && A.sinks - j0 <= row)) {
#pragma unroll
                        for (int d = 0; d < kHalves; ++d) {  // neighbours begin 16 bytes apart: other banks
                            uint4 *z = reinterpret_cast<uint4 *>(sh.v[v_stage] + d * kTaKeys * 128 + row * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) z[(i + row) & 7] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async();
                    return true;
                };
                // a tile's weights and values in two halves of 64 keys: one half's products
                // run while the other half's weights are formed, and 64 scores fit the registers.
                // The weights overwrite those of the tile before, whose values are through: they
                // were issued before these scores, whose commit covers all products before it
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int jh = j0 + h * (kTaKeys / 2);
                    const uint32_t th = ts + (uint32_t)(h * (kTaKeys / 2));
                    if (h == 0) {
                        ok = !(kEarly && clear) || clear_v();
                        ok = ok && __all_sync(0xFFFFFFFFu, ta_wait(&sh.s_full[stream], use & 1u, abort, A.tries));
                        if (!ok) break;
                        tc_fence_after();
                        ok = !(!kEarly && clear) || clear_v();
                        if (!ok) break;
                    }
                    if (warp_works) {
                        uint32_t x[64];
                        tmem_load(th, x);
                        const bool whole = g.c - jh >= 64 && (jh >= low || A.sinks - jh >= 64);
                        if (!__all_sync(0xFFFFFFFFu, whole || !valid)) {
                            const unsigned long long bits = valid ? seen_bits(jh, g.c, low, sinks, path) : 0ull;
                            const uint32_t b0 = (uint32_t)bits, b1 = (uint32_t)(bits >> 32);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (!(b0 & (1u << i))) x[i] = 0xFF800000u;
                                if (!(b1 & (1u << i))) x[32 + i] = 0xFF800000u;
                            }
                            __syncwarp();
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 64; i += 8) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(x[i + 2 * e]),
                                                           __uint_as_float(x[i + 2 * e + 1])));
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * A.scale_log2;
                        // (rows past the last one hold whatever the shared memory held: no vote)
                        if (__any_sync(0xFFFFFFFFu, valid && top > m + (kLift + kTaGrow))) {
                            const float m_new = top > m + kLift ? top - kLift : m;
                            const float f = m_new == -INFINITY ? 1.f : ex2(m - m_new);
                            m = m_new;
                            l2 = make_float2(l2.x * f, l2.y * f);
                            if (h > 0 || !first) {  // O holds the halves before this one
                                uint64_t *done = h > 0 ? &sh.pv_done[stream][0] : &sh.pv_done[stream][1];
                                ok = __all_sync(0xFFFFFFFFu,
                                                ta_wait(done, (h > 0 ? use : use - 1) & 1u, abort, A.tries));
                                if (!ok) break;
                                tc_fence_after();
#pragma unroll 1
                                for (int d = 0; d < DP; d += 32) {
                                    uint32_t o[32];
                                    tmem_load(to + d, o);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                    tmem_store(to + d, o);
                                }
                            }
                        }
                        const float mu = m == -INFINITY ? 0.f : m;
                        const float2 c2 = make_float2(A.scale_log2, A.scale_log2), nm2 = make_float2(-mu, -mu);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t p[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 z = fma2(make_float2(__uint_as_float(x[32 * q + 2 * i]),
                                                                  __uint_as_float(x[32 * q + 2 * i + 1])), c2, nm2);
                                const float2 e = make_float2(ex2(z.x), ex2(z.y));
                                sum[i & 1] = add2(sum[i & 1], e);
                                // rounded to V's type, as operands of one product have to be; the sum
                                // takes them unrounded, so the errors (2^-9 or 2^-12 each) average out
                                p[i] = pack2<DT>(e.x, e.y);
                            }
                            tmem_store(tp + (uint32_t)(h * kPHalf + 16 * q), p);
                        }
                        l2 = add2(l2, add2(sum[0], sum[1]));
                        tmem_wait_store();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(&sh.p_full[stream][h]));
                }
            }
            if (!ok) break;
            base += (uint32_t)s.n;
            float l = l2.x + l2.y;
            if (!valid) l = 0.f, m = -INFINITY;
            if (l != l) m = fmaxf(m, 0.f);  // NaN scores leave m alone: the row's part must not pass for empty

            // ---- the segment's result
            const uint32_t e1 = base - 1u;                   // its last tile
            const int a = MODE == kTaSplitKeys ? (int)(e1 & 1u) : stream;  // a stream that holds a part
            const bool whole_item = s.n == g.nt;
            // a cut item: its first part in this CTA's slot 1, any later one in slot 0
            const long long slot = (long long)blockIdx.x * 2 + (s.i0 == 0 ? 1 : 0);
            constexpr int kCols = MODE == kTaSplitKeys ? DP / 2 : DP;  // columns of O this thread writes
            const int col0 = MODE == kTaSplitKeys ? stream * kCols : 0;
            const bool two = MODE == kTaSplitKeys && s.n > 1;  // both streams hold a part
            float w_a = 1.f, w_b = 0.f;                      // weights of its part and of the other's
            if (MODE == kTaSplitKeys) {
                sh.ml[seg_no & 1][stream][row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(&sh.ml_full));
                ok = ta_wait(&sh.ml_full, seg_no & 1, abort, A.tries);
                ok = ok && ta_wait(&sh.pv_done[a][1], (e1 >> 1) & 1u, abort, A.tries);
                if (two) ok = ok && ta_wait(&sh.pv_done[a ^ 1][1], ((e1 - 1u) >> 1) & 1u, abort, A.tries);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const float2 x = sh.ml[seg_no & 1][a][row], y = sh.ml[seg_no & 1][a ^ 1][row];
                m = fmaxf(x.x, y.x);
                w_a = m == -INFINITY ? 0.f : ex2(x.x - m);
                w_b = m == -INFINITY ? 0.f : ex2(y.x - m);
                l = x.y * w_a + y.y * w_b;
            } else {
                ok = __all_sync(0xFFFFFFFFu, ta_wait(&sh.pv_done[stream][1], e1 & 1u, abort, A.tries));
                if (!ok) break;
            }
            tc_fence_after();
            // a row sees itself at least, so in some part its sum is above 0 unless all its scores
            // are -inf, which then makes it NaN (0 / 0); a part of which it sees nothing has a
            // finite reference all the same, by which the join knows it from rows that do not exist
            if (valid) m = fmaxf(m, -FLT_MAX);
            const float inv = 1.f / l;
            const bool writes = row < rows_used && node < A.N;
            const int head = (MODE == kTaSplitHeads ? 2 * s.hk + stream : s.hk) * A.G + (row - local * A.G);
            const long long orow = ((long long)s.b * A.N + node) * A.Hq + head;
            const int prow = (MODE == kTaSplitKeys ? 0 : stream * rows_used) + row;
            const int rows_cta = rows_used * (MODE == kTaSplitKeys ? 1 : 2);
            const bool any_write = __any_sync(0xFFFFFFFFu, writes);
            const uint32_t o_cols = tmem + lanes + 256u + (uint32_t)col0;
            if (any_write && __any_sync(0xFFFFFFFFu, *(volatile int *)bad_v == seg_no + 1))
                ta_add_not_finite<DT, DP, MODE>(A, s, MODE == kTaSplitHeads ? 2 * s.hk + stream : s.hk, o_cols, col0, a,
                                                two, valid, sinks, edge, low, path, base - (uint32_t)s.n);
            if (any_write) {
#pragma unroll 1
                for (int d = 0; d < kCols; d += 32) {
                    uint32_t o[32];
                    tmem_load(o_cols + (uint32_t)(a * DP + d), o);
                    if (MODE == kTaSplitKeys) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * w_a);
                        if (two) {
                            uint32_t o2[32];
                            tmem_load(o_cols + (uint32_t)((a ^ 1) * DP + d), o2);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(fmaf(__uint_as_float(o2[i]), w_b, __uint_as_float(o[i])));
                        }
                    }
                    if (!writes) {
                    } else if (whole_item) {
                        uint4 *dst = reinterpret_cast<uint4 *>(A.out + orow * A.D + col0 + d);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            if (col0 + d + i < A.D) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = valid ? pack2<DT>(__uint_as_float(o[i + 2 * e]) * inv,
                                                             __uint_as_float(o[i + 2 * e + 1]) * inv)
                                                 : 0u;
                                dst[i / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                    } else if (valid) {
                        uint4 *dst = reinterpret_cast<uint4 *>(A.part_o + (slot * rows_cta + prow) * A.D + col0 + d);
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (col0 + d + i < A.D) dst[i / 4] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(&sh.o_free[stream]));
            if (writes && col0 == 0) {
                if (whole_item) {
                    if (A.lse) A.lse[orow] = ta_lse(valid, m, l);
                } else {
                    A.part_ml[slot * rows_cta + prow] = make_float2(m, l);
                }
            }
        }
        if (!ok) *abort = 1;
    }

    if (warp < 8 && fewer) {  // the nodes past every row tile (past the counts) see nothing
        const int npt = ta_nodes<MODE>(A);
        for (int b = blockIdx.x; b < A.B; b += gridDim.x) {
            const int2 lens = ta_lens(A, b);
            const int n0 = lens.y > 0 ? min(A.N, ta_row_tiles<MODE>(A, lens.y) * npt) : 0;
            if (n0 >= A.N) continue;
            const long long r0 = ((long long)b * A.N + n0) * A.Hq, r1 = ((long long)b * A.N + A.N) * A.Hq;
            uint4 *o = reinterpret_cast<uint4 *>(A.out);
#pragma unroll 1
            for (long long i = r0 * A.D / 8 + threadIdx.x; i < r1 * A.D / 8; i += 256)
                o[i] = make_uint4(0u, 0u, 0u, 0u);
            if (A.lse)
#pragma unroll 1
                for (long long i = r0 + threadIdx.x; i < r1; i += 256) A.lse[i] = -INFINITY;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTaWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && sh.abort) flag(A.status, SPEC_DEV_TIMEOUT);
}

// The parts of an item that cuts fell into, joined in the order of the keys.
// joins[j]: the first cut of an item lies at CTA j's first unit; its parts are
// slot 1 of the CTA before, where it begins, and slot 0 of CTA j and those after.
// 16 lanes per row, two vectors of four columns each: bound by the latency of three
// dependent loads at few rows (3.4 us of a call of one token at one request) and
// by instructions at many (10 us at 64 nodes and 64 requests); a warp per row
// took 16.7 us there, 8 lanes 9.5 but 3 us more with 20 parts of 64 rows.
template <int DT>
__global__ void __launch_bounds__(256) tree_attn_join(TaArgs A, int rows_used, int rows_cta, int mode) {
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
    const bool works = prow < rows_cta && node < A.N;
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
            w = ex2(x.x - m);
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
    if (lane == 0 && A.lse) A.lse[orow] = ta_lse(some, m, l);
}

// ------------------------------------------------------------------ host

// A 4D tensor map over 16-bit elements, 64 of them (128 bytes, the swizzle
// span) wide; elements past an extent read as zero.
static bool ta_tmap(CUtensorMap *tm, int dtype, const void *base, const cuuint64_t (&dims)[4],
                    const cuuint64_t (&strides)[3], cuuint32_t box1, cuuint32_t box2) {
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
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a stream: whole nodes, at most 128 rows.  Up to one stream's worth
// the streams share the rows and split the keys, or take a key head each; more
// nodes are spread evenly over the streams of as few row tiles as hold them.
struct TaRows {
    int np, used, cta, mode;
};
static TaRows ta_rows(int N, int G, bool pairs) {
    TaRows r;
    const int most = kTaRows / G;
    r.mode = N > most ? kTaSplitRows : pairs ? kTaSplitHeads : kTaSplitKeys;
    const int tiles = (N + 2 * most - 1) / (2 * most), nodes = (N + tiles - 1) / tiles;
    r.np = r.mode == kTaSplitRows ? (nodes + 1) / 2 : N;
    r.used = r.np * G;
    r.cta = r.used * (r.mode == kTaSplitKeys ? 1 : 2);
    return r;
}

struct TaLayout {
    size_t o, ml, joins, total;
};
static TaLayout ta_layout(int N, int Hq, int heads, int D) {
    TaLayout L;
    const size_t rows = (size_t)kTaMaxCtas * 2 * ta_rows(N, Hq / heads, true).cta;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    L.o = 0;
    L.ml = up(rows * (size_t)D * sizeof(float));
    L.joins = up(L.ml + rows * sizeof(float2));
    L.total = up(L.joins + (size_t)kTaMaxCtas * sizeof(int4));
    return L;
}

template <int DT, int DP, int MODE>
static spec_status_t ta_launch(const TaArgs &A, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                               const TaRows &r, int ctas, int dev, cudaStream_t s) {
    constexpr size_t smem = sizeof(TaShared<DP, MODE>) + 1024;
    static_assert(smem <= 232448, "shared memory of a CTA");
    static bool ready[64] = {};
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(tree_attn<DT, DP, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess)
            return SPEC_ERR_CUDA;
        ready[dev] = true;
    }
    const spec_status_t st =
        launch_pdl(tree_attn<DT, DP, MODE>, dim3((unsigned)ctas), dim3(kTaThreads), smem, s, q, k, v, A);
    if (st != SPEC_OK) return st;
    constexpr int rows = 256 / kTaJoinLanes;
    return launch_pdl(tree_attn_join<DT>, dim3((unsigned)ctas, (unsigned)((r.cta + rows - 1) / rows)), dim3(256), 0, s,
                      A, r.used, r.cta, MODE);
}

template <int DT, int DP>
static spec_status_t ta_launch_mode(const TaArgs &A, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                    const TaRows &r, int ctas, int dev, cudaStream_t s) {
    switch (r.mode) {
    case kTaSplitRows: return ta_launch<DT, DP, kTaSplitRows>(A, q, k, v, r, ctas, dev, s);
    case kTaSplitHeads: return ta_launch<DT, DP, kTaSplitHeads>(A, q, k, v, r, ctas, dev, s);
    default: return ta_launch<DT, DP, kTaSplitKeys>(A, q, k, v, r, ctas, dev, s);
    }
}

} // namespace sv

extern "C" {

size_t spec_tree_attention_workspace_bytes(int B, int N, int Hq, int heads, int head_dim) {
    if (B < 1 || B >= (1 << 16) || N < 1 || N > SPEC_MAX_TREE || heads < 1 || heads > 1024 || Hq < heads ||
        Hq % heads || Hq / heads > 64 || head_dim < 8 || head_dim % 8 || head_dim > SPEC_MAX_HEAD_DIM)
        return 0;
    return sv::ta_layout(N, Hq, heads, head_dim).total;
}

spec_status_t spec_tree_attention(const void *q, long long q_stride_b, long long q_stride_n,
                                  long long q_stride_h, const spec_pages_t *pages,
                                  const int32_t *page_table, const int32_t *cache_len,
                                  const int32_t *parent, const int32_t *node_count, int B, int N,
                                  int Hq, int max_pages, float scale, int window, int sinks,
                                  void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  uint32_t *dev_status, void *stream) {
    sv::Pool P;
    const spec_status_t st = sv::make_pool(pages, P);
    if (st != SPEC_OK) return st;
    if (pages->dtype != SPEC_DTYPE_BF16 && pages->dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    const int D = pages->head_dim, H = pages->heads;
    const size_t need = spec_tree_attention_workspace_bytes(B, N, Hq, H, D);
    if (!q || !page_table || !cache_len || !out || need == 0 || pages->layers != 1 || max_pages < 1 ||
        ((uintptr_t)q & 15) || ((uintptr_t)out & 15) || window < 0 || sinks < 0 || !(scale > 0.f) ||
        !(scale < 3.0e38f))
        return SPEC_ERR_INVALID_ARG;
    const long long qst[3] = {q_stride_h, q_stride_n, q_stride_b};
    const int qext[3] = {Hq, N, B};
    for (int i = 0; i < 3; ++i)
        if (qst[i] % 8 || qst[i] < (qext[i] > 1 ? D : 0)) return SPEC_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need) return SPEC_ERR_WORKSPACE;
    int dev = 0;
    static int sms[64] = {};
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
    if (sms[dev] == 0 && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SPEC_ERR_CUDA;
    const int ctas = sms[dev] < sv::kTaMaxCtas ? sms[dev] : sv::kTaMaxCtas;

    // A key head per stream once there is one for every CTA: the streams then share
    // nothing but the CTA, where streams that divide the keys meet at the end of
    // every (request, head), which costs most where those are short.  us, by heads /
    // by keys, 8 key heads:
    //   head_dim 64, window 128, 9 nodes:  B = 24 13.7 / 16.3, 64 19.3 / 24.6, 512 90 / 121
    //   head_dim 128, 500 tokens, 1 node:  B = 32 18.3 / 22.5;  window 1024, 9 nodes: 256 194 / 211
    //   head_dim 128, 4096 tokens, 9 nodes: B = 32 96 / 96, 256 656 / 664
    // With fewer heads a unit of twice the work is cut more coarsely:
    //   head_dim 128, 500 tokens, 1 node:  B = 16 14.5 / 13.3, 1 10.7 / 10.4; 20000 tokens, 2 nodes: B = 1 29.5 / 26.8
    const bool pairs = H % 2 == 0 && (long long)B * H >= ctas;
    const sv::TaRows r = sv::ta_rows(N, Hq / H, pairs);
    const sv::TaLayout L = sv::ta_layout(N, Hq, H, D);
    sv::TaArgs A = {};
    A.table = page_table;
    A.len = cache_len;
    A.parent = parent;
    A.node_count = node_count;
    A.B = B;
    A.N = N;
    A.Hq = Hq;
    A.H = r.mode == sv::kTaSplitHeads ? H / 2 : H;
    A.G = Hq / H;
    A.D = D;
    A.max_pages = max_pages;
    A.num_pages = P.num_pages;
    A.page = P.page;
    A.page_shift = P.page_shift;
    A.window = window;
    A.sinks = sinks;
    A.np = r.np;
    A.box = P.page < sv::kTaKeys ? P.page : sv::kTaKeys;
    A.scale_log2 = scale * 1.44269504089f;
    A.out = static_cast<uint16_t *>(out);
    A.lse = lse;
    char *ws = static_cast<char *>(workspace);
    A.part_o = reinterpret_cast<float *>(ws + L.o);
    A.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
    A.joins = reinterpret_cast<int4 *>(ws + L.joins);
    A.v = static_cast<const uint16_t *>(pages->v);
    A.v_page = pages->page_stride;
    A.v_token = pages->token_stride;
    A.v_head = pages->head_stride;
    A.status = dev_status;
    A.tries = sv::g_diag_timeout ? 0u : sv::kTaTries;

    CUtensorMap tq, tk, tv;
    // an extent of one is never stepped over: any valid stride stands for it
    auto bytes = [&](long long stride, int extent) { return (cuuint64_t)(extent > 1 ? stride : D) * 2; };
    const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t qs[3] = {bytes(q_stride_h, Hq), bytes(q_stride_n, N), bytes(q_stride_b, B)};
    const cuuint64_t kd[4] = {(cuuint64_t)D, (cuuint64_t)P.page, (cuuint64_t)H, (cuuint64_t)P.num_pages};
    const cuuint64_t ks[3] = {bytes(pages->token_stride, P.page), bytes(pages->head_stride, H),
                              bytes(pages->page_stride, P.num_pages)};
    if (!sv::ta_tmap(&tq, pages->dtype, q, qd, qs, (cuuint32_t)A.G, (cuuint32_t)r.np) ||
        !sv::ta_tmap(&tk, pages->dtype, pages->k, kd, ks, (cuuint32_t)A.box, 1) ||
        !sv::ta_tmap(&tv, pages->dtype, pages->v, kd, ks, (cuuint32_t)A.box, 1))
        return SPEC_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf = pages->dtype == SPEC_DTYPE_BF16;
    if (bf)
        return D <= 64 ? sv::ta_launch_mode<SPEC_DTYPE_BF16, 64>(A, tq, tk, tv, r, ctas, dev, s)
                       : sv::ta_launch_mode<SPEC_DTYPE_BF16, 128>(A, tq, tk, tv, r, ctas, dev, s);
    return D <= 64 ? sv::ta_launch_mode<SPEC_DTYPE_F16, 64>(A, tq, tk, tv, r, ctas, dev, s)
                   : sv::ta_launch_mode<SPEC_DTYPE_F16, 128>(A, tq, tk, tv, r, ctas, dev, s);
}

} // extern "C"
