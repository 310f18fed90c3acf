// tree_attn4.cu -- attention of drafted trees over a 4-bit paged cache on the
// sm_103a tensor cores.
//
// Mathematics: that of tree_attn.cu (one pass over the keys with a reference near
// the running maximum, parts over disjoint keys joined), on keys and values (c -
// 8) s with a 4-bit code c and a scale s per 32 channels.  References are kept unscaled, and where
// float32 holds their scaled form to 1 or more they are taken off the scores before scaling, so that large
// scores weigh what their exact difference says wherever the keys lie.  Keys and values are formed exactly:
// a code is put into the low mantissa bits of a 16-bit float of fixed exponent
// (which then is 128 + c in bfloat16, 16 + c in float16), and one fused
// multiply-add with s and -136 s, or s/4 and -6 s, gives (c - 8) s or a quarter of
// it; all of these numbers fit the type.
//
// What bounds it.  A key and value of a head of 128 are 136 bytes, so at the copy
// rate an SM has 784 cycles (at 1.92 GHz) for a tile of 128 keys, in which 32768
// codes become operands.  Written to shared memory and read back by the tensor
// cores they would take its port 768 cycles alone.  So the products are turned
// around: K and V^T are the A operands, which tcgen05.mma takes from the tensor
// memory, where a thread writes 32 bits a column straight from its registers.
//     S^T = K Q^T    [128 keys  x rows]     A: a lane per key, two channels a column
//     O^T = V^T P^T  [channels  x rows]     A: a lane per channel, two keys a column
// with the rows (nodes x query heads of the group) as the N dimension, 16 to 64 of
// them, so that decoding single tokens multiplies 16 columns and not 128 padded
// rows.  The cache's layout follows from this: a thread's codes of a key are 16 bytes
// per 32 channels, those of a channel 4 bytes per 8 tokens, each without bank
// conflicts, and the scales of a warp's 32 channels of V are the same for all lanes.
//
// One CTA per SM.  Eight warps form the weights, two warpgroups with a tile each in turn (of 64 columns: half of every
// tile's), four warps unpack K and four V (of 16 columns: eight each, in turn), two load, a bulk copy for each block of
// the cache, one issues the products and one schedules.  Tiles of keys go round two or three buffers of K, V, S and P, so
// the stages of consecutive tiles overlap.  Heads of up to 64 are taken in pairs (the lanes of V^T are two heads'
// channels; the quarter of the product that mixes them is not read).  More rows than a tile has are cut into row tiles.
//
// Measured: 64 single tokens of 32 query heads and 8 key heads of 128 after up to 8192 positions, 141 us for their
// 428 MB, 3.1 TB/s or 45 % of a copy's rate (the same with 16 bits a number: 248 us).  16 nodes after 131071 positions:
// 78.8 us (99).  Chains of 9 of 32 requests, up to 4096 positions, 8 key heads of 64: 65 us (60.5: two row tiles, each
// of which unpacks every key; chains of 8 fit in one, 42 us against 56).  With more rows, or in short segments, 16 bits
// are faster: 64 requests of 64 nodes after up to 2000 positions 342 us (130), 512 of 9 with a window of 128 212 (103).
// What bounds it is the
// issuing of instructions: 4180 warp instructions to a tile of 128 keys, of which a code's pair takes three (a shift, the
// mask, the multiply-add); 68 % of the issue slots, 50 % of the integer pipe, the rest lost to the barriers between the
// stages.  The roles run from one instruction cache, so a shorter loop gains more than one unrolled.
#include "attn_plan.cuh"
#include "cache4.cuh"

#include <climits>

namespace sv {

struct T4Args {
    TaArgs a;             // a.H: packs of heads
    const uint8_t *data;  // the pool
    long long page_st, head_st;
    int heads;            // key heads
    int C, groups;        // channels kept and groups of 32 of them
    int block, block_shift, bytes;  // tokens of a block, its bytes
    int value[kTaKeys / 8];         // where a tile's values lie in a head's blocks, 8 tokens at a time
};

template <int DP, int PACK, int RP> struct T4Cfg {
    static constexpr int kCols = PACK * RP;              // rows of all heads of a pack
    static constexpr int kRowP = kCols * 2;              // bytes of a key's weights
    static constexpr int kStage = PACK * DP * 136;       // one tile, packed
    static constexpr int kStages = kCols == 64 ? 6 : 8;
    static constexpr int kQ = PACK * RP * DP * 2;
    static constexpr int kW = kCols < 32 ? kCols : 32;   // columns of a softmax warp
    // two warpgroups of softmax: a tile each in turn, or with 64 columns half of every tile's
    static constexpr int kStreams = kCols > 32 ? 1 : 2;
    // K and V: a warpgroup each, or two in turn with 16 columns, where the softmax leaves most of the issue slots to
    // them (64 requests of 8192 positions: 152 us so, 182 with one).  With more columns a second one only takes
    // registers and turns from the softmax (16 nodes after 131071 positions: 122 us against 85 with one).
    static constexpr int kTurns = kCols == 16 ? 2 : 1;
    static constexpr int kSoft = 8, kV = kSoft + 4 * kTurns;  // softmax warps, then K's, then V's
    static constexpr int kLoad = kV + 4 * kTurns, kMma = kLoad + 2, kPlan = kLoad + 3;  // (two warps load)
    static constexpr int kWarps = kLoad + 4, kThreads = kWarps * 32;
    // registers: at launch as many as fit; then the softmax takes what the others give back
    static constexpr int kRegs = kTurns == 2 ? 72 : 96;
    static constexpr int kRegSoft = kTurns == 2 ? 104 : 136, kRegUnpack = kTurns == 2 ? 56 : 72;
    static constexpr int kRegHelp = kTurns == 2 ? 72 : 64;
    static_assert(kSoft * kRegSoft + 8 * kTurns * kRegUnpack + 4 * kRegHelp <= kWarps * kRegs &&
                      kWarps * kRegs * 32 <= 65536,
                  "more registers than the CTA has: setmaxnreg would wait for ever");
    // buffers of K, V, S and P: three where the tensor memory has room for them, so that a warpgroup need not
    // wait for the products of the other's tile
    static constexpr uint32_t kBufs = kCols == 16 ? 3 : 2;
    // tensor-memory columns: 64 for each K and V, then S, then an O for each stream
    static constexpr uint32_t kTK = 0, kTV = kBufs * 64, kTS = 2 * kTV, kSStep = kBufs == 3 ? 16 : 64;
    static constexpr uint32_t kTO = kTS + (kBufs == 3 ? 64 : 128), kOStep = kBufs == 3 ? 32 : 64;
    static_assert(kTS + kBufs * kSStep <= kTO && kTO + (kCols > 32 ? kCols : kOStep + kCols) <= 512, "tensor memory");
    static constexpr int kSwizzle = kCols == 64 ? 2 : kCols == 32 ? 4 : 6;  // 128, 64 or 32 bytes
};

template <int DP, int PACK, int RP> struct T4Shared {
    using C = T4Cfg<DP, PACK, RP>;
    uint8_t q[kTaSlots][C::kQ];
    uint8_t p[C::kBufs][kTaKeys * C::kRowP];
    uint8_t tile[C::kStages][C::kStage];     // per head: its blocks, as they lie in memory
    const uint8_t *places[2][32];            // of a loading warp: where the next blocks lie in memory
    uint4 scale[4 * C::kTurns][32];                      // of a V warp: V's multipliers and addends for its keys
    // per warp: the largest scores so far as references, what z adds for them, and the factors of the last change
    float ref[C::kSoft][C::kW], m[C::kSoft][C::kW], f[C::kSoft][C::kW];
    float top[C::kSoft][C::kW], sum[C::kSoft][C::kW];
    float w[2][C::kCols];                    // the streams' factors in the result
    long long row[C::kCols];                 // where a row goes: twice its first element (of out, or of the parts), one
                                             // more if it sees nothing; -1: nowhere
    long long incl[kTaChunks];
    SegSlot seg[kTaSlots];
    uint64_t seg_full[kTaSlots], path_full[kTaSlots], seg_free[kTaSlots], q_full[kTaSlots], q_free[kTaSlots];
    uint64_t full[C::kStages], empty[C::kStages];
    uint64_t s_ready[C::kBufs], s_full[C::kBufs];          // K is there and the scores before are read; scores are there
    uint64_t pv_ready[C::kBufs], pv_done[C::kBufs];        // V and the weights are there; their product is in O
    uint64_t o_free, done;
    uint32_t tmem_base;
    int abort;
};

// ------------------------------------------------------------------ PTX

// ta_wait in one statement: the compiler's code around its loop doubles the 67 cycles of a look that succeeds at
// once, and a tile's stages wait for each other half a dozen times.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, int *abort, uint32_t tries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 n, a;\n\t"
        "mov.u32 n, %4;\n\t"
        "mov.u32 %0, 1;\n\t"
        "LOOK%=: mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE%=;\n\t"
        "ld.volatile.shared.u32 a, [%3];\n\t"
        "setp.ne.u32 p, a, 0;\n\t"
        "@p bra GIVEUP%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 p, n, 0;\n\t"
        "@p bra LOOK%=;\n\t"
        "mov.u32 a, 1;\n\t"
        "st.volatile.shared.u32 [%3], a;\n\t"
        "GIVEUP%=: mov.u32 %0, 0;\n\t"
        "DONE%=:\n\t}"
        : "=&r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(smem_u32(abort)), "r"(tries)
        : "memory");
    return ok != 0;
}

// A barrier of THREADS threads, the softmax warps or a warpgroup of them; whether any of them says so.
template <int THREADS> __device__ __forceinline__ bool meet(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "n"(THREADS)
        : "memory");
    return r != 0;
}
template <int N> __device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Shared-memory descriptor of the weights as the B operand [keys x rows]: the rows (N) are
// contiguous, kRowP bytes to a key, which is the swizzle's span; 8 keys an atom, the next 8
// keys right behind (stride byte offset).
template <int ROWP, int SWIZZLE> __device__ __forceinline__ uint64_t p_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1u << 16;
    d |= (uint64_t)((uint32_t)(ROWP * 8) >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)SWIZZLE << 61;
    return d;
}

__device__ __forceinline__ uint32_t hfma2(int dt, uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if (dt == SPEC_DTYPE_BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// The bits of 128 (bfloat16) or 16 (float16) in both halves, kept in a register: as a known constant beside the
// mask it would take an instruction of its own, since one instruction holds one constant (64 of 1176
// instructions a tile for each of K and V).
template <int DT> __device__ __forceinline__ uint32_t code_base() {
    uint32_t x;
    asm volatile("mov.b32 %0, %1;" : "=r"(x) : "n"(DT == SPEC_DTYPE_BF16 ? 0x43004300 : 0x4C004C00));
    return x;
}
// Two codes of a word as numbers, times a scale (see the head of the file): pair i of the word
// lies at bits 4 i and 4 i + 16.
template <int DT>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i, uint32_t s, uint32_t b, uint32_t base) {
    uint32_t x;  // (y & mask) | base
    if (DT == SPEC_DTYPE_BF16) {
        asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(x) : "r"(w >> (4 * i)), "r"(base));
    } else {
        const uint32_t y = i == 0 ? w << 6 : i == 1 ? w << 2 : i == 2 ? w >> 2 : w >> 6;
        asm("lop3.b32 %0, %1, 0x03C003C0, %2, 0xEA;" : "=r"(x) : "r"(y), "r"(base));
    }
    return hfma2(DT, x, s, b);
}
// The multiplier and addend of unpack_pair for the scale(s) lo and hi.
template <int DT> __device__ __forceinline__ uint2 unpack_scale(float lo, float hi) {
    if (DT == SPEC_DTYPE_BF16) return make_uint2(pack2<DT>(lo, hi), pack2<DT>(-136.f * lo, -136.f * hi));
    return make_uint2(pack2<DT>(0.25f * lo, 0.25f * hi), pack2<DT>(-6.f * lo, -6.f * hi));
}

// ------------------------------------------------------------------ the kernel

constexpr float kLift = 7.f;  // weights up to 2^15: those 2^-29 below the maximum are still normal in float16

// The factor of the scores, of which float16 has a quarter (see unpack_scale).
template <int DT> constexpr float kKeyPart = DT == SPEC_DTYPE_F16 ? 4.f : 1.f;
template <int DT> __host__ __device__ __forceinline__ float t4_scale(const TaArgs &A) {
    return A.scale_log2 * kKeyPart<DT>;
}

template <int DT, int DP, int PACK, int RP>
__global__ void __launch_bounds__((T4Cfg<DP, PACK, RP>::kThreads), 1)
    tree_attn4(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ T4Args T) {
    using C = T4Cfg<DP, PACK, RP>;
    using Sh = T4Shared<DP, PACK, RP>;
    extern __shared__ uint8_t t4_raw[];
    // (an offset, so that the compiler keeps knowing the address to be in shared memory)
    Sh &sh = *reinterpret_cast<Sh *>(t4_raw + ((0u - smem_u32(t4_raw)) & 1023u));
    const TaArgs &A = T.a;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    constexpr int kCols = C::kCols, kStages = C::kStages, kW = C::kW, kSoft = C::kSoft, kStreams = C::kStreams,
                  kTurns = C::kTurns;
    constexpr uint32_t kBufs = C::kBufs;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kTaSlots; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.path_full[i], 1);
            mbar_init(&sh.seg_free[i], kSoft + 3);
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_free[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 8);
        }
        for (int i = 0; i < (int)C::kBufs; ++i) {
            mbar_init(&sh.s_ready[i], 4 + kSoft / kStreams);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.pv_ready[i], 4 + kSoft / kStreams);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.o_free, kSoft);
        mbar_init(&sh.done, 1);
        sh.abort = A.tries == 0;  // (a wait in vain then gives up at its first look)
        fence_mbar_init();
        tma_prefetch_map(&tm_q);
    }
    // the rows of Q past the last one stay 0
    for (int i = threadIdx.x; i < (int)sizeof(sh.q) / 16; i += C::kThreads)
        reinterpret_cast<uint4 *>(sh.q)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    if (warp == C::kMma) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    pdl_trigger();
    pdl_wait();
    Walk<kTaSplitKeys> w;
    if (warp == C::kPlan) w.fetch(A, 0);
    bool fewer = false;
    if (threadIdx.x < kTaChunks) fewer = ta_sum_units<kTaSplitKeys>(A, sh.incl);
    tc_fence_before();
    fewer = __syncthreads_or(fewer) != 0;
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
    volatile int *abort = &sh.abort;
    long long total = 0;
    for (int i = 31; i < kTaChunks; i += 32) total += sh.incl[i];
    const long long run = ta_div(total + gridDim.x - 1, gridDim.x);
    const long long u_first = min(total, (long long)blockIdx.x * run), u_last = min(total, u_first + run);
    const uint32_t tiles = (uint32_t)(u_last - u_first);

    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity & 1u, &sh.abort, A.tries)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(bar));
    };
    // segment k, or nothing when the wait for it ran out
    auto take = [&](uint64_t *bars, int k) -> const SegSlot * {
        return wait(&bars[k % kTaSlots], (uint32_t)(k / kTaSlots)) ? &sh.seg[k % kTaSlots] : nullptr;
    };

    if (C::kRegHelp < C::kRegs && warp >= C::kLoad) fewer_registers<C::kRegHelp>();
    if (warp == C::kPlan) {  // ------------------------------------------- scheduling
        ta_schedule<kTaSplitKeys>(A, w, sh.incl, sh.seg, sh.seg_full, sh.path_full, sh.seg_free, u_first, u_last, run,
                                  abort);
    } else if (warp == C::kLoad || warp == C::kLoad + 1) {  // ---------------- loads
        const uint32_t turn = (uint32_t)(warp - C::kLoad);   // the warps take the tiles in turn
        const int recs = kTaKeys >> T.block_shift;           // blocks of a head's tile
        const int nb = PACK * recs, ahead = 32 / nb;         // blocks of a tile, tiles whose pages are fetched at once
        const int slot = lane % nb / recs, rec = lane % recs;  // of the pages that the lane fetches
        const uint8_t **places = sh.places[turn];
        uint32_t e = 0, stage = 0, fill = 0;
        int seg_no = 0;
        bool ok = true;
        for (; ok; ++seg_no) {
            const SegSlot *sp = take(sh.seg_full, seg_no);
            if (!sp || sp->s.n == 0) break;
            const Seg s = sp->s;
            arrive(&sh.seg_free[seg_no % kTaSlots]);
            const int qb = seg_no % kTaSlots;
            if (turn == 0 && seg_no >= kTaSlots && !wait(&sh.q_free[qb], (uint32_t)(seg_no / kTaSlots - 1))) break;
            if (turn == 0 && elect_one()) {
                mbar_expect_tx(&sh.q_full[qb], (uint32_t)(PACK * (DP / 64) * A.np * A.G * 128));
#pragma unroll
                for (int x = 0; x < PACK; ++x)
#pragma unroll
                    for (int h = 0; h < DP / 64; ++h)
                        tma_load_4d(sh.q[qb] + (x * (DP / 64) + h) * RP * 128, &tm_q, h * 64,
                                    (s.hk * PACK + x) * A.G, s.node0, s.b, &sh.q_full[qb]);
            }
            __syncwarp();
            const int head = s.hk * PACK + slot, i_end = s.i0 + s.n;
            const int have = min(nb, (T.heads - s.hk * PACK) * recs);  // blocks of heads that there are
            const int *row = A.table + s.b * A.row_b + head * A.row_h;
            // the place in memory of this lane's block of tile i0 + lane / nb; that of any block where no node sees it
            auto fetch = [&](int i0) -> const uint8_t * {
                const int i = i0 + lane / nb;
                if (i >= i_end || head >= T.heads) return T.data;
                const int j = s.g.tile(i) * kTaKeys + (rec << T.block_shift);  // its first position
                if (j >= s.g.end || (s.g.wlo - j >= T.block && j >= A.sinks)) return T.data;
                int p = __ldcg(row + (j >> A.page_shift));
                if ((unsigned)p >= (unsigned)A.num_pages) {
                    flag(A.status, SPEC_DEV_BAD_PAGE);
                    p = 0;
                }
                return T.data + p * T.page_st + head * T.head_st + ((j & (A.page - 1)) >> T.block_shift) * T.bytes;
            };
            int base = s.i0 - ahead;
            const uint8_t *next = T.data;
            for (int i = s.i0; i < i_end; ++i, ++e) {
                if (i == base + ahead) {
                    // at first these blocks' places and then the next ones', one load ahead
#pragma unroll 1
                    for (int at = i == s.i0 ? i : i + ahead; at <= i + ahead; at += ahead) {
                        if (at > i) {
                            __syncwarp();
                            places[lane] = next;
                            __syncwarp();
                        }
                        next = fetch(at);
                    }
                    base = i;
                }
                if ((e & 1u) != turn) {
                    if (++stage == kStages) stage = 0, ++fill;
                    continue;
                }
                if (fill > 0 && !wait(&sh.empty[stage], fill - 1)) {
                    ok = false;
                    break;
                }
                // (One lane issues, in a loop: copies by a lane each are issued one after the other all the same.  A copy
                // takes the warp 100 cycles and more, so blocks come whole, codes and scales.  What an odd last head's
                // place in a pair holds is finite whatever its bits are, and meets rows of zeros that nobody reads.)
                if (elect_one()) {
                    const uint8_t *const *from = places + (i - base) * nb;
                    uint8_t *to = sh.tile[stage];
                    mbar_expect_tx(&sh.full[stage], (uint32_t)(have * T.bytes));
#pragma unroll 4
                    for (int r = 0; r < have; ++r, to += T.bytes) bulk_g2s(to, from[r], (uint32_t)T.bytes, &sh.full[stage]);
                }
                __syncwarp();
                if (++stage == kStages) stage = 0, ++fill;
            }
        }
        // every copy has landed before the CTA may exit
        for (uint32_t x = turn; x < (uint32_t)kStages; x += 2) {
            const uint32_t n = fill + (x < stage ? 1u : 0u);
            if (n > 0) mbar_wait_bounded(&sh.full[x], (n - 1) & 1u, kTaWaitNs);
        }
        for (int x = 0; x < kTaSlots && turn == 0; ++x) {
            const int n = (seg_no + kTaSlots - 1 - x) / kTaSlots;
            if (n > 0) mbar_wait_bounded(&sh.q_full[x], (uint32_t)(n - 1) & 1u, kTaWaitNs);
        }
        __syncwarp();
    } else if (warp == C::kMma) {  // -------------------------------------- products
        constexpr uint32_t kIdS = (ta_idesc<DT>(RP, false)), kIdO = ta_idesc<SPEC_DTYPE_F16>(kCols, true);
        const uint64_t q_desc = umma_desc_sw128(smem_u32(sh.q[0]));
        const uint64_t w_desc = p_desc<C::kRowP, C::kSwizzle>(smem_u32(sh.p[0]));
        int s_seg = 0, s_left = 0, v_seg = 0, v_left = 0;
        bool ok = true;
        uint32_t fresh = 0;  // streams whose next values are the segment's first
        // The next tile's scores go before a tile's values, whose weights take longer.  (Groups of channels that
        // the head does not have were written with another's codes, and meet zeros of Q.)
#pragma unroll 1
        for (uint32_t e = 0; e <= tiles && tiles > 0 && ok; ++e) {
            if (e < tiles) {
                const uint32_t buf = e % kBufs, use = e / kBufs;
                if (s_left == 0) {
                    if (!take(sh.seg_full, s_seg)) break;
                    s_left = __shfl_sync(0xFFFFFFFFu, sh.seg[s_seg % kTaSlots].s.n, 0);
                    if (!wait(&sh.q_full[s_seg % kTaSlots], (uint32_t)(s_seg / kTaSlots))) break;
                    ++s_seg;
                }
                const int qb = (s_seg - 1) % kTaSlots;
                if (!wait(&sh.s_ready[buf], use)) break;
                tc_fence_after();
                --s_left;
                const uint32_t d = tmem + C::kTS + buf * C::kSStep, a = tmem + C::kTK + buf * 64;
                const uint64_t qd = q_desc + (uint64_t)(qb * (C::kQ / 16));
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < PACK; ++x)
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k)
                            mma_ts(d + (uint32_t)(x * RP), a + (uint32_t)(x * DP / 2 + k * 8),
                                   qd + (uint64_t)((x * RP * DP * 2 + (k >> 2) * (RP * 128) + (k & 3) * 32) / 16), kIdS,
                                   k > 0 ? 1u : 0u);
                    umma_commit(&sh.s_full[buf]);
                    if (s_left == 0) umma_commit(&sh.q_free[qb]);
                }
                __syncwarp();
            }
            if (e > 0) {
                const uint32_t buf = (e - 1) % kBufs, use = (e - 1) / kBufs, stream = kStreams == 2 ? (e - 1) & 1u : 0u;
                if (v_left == 0) {
                    v_left = __shfl_sync(0xFFFFFFFFu, sh.seg[v_seg % kTaSlots].s.n, 0);
                    if (v_seg > 0 && !wait(&sh.o_free, (uint32_t)(v_seg - 1))) break;
                    ++v_seg;
                    fresh = 3;
                }
                if (!wait(&sh.pv_ready[buf], use)) break;
                tc_fence_after();
                const uint32_t d = tmem + C::kTO + stream * C::kOStep, a = tmem + C::kTV + buf * 64;
                const uint64_t wd = w_desc + (uint64_t)(buf * (uint32_t)(kTaKeys * C::kRowP / 16));
                const uint32_t add = (fresh >> stream) & 1u ? 0u : 1u;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kTaKeys / 16; ++k)
                        mma_ts(d, a + (uint32_t)(k * 8), wd + (uint64_t)(k * C::kRowP), kIdO, k > 0 ? 1u : add);
                    umma_commit(&sh.pv_done[buf]);
                }
                __syncwarp();
                fresh &= ~(1u << stream);
                if (--v_left == 0) arrive(&sh.seg_free[(v_seg - 1) % kTaSlots]);
            }
        }
        // every MMA has finished before the TMEM is freed
        if (elect_one()) umma_commit(&sh.done);
        mbar_wait_bounded(&sh.done, 0u, kTaWaitNs);
        __syncwarp();
    } else if (warp >= C::kV && warp < C::kLoad) {  // ------------------------- V
        fewer_registers<C::kRegUnpack>();
        const uint32_t turn = kTurns == 2 ? (uint32_t)(warp - C::kV) >> 2 : 0u;  // the warpgroups take the tiles in turn
        const int quad = warp & 3, slot = quad * 32 / DP, ch = (quad * 32 + lane) % DP;
        const bool works = slot < PACK && ch - lane < T.C;  // the warp's lanes alike
        const int t = 4 * lane;                             // the keys whose scales the lane unpacks
        const int head_off = slot * (kTaKeys / 16 * 17) * T.C, word_off = head_off + ch * 4;
        const int scale_off = head_off + (t >> T.block_shift) * T.bytes + T.block * (T.C + T.groups + (ch >> 5)) +
                              (t & (T.block - 1));
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + C::kTV;
        uint4 *scale = sh.scale[warp - C::kV];
        const uint32_t zero = code_base<SPEC_DTYPE_F16>();  // code 0
        for (uint32_t e = turn, stage = turn, fill = 0, buf = turn, use = 0; e < tiles; e += kTurns) {
            if (!wait(&sh.full[stage], fill)) break;
            const uint8_t *tile = sh.tile[stage];
            if (works) {
                const uint32_t x = *reinterpret_cast<const uint32_t *>(tile + scale_off);
                const uint2 a = unpack_scale<SPEC_DTYPE_F16>(scale_of(x & 255u), scale_of((x >> 8) & 255u));
                const uint2 b = unpack_scale<SPEC_DTYPE_F16>(scale_of((x >> 16) & 255u), scale_of(x >> 24));
                scale[lane] = make_uint4(a.x, a.y, b.x, b.y);
            }
            if (use > 0 && !wait(&sh.pv_done[buf], use - 1)) break;
            if (works) {
                tc_fence_after();
                __syncwarp();
                // (a loop, as for K: the roles' code passes through one instruction cache)
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    uint32_t v[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 a = scale[(h * 4 + i) * 2], b = scale[(h * 4 + i) * 2 + 1];
                        const uint32_t x = *reinterpret_cast<const uint32_t *>(tile + word_off + T.value[h * 4 + i]);
                        v[4 * i] = unpack_pair<SPEC_DTYPE_F16>(x, 0, a.x, a.y, zero);
                        v[4 * i + 1] = unpack_pair<SPEC_DTYPE_F16>(x, 1, a.z, a.w, zero);
                        v[4 * i + 2] = unpack_pair<SPEC_DTYPE_F16>(x, 2, b.x, b.y, zero);
                        v[4 * i + 3] = unpack_pair<SPEC_DTYPE_F16>(x, 3, b.z, b.w, zero);
                    }
                    tmem_store(to + buf * 64 + (uint32_t)(h * 16), v);
                }
                tmem_wait_store();
                tc_fence_before();
            }
            arrive(&sh.empty[stage]);
            arrive(&sh.pv_ready[buf]);
            if ((stage += kTurns) >= (uint32_t)kStages) stage = turn, ++fill;
            if ((buf += kTurns) >= kBufs) buf -= kBufs, ++use;
        }
    } else if (warp >= kSoft && warp < C::kV) {  // ---------------------------- K
        fewer_registers<C::kRegUnpack>();
        const uint32_t turn = kTurns == 2 ? (uint32_t)(warp - kSoft) >> 2 : 0u;
        const int quad = warp & 3, key = quad * 32 + lane;
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + C::kTK;
        const uint32_t zero = code_base<DT>();  // code 0
        const int in_block = key & (T.block - 1), block_off = (key >> T.block_shift) * T.bytes;
        const int code_off = block_off + ((in_block >> 3) * T.groups * 8 + (in_block & 7)) * 16;
        const int scale_off = block_off + T.block * T.C + in_block;
        for (uint32_t e = turn, stage = turn, fill = 0, buf = turn, use = 0; e < tiles; e += kTurns) {
            if (!wait(&sh.full[stage], fill)) break;
            if (use > 0 && !wait(&sh.s_full[buf], use - 1)) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < PACK * DP / 32; ++x) {
                const uint8_t *tile = sh.tile[stage] + x / (DP / 32) * (kTaKeys / 16 * 17) * T.C;
                const int g = x % (DP / 32) < T.groups ? x % (DP / 32) : 0;  // (past the last group: not multiplied)
                const uint4 code = *reinterpret_cast<const uint4 *>(tile + code_off + g * 128);
                const float f = scale_of(tile[scale_off + g * T.block]);
                const uint2 s = unpack_scale<DT>(f, f);
                const uint32_t word[4] = {code.x, code.y, code.z, code.w};
                uint32_t k[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) k[i] = unpack_pair<DT>(word[i / 4], i % 4, s.x, s.y, zero);
                tmem_store(to + buf * 64 + (uint32_t)(x * 16), k);
            }
            arrive(&sh.empty[stage]);
            tmem_wait_store();
            tc_fence_before();
            arrive(&sh.s_ready[buf]);
            if ((stage += kTurns) >= (uint32_t)kStages) stage = turn, ++fill;
            if ((buf += kTurns) >= kBufs) buf -= kBufs, ++use;
        }
    } else if (warp < kSoft) {  // ---------------------------------------------- softmax
        more_registers<C::kRegSoft>();
        const int wg = warp >> 2, quad = warp & 3;
        const int stream = kStreams == 2 ? wg : 0;     // takes the tiles of this parity, or all
        const int key = quad * 32 + lane;              // of a tile; and the channel (of all heads) in O
        const uint32_t col0 = kStreams == 2 ? 0u : (uint32_t)(wg * kW);  // the warp's columns
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t ts = tmem + lanes + C::kTS + col0, to = tmem + lanes + C::kTO + (uint32_t)stream * C::kOStep + col0;
        const int slot = quad * 32 / DP, ch = key % DP;
        const int rows_used = A.np * A.G, rows_cta = PACK * rows_used;
        const float scale = t4_scale<DT>(A);
        const int sinks = A.window ? A.sinks : 0;
        float *m = sh.m[warp], *f = sh.f[warp], *top = sh.ref[warp];
        // A column's reference is its largest score so far, `top`.  What its weights 2^z hold of that is the scaled form
        // as float32 rounds it, z = x scale - in_base2(top); of a top that is `far`, whose scaled form float32 holds
        // to 1 or more, all of it, z = (x - top) scale + kLift.  Which of the two follows from the top alone, so
        // sums over other tiles, streams and parts are brought together by what each of them holds.
        auto in_base2 = [&](float y) -> float { return fmaxf(y * scale, -FLT_MAX) - kLift; };
        auto far = [&](float y) -> bool { return y > -FLT_MAX && fabsf(y * scale) > 0x1p24f; };
        // the row of which this thread writes the sum: its head in the pack, node of the tile and head of the group
        const int c = (int)threadIdx.x, of = c / RP, r = c % RP, local = r / A.G, in_group = r - local * A.G;
        uint32_t base = 0;  // the CTA's tiles before this segment
        bool ok = true;
        for (int i = stream; i < (int)kBufs; i += kStreams) arrive(&sh.s_ready[i]);  // no scores to be read yet
        // The warps leave together: a wait in vain is told at their next meeting, so that no warp stands
        // at a barrier that another one has left for good.
        for (int seg_no = 0;; ++seg_no) {
            const SegSlot *sp = take(sh.path_full, seg_no);
            if (meet<256>(3, !sp)) {
                ok = false;
                break;
            }
            const Seg &s = sp->s;
            const int n = s.n;
            if (n == 0) break;
            const Geo g = s.g;
            // positions from `whole` on (to g.c) are seen by all nodes
            const int whole = A.window ? max(g.wlo, min(g.c, g.c + g.cnt - A.window)) : 0;
            float l[kW];
#pragma unroll
            for (int i = 0; i < kW; ++i) l[i] = 0.f;
            if (lane < kW) top[lane] = -FLT_MAX;
            bool coarse = false;
            __syncwarp();
            const int t0 = kStreams == 2 ? (int)((base + (uint32_t)stream) & 1u) : 0;
            const int i0 = s.i0;
#pragma unroll 1
            for (int t = t0; t < n; t += kStreams) {
                const int j0 = g.tile(i0 + t) * kTaKeys;
                const uint32_t e = base + (uint32_t)t, buf = e % kBufs, use = e / kBufs;
                const bool all = g.c - j0 >= kTaKeys && (j0 >= whole || sinks - j0 >= kTaKeys);
                unsigned long long seen = ~0ull;  // the rows of a head that see this key
                if (!all) {
                    const int j = j0 + key;
                    seen = 0ull;
                    if (j < g.end) {
                        const unsigned long long one = A.G >= 64 ? ~0ull : (1ull << A.G) - 1ull;
#pragma unroll 1
                        for (int x = 0; x < A.np; ++x) {
                            const int node = s.node0 + x;
                            if (node >= g.cnt) break;
                            const bool yes = j < g.c ? j >= sp->low[node] || j < sinks
                                                     : ((sp->path[node] >> (j - g.c)) & 1ull) != 0;
                            if (yes) seen |= one << (x * A.G);
                        }
                    }
                    if (PACK == 1) seen >>= col0;
                    __syncwarp();
                }
                ok = ok && wait(&sh.s_full[buf], use);
                tc_fence_after();
                float2 z[kW / 2];
                auto scores = [&](uint32_t (&x)[kW]) {  // -inf where they are not seen
                    tmem_load(ts + buf * C::kSStep, x);
                    if (!all) {
#pragma unroll
                        for (int i = 0; i < kW; ++i)
                            if (!((seen >> (i % RP)) & 1ull)) x[i] = 0xFF800000u;
                        __syncwarp();
                    }
                };
                auto shift = [&](const uint32_t (&x)[kW]) -> float {  // scaled, less the references; the largest
                    const float2 c2 = make_float2(scale, scale);
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kW; i += 4) {
                        const float4 r = *reinterpret_cast<const float4 *>(m + i);
                        z[i / 2] = fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2,
                                        make_float2(r.x, r.y));
                        z[i / 2 + 1] = fma2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), c2,
                                            make_float2(r.z, r.w));
                        mx[0] = fmaxf(fmaxf(mx[0], z[i / 2].x), z[i / 2].y);
                        mx[1] = fmaxf(fmaxf(mx[1], z[i / 2 + 1].x), z[i / 2 + 1].y);
                    }
                    return fmaxf(mx[0], mx[1]);
                };
                // The scores less the references; where one has grown, or at the stream's first tile, after new references.
                // (One copy of each step: the roles' code passes through one instruction cache.)
                bool gone = false;
                // 0: whether one has grown, 1: new references, 2: with those, which none exceeds by more than a rounding.
                int step = t == t0 || coarse ? 1 : 0;
#pragma unroll 1
                for (; step <= 2; ++step) {
                    uint32_t x[kW];
                    scores(x);
                    if (step != 1) {
                        const float largest = shift(x);
                        if (step == 2 || !meet<128>(1 + wg, !ok || largest > kLift + kTaGrow)) break;
                        gone = meet<128>(1 + wg, !ok);
                        if (gone) break;
                        continue;
                    }
                    // the columns' maxima over the four warps' keys
                    float mine = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kW; ++i) {
                        // (as integers that order alike; a NaN's column is NaN whatever its reference)
                        const int u = (int)x[i], y = __reduce_max_sync(0xFFFFFFFFu, u ^ ((u >> 31) & 0x7FFFFFFF));
                        if (lane == i) mine = __int_as_float(y ^ ((y >> 31) & 0x7FFFFFFF));
                    }
                    if (lane < kW) sh.top[warp][lane] = mine;
                    meet<128>(1 + wg, false);
                    bool large = false;
                    if (lane < kW) {
                        const int w0 = wg * 4;
                        float y = fmaxf(fmaxf(sh.top[w0][lane], sh.top[w0 + 1][lane]),
                                        fmaxf(sh.top[w0 + 2][lane], sh.top[w0 + 3][lane]));
                        const float old = top[lane];
                        y = fmaxf(y, old);
                        large = far(y);
                        const bool was = far(old);
                        const float now = large ? 0.f : in_base2(y), before = was ? 0.f : in_base2(old);
                        f[lane] = y == old ? 1.f
                                           : ex2(fmaf((was ? old : 0.f) - (large ? y : 0.f), scale, before - now) +
                                                 ((large ? kLift : 0.f) - (was ? kLift : 0.f)));
                        top[lane] = y;
                        m[lane] = large ? kLift : -now;
                    }
                    coarse = __any_sync(0xFFFFFFFFu, large) != 0;
                    __syncwarp();
                    if (t > t0) {  // O and the sums hold the stream's tiles before this one
#pragma unroll
                        for (int i = 0; i < kW; ++i) l[i] *= f[i];
                        // (their products are through, of two streams, since before these scores: see below)
                        if (kStreams == 1) ok = ok && wait(&sh.pv_done[(e - 1) % kBufs], (e - 1) / kBufs);
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < kW && ok; d += 16) {
                            uint32_t o[16];
                            tmem_load(to + (uint32_t)d, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[d + i]);
                            tmem_store(to + (uint32_t)d, o);
                        }
                        tmem_wait_store();
                    }
                    // A reference that is far is taken off the scores first, which is exact near it, so that their weights
                    // neither overflow nor vanish.  Every tile goes this way then.
                    if (coarse) {
                        __syncwarp();
                        if (lane < kW) f[lane] = far(top[lane]) ? top[lane] : 0.f;
                        __syncwarp();
#pragma unroll 1
                        for (int d = 0; d < kW; d += 16) {
                            uint32_t y[16];
                            tmem_load(ts + buf * C::kSStep + (uint32_t)d, y);
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) - f[d + i]);
                            tmem_store(ts + buf * C::kSStep + (uint32_t)d, y);
                        }
                        tmem_wait_store();
                        meet<128>(1 + wg, false);  // (the next tile's maxima are written where these were read)
                    }
                }
                if (gone) {
                    ok = false;
                    break;
                }
                tc_fence_before();
                arrive(&sh.s_ready[buf]);
                // (the weights before the last are through: their product was issued before these scores,
                // whose commit covers all products before it)
                uint8_t *p_row = sh.p[buf] + key * C::kRowP;
                const int swap = C::kRowP == 128 ? key & 7 : C::kRowP == 64 ? (key >> 1) & 3 : (key >> 2) & 1;
#pragma unroll
                for (int i = 0; i < kW; i += 8) {
                    uint32_t p[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float2 w2 = make_float2(ex2(z[i / 2 + y].x), ex2(z[i / 2 + y].y));
                        const float2 sum = add2(make_float2(l[i + 2 * y], l[i + 2 * y + 1]), w2);
                        l[i + 2 * y] = sum.x, l[i + 2 * y + 1] = sum.y;
                        // rounded to float16 for the product, up to 2^-11 of each; the sum takes them unrounded.
                        // In a float16 result that is seen: its rms error is 1.25 to 1.3 times that of one rounding
                        // (2.6e-4 against 2.1e-4 over 2000 keys); in bfloat16 it is not.
                        p[y] = pack2<SPEC_DTYPE_F16>(w2.x, w2.y);
                    }
                    *reinterpret_cast<uint4 *>(p_row + ((((int)col0 / 8 + i / 8) ^ swap) * 16)) =
                        make_uint4(p[0], p[1], p[2], p[3]);
                }
                fence_proxy_async();
                tc_fence_before();
                arrive(&sh.pv_ready[buf]);
            }

            // ---- the segment's result: sums over the warp's keys, a column to a lane
#pragma unroll
            for (int o = 16, w = kW; o > 0; o >>= 1) {
                if (w > 1) {  // lanes o apart take half of the columns each
                    w >>= 1;
#pragma unroll
                    for (int i = 0; i < kW / 2; ++i) {
                        if (i >= w) break;
                        const bool up = (lane & o) != 0;
                        const float give = up ? l[i] : l[i + w];
                        l[i] = (up ? l[i + w] : l[i]) + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                    }
                } else {
                    l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], o);
                }
            }
            // the lane's bits, from the top, chose the upper halves: lane i holds column i of 32, lanes 2 i and
            // 2 i + 1 column i of 16
            if (kW == 32 || (lane & 1) == 0) sh.sum[warp][kW == 32 ? lane : lane >> 1] = l[0];
            base += (uint32_t)n;
            // the last tiles' products (of the other stream's last tile too, if the segment has two)
            const uint32_t last = base - 1;
            ok = ok && wait(&sh.pv_done[last % kBufs], last / kBufs);
            if (kStreams == 2 && n > 1) ok = ok && wait(&sh.pv_done[(last - 1) % kBufs], (last - 1) / kBufs);
            if (meet<256>(3, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool whole_item = n == g.nt;
            const long long place = (long long)blockIdx.x * 2 + (i0 == 0 ? 1 : 0);  // a cut item's part
            const int only = kStreams == 2 && n == 1 ? (int)(last & 1u) : -1;      // the one stream with a part
            if (c < kCols) {  // a thread per row: its sum and lse, and the factors of its parts
                float ref, total;
                // of the warps wa .. wa + 3: the reference, the sum, and the factor that makes their weights
                // 2^((x - top) scale + kLift) where the reference was held rounded
                auto part = [&](int wa, int at, float &mm, float &ll, float &ww) {
                    mm = sh.ref[wa][at];
                    ll = sh.sum[wa][at] + sh.sum[wa + 1][at] + sh.sum[wa + 2][at] + sh.sum[wa + 3][at];
                    ww = mm == -FLT_MAX || far(mm) ? 1.f : ex2(fmaf(-mm, scale, in_base2(mm)) + kLift);
                };
                float w0, w1 = 0.f;
                if (kStreams == 1 || only >= 0) {
                    part(kStreams == 1 ? c / kW * 4 : only * 4, c % kW, ref, total, w0);
                    total *= w0;
                } else {
                    float ma, la, mb, lb;
                    part(0, c, ma, la, w0);
                    part(4, c, mb, lb, w1);
                    ref = fmaxf(ma, mb);
                    w0 *= ex2((ma - ref) * scale), w1 *= ex2((mb - ref) * scale);
                    total = la * w0 + lb * w1;
                }
                const int node = s.node0 + local, hk = s.hk * PACK + of;
                const bool exists = r < rows_used && node < A.N && hk < T.heads, valid = exists && node < g.cnt;
                const float inv = whole_item ? 4.f / total : 4.f;  // (O is a quarter of itself)
                sh.w[0][c] = w0 * inv, sh.w[1][c] = w1 * inv;
                const long long orow = ((long long)s.b * A.N + node) * A.Hq + hk * A.G + in_group;
                const long long prow = place * rows_cta + of * rows_used + r;
                sh.row[c] = whole_item ? (exists ? 2 * orow * A.D + (valid ? 0 : 1) : -1) : (valid ? 2 * prow * A.D : -1);
                if (exists && whole_item && A.lse) A.lse[orow] = ta_lse(valid, in_base2(ref), total);
                if (exists && !whole_item)
                    A.part_ml[prow] = valid ? make_float2(ref, total) : make_float2(-INFINITY, 0.f);
            }
            meet<256>(3, false);
            // a warpgroup writes half of the columns of every head
            const int hk = s.hk * PACK + slot;
            constexpr int kO = RP / 2;
            const int r0 = wg * kO, c0 = slot * RP + r0;
            if (slot < PACK && hk < T.heads && ch - lane < A.D && r0 < rows_used) {
                uint32_t o[kO];
                tmem_load(tmem + lanes + C::kTO + (only > 0 ? C::kOStep : 0u) + (uint32_t)c0, o);
#pragma unroll
                for (int i = 0; i < kO; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.w[0][c0 + i]);
                if (kStreams == 2 && only < 0) {
                    uint32_t y[kO];
                    tmem_load(tmem + lanes + C::kTO + C::kOStep + (uint32_t)c0, y);
#pragma unroll
                    for (int i = 0; i < kO; ++i)
                        o[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), sh.w[1][c0 + i], __uint_as_float(o[i])));
                }
#pragma unroll
                for (int i = 0; i < kO; ++i) {
                    const long long row = sh.row[c0 + i], at = (row >> 1) + ch;
                    if (row < 0 || ch >= A.D) continue;
                    if (whole_item) A.out[at] = row & 1 ? (uint16_t)0 : (uint16_t)pack2<DT>(__uint_as_float(o[i]), 0.f);
                    else A.part_o[at] = __uint_as_float(o[i]);
                }
            }
            tc_fence_before();
            arrive(&sh.o_free);
            arrive(&sh.seg_free[seg_no % kTaSlots]);
        }
        if (!ok) *abort = 1;
        if (fewer) {  // the nodes past every row tile (past the counts) see nothing
            for (int b = blockIdx.x; b < A.B; b += gridDim.x) {
                const int2 lens = ta_lens(A, b);
                const int n0 = lens.y > 0 ? min(A.N, ta_row_tiles<kTaSplitKeys>(A, lens.y) * A.np) : 0;
                if (n0 >= A.N) continue;
                const long long r0 = ((long long)b * A.N + n0) * A.Hq, r1 = ((long long)b * A.N + A.N) * A.Hq;
                uint4 *o = reinterpret_cast<uint4 *>(A.out);
#pragma unroll 1
                for (long long i = r0 * A.D / 8 + threadIdx.x; i < r1 * A.D / 8; i += kSoft * 32)
                    o[i] = make_uint4(0u, 0u, 0u, 0u);
                if (A.lse)
#pragma unroll 1
                    for (long long i = r0 + threadIdx.x; i < r1; i += kSoft * 32) A.lse[i] = -INFINITY;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && sh.abort) flag(A.status, SPEC_DEV_TIMEOUT);
}

// ------------------------------------------------------------------ host

// How the rows are laid out: heads to a pack, rows of a head (as columns of the products), nodes of a row tile.
struct T4Rows {
    int dp, pack, rp, np;
};
static T4Rows t4_rows(int N, int G, int heads, int D) {
    T4Rows r;
    r.dp = D <= 64 ? 64 : 128;
    auto tiles = [&](int most) { return most < G ? INT_MAX / 2 : (N + most / G - 1) / (most / G); };
    // Heads of up to 64 go in pairs of 32 rows each where that makes no more pairs and row tiles than heads alone with
    // 64 rows, which leave half of V's lanes empty (64 requests of 4096 positions, 8 key heads of 64: 32 rows of a
    // head 67 us in pairs and 114 alone, 36 rows 113 and 115, 64 rows 116 and 122).
    r.pack = r.dp == 64 && (long long)tiles(32) * ((heads + 1) / 2) <= (long long)tiles(64) * heads ? 2 : 1;
    const int count = tiles(r.pack == 2 ? 32 : 64);
    r.np = (N + count - 1) / count;
    // The fewest columns that hold the rows (64 requests of 4096 positions, heads of 128: 4 rows of a head 84 us with
    // 16 columns, 87 with 32, 105 with 64; 20 rows 93 with 32, 113 with 64; pairs of 4 rows at 8192 positions 94 with
    // 16 for each, 103 with 32).  A head of 64 alone has more than 32 rows.
    const int rows = r.np * G;
    r.rp = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    if (r.dp == 64 && r.pack == 1) r.rp = 64;
    return r;
}

struct T4Layout {
    size_t o, ml, joins, total;
};
static T4Layout t4_layout(const T4Rows &r, int G, int D) {
    T4Layout L;
    const size_t rows = (size_t)kTaMaxCtas * 2 * r.pack * r.np * G;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    L.o = 0;
    L.ml = up(rows * (size_t)D * sizeof(float));
    L.joins = up(L.ml + rows * sizeof(float2));
    L.total = up(L.joins + (size_t)kTaMaxCtas * sizeof(int4));
    return L;
}

template <int DT, int DP, int PACK, int RP>
static spec_status_t t4_launch(const T4Args &T, const CUtensorMap &q, int ctas, int dev, cudaStream_t s) {
    constexpr size_t smem = sizeof(T4Shared<DP, PACK, RP>) + 1024;
    static_assert(smem <= 232448, "shared memory of a CTA");
    static bool ready[kMaxDevices] = {};
    if (!ready[dev]) {
        // (compiled with fewer registers than are divided between the warps, setmaxnreg would wait for ever)
        cudaFuncAttributes made = {};
        if (cudaFuncGetAttributes(&made, tree_attn4<DT, DP, PACK, RP>) != cudaSuccess ||
            made.numRegs < T4Cfg<DP, PACK, RP>::kRegs ||
            cudaFuncSetAttribute(tree_attn4<DT, DP, PACK, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess)
            return SPEC_ERR_CUDA;
        ready[dev] = true;
    }
    const spec_status_t st =
        launch_pdl(tree_attn4<DT, DP, PACK, RP>, dim3((unsigned)ctas), dim3(T4Cfg<DP, PACK, RP>::kThreads), smem, s, q, T);
    if (st != SPEC_OK) return st;
    constexpr int rows = 256 / kTaJoinLanes;
    const int used = T.a.np * T.a.G, cta = PACK * used;
    return launch_pdl(tree_attn_join<DT, true>, dim3((unsigned)ctas, (unsigned)((cta + rows - 1) / rows)), dim3(256), 0, s,
                      T.a, used, cta, PACK == 2 ? (int)kTaSplitHeads : (int)kTaSplitKeys, t4_scale<DT>(T.a), kLift);
}

template <int DT>
static spec_status_t t4_launch_rows(const T4Args &T, const CUtensorMap &q, const T4Rows &r, int ctas, int dev,
                                    cudaStream_t s) {
    if (r.dp == 64) {
        if (r.pack == 1) return t4_launch<DT, 64, 1, 64>(T, q, ctas, dev, s);
        return r.rp == 16 ? t4_launch<DT, 64, 2, 16>(T, q, ctas, dev, s) : t4_launch<DT, 64, 2, 32>(T, q, ctas, dev, s);
    }
    switch (r.rp) {
    case 16: return t4_launch<DT, 128, 1, 16>(T, q, ctas, dev, s);
    case 32: return t4_launch<DT, 128, 1, 32>(T, q, ctas, dev, s);
    default: return t4_launch<DT, 128, 1, 64>(T, q, ctas, dev, s);
    }
}

} // namespace sv

extern "C" {

size_t spec_tree_attention4_workspace_bytes(int B, int N, int Hq, int heads, int head_dim) {
    if (B < 1 || B >= (1 << 16) || N < 1 || N > SPEC_MAX_TREE || heads < 1 || heads > 1024 || Hq < heads ||
        Hq % heads || Hq / heads > 64 || head_dim < 8 || head_dim % 8 || head_dim > SPEC_MAX_HEAD_DIM)
        return 0;
    return sv::t4_layout(sv::t4_rows(N, Hq / heads, heads, head_dim), Hq / heads, head_dim).total;
}

spec_status_t spec_tree_attention4(const void *q, spec_dtype_t dtype, long long q_stride_b, long long q_stride_n,
                                   long long q_stride_h, const spec_pages4_t *pages, const int32_t *page_table,
                                   int per_head, const int32_t *cache_len, const int32_t *parent,
                                   const int32_t *node_count, int B, int N, int Hq, int max_pages, float scale,
                                   int window, int sinks, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, uint32_t *dev_status, void *stream) {
    sv::Pool4 P;
    const spec_status_t st = sv::make_pool4(pages, P);
    if (st != SPEC_OK) return st;
    if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    const int D = P.D, H = P.heads;
    const size_t need = spec_tree_attention4_workspace_bytes(B, N, Hq, H, D);
    if (!q || !page_table || !cache_len || !out || need == 0 || pages->layers != 1 || max_pages < 1 ||
        ((uintptr_t)q & 15) || ((uintptr_t)out & 15) || window < 0 || sinks < 0 ||
        !sv::ta_scale_ok(scale, dtype == SPEC_DTYPE_F16 ? sv::kKeyPart<SPEC_DTYPE_F16> : 1.f) ||
        (per_head != 0 && per_head != 1))
        return SPEC_ERR_INVALID_ARG;
    const long long qst[3] = {q_stride_h, q_stride_n, q_stride_b};
    const int qext[3] = {Hq, N, B};
    for (int i = 0; i < 3; ++i)
        if (qst[i] % 8 || qst[i] < (qext[i] > 1 ? D : 0)) return SPEC_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need) return SPEC_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    if (!sv::current_device(dev, sms)) return SPEC_ERR_CUDA;
    const int ctas = sms < sv::kTaMaxCtas ? sms : sv::kTaMaxCtas;

    const sv::T4Rows r = sv::t4_rows(N, Hq / H, H, D);
    const sv::T4Layout L = sv::t4_layout(r, Hq / H, D);
    sv::T4Args T = {};
    sv::TaArgs &A = T.a;
    A.table = page_table;
    A.row_b = (long long)max_pages * (per_head ? H : 1);
    A.row_h = per_head ? max_pages : 0;
    A.len = cache_len;
    A.parent = parent;
    A.node_count = node_count;
    A.B = B;
    A.N = N;
    A.Hq = Hq;
    A.H = (H + r.pack - 1) / r.pack;
    A.G = Hq / H;
    A.D = D;
    A.max_pages = max_pages;
    A.num_pages = P.num_pages;
    A.page = P.page;
    A.page_shift = P.page_shift;
    A.window = window;
    A.sinks = sinks;
    A.np = r.np;
    A.scale_log2 = scale * sv::kTaLog2e;
    A.out = static_cast<uint16_t *>(out);
    A.lse = lse;
    char *ws = static_cast<char *>(workspace);
    A.part_o = reinterpret_cast<float *>(ws + L.o);
    A.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
    A.joins = reinterpret_cast<int4 *>(ws + L.joins);
    A.status = dev_status;
    A.tries = sv::g_diag_timeout ? 0u : sv::kTaTries;
    T.data = P.data;
    T.page_st = P.page_st;
    T.head_st = P.head;
    T.heads = H;
    T.C = P.C;
    T.groups = P.groups;
    T.block = P.block;
    while ((1 << T.block_shift) < P.block) ++T.block_shift;
    T.bytes = P.bytes;
    for (int i = 0; i < sv::kTaKeys / 8; ++i)
        T.value[i] = (i * 8 >> T.block_shift) * P.bytes + P.block * P.C / 2 + (i * 8 & (P.block - 1)) / 8 * P.C * 4;

    CUtensorMap tq;
    // an extent of one is never stepped over: any valid stride stands for it
    auto bytes = [&](long long stride, int extent) { return (cuuint64_t)(extent > 1 ? stride : D) * 2; };
    const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)N, (cuuint64_t)B};
    const cuuint64_t qs[3] = {bytes(q_stride_h, Hq), bytes(q_stride_n, N), bytes(q_stride_b, B)};
    if (!sv::ta_tmap(&tq, dtype, q, qd, qs, (cuuint32_t)A.G, (cuuint32_t)r.np)) return SPEC_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_DTYPE_BF16 ? sv::t4_launch_rows<SPEC_DTYPE_BF16>(T, tq, r, ctas, dev, s)
                                    : sv::t4_launch_rows<SPEC_DTYPE_F16>(T, tq, r, ctas, dev, s);
}

} // extern "C"
