// tree_attn4.cu -- attention of drafted trees over a 4-bit paged cache on the
// sm_103a tensor cores.
//
// Mathematics: that of tree_attn.cu (one pass over the keys with a reference near
// the running maximum, parts over disjoint keys joined), on keys and values (c -
// 8) s with a 4-bit code c and a scale s per 32 channels.  Both are formed exactly:
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
// One CTA per SM: four warps unpack K, four V, four form the weights, and a warp
// each loads (one bulk copy per page and head), issues the products and
// schedules.  Tiles of keys alternate between two buffers of K, V, S and P, so the
// stages of consecutive tiles overlap.  Heads of up to 64 are taken in pairs (the
// lanes of V^T are two heads' channels; the quarter of the product that mixes them is
// not read).  More than 64 rows are cut into row tiles.
#include "attn_plan.cuh"
#include "cache4.cuh"

namespace sv {

constexpr int kT4Threads = 480;  // 4 softmax warps, 4 of K, 4 of V, then loads, products, scheduling
constexpr int kT4WarpLoad = 12, kT4WarpMma = 13, kT4WarpPlan = 14;
// tensor-memory columns: K, V and S two buffers each, then O
constexpr uint32_t kT4K = 0, kT4V = 128, kT4S = 256, kT4O = 384, kT4Buf = 64;

struct T4Args {
    TaArgs a;             // a.H: packs of heads
    const uint8_t *data;  // the pool
    long long page_st, head_st;
    int heads;            // key heads
    int C, groups;        // channels kept and groups of 32 of them
    int block, block_shift, bytes;  // tokens of a block, its bytes
};

template <int DP, int PACK, int RP> struct T4Cfg {
    static constexpr int kCols = PACK * RP;              // rows of all heads of a pack
    static constexpr int kRowP = kCols * 2;              // bytes of a key's weights
    static constexpr int kStage = PACK * DP * 136;       // one tile, packed
    static constexpr int kStages = kCols == 64 ? 6 : 8;
    static constexpr int kQ = PACK * RP * DP * 2;
    static constexpr int kW = kCols < 32 ? kCols : 32;   // columns a softmax warp has in hand at a time
    static constexpr int kSwizzle = kCols == 64 ? 2 : kCols == 32 ? 4 : 6;  // 128, 64 or 32 bytes
};

template <int DP, int PACK, int RP> struct T4Shared {
    using C = T4Cfg<DP, PACK, RP>;
    uint8_t q[kTaSlots][C::kQ];
    uint8_t p[2][kTaKeys * C::kRowP];
    uint8_t tile[C::kStages][C::kStage];
    uint4 scale[4][32];                      // V's scales and their biases, four keys of a warp's group each
    uint4 bias[4][32];
    float m[4][C::kCols], f[4][C::kCols];    // per warp: references and their last factors
    float top[4][C::kCols], sum[4][C::kCols];
    long long incl[kTaChunks];
    SegSlot seg[kTaSlots];
    uint64_t seg_full[kTaSlots], path_full[kTaSlots], seg_free[kTaSlots], q_full[kTaSlots], q_free[kTaSlots];
    uint64_t full[C::kStages], empty[C::kStages];
    uint64_t k_full[2], v_full[2], s_full[2], s_free[2], p_full[2], pv_done[2], o_free, meet, done;
    int4 votes[2];                           // of the softmax warps, by the parity of their meeting
    uint32_t tmem_base;
    int abort;
};

// ------------------------------------------------------------------ PTX

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
// Two codes of a word as numbers, times a scale (see the head of the file): pair i of the word
// lies at bits 4 i and 4 i + 16.
template <int DT> __device__ __forceinline__ uint32_t unpack_pair(uint32_t w, int i, uint32_t s, uint32_t b) {
    if (DT == SPEC_DTYPE_BF16) return hfma2(DT, ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, s, b);
    const uint32_t y = i == 0 ? w << 6 : i == 1 ? w << 2 : i == 2 ? w >> 2 : w >> 6;
    return hfma2(DT, (y & 0x03C003C0u) | 0x4C004C00u, s, b);
}
// The multiplier and addend of unpack_pair for the scale(s) lo and hi.
template <int DT> __device__ __forceinline__ uint2 unpack_scale(float lo, float hi) {
    if (DT == SPEC_DTYPE_BF16) return make_uint2(pack2<DT>(lo, hi), pack2<DT>(-136.f * lo, -136.f * hi));
    return make_uint2(pack2<DT>(0.25f * lo, 0.25f * hi), pack2<DT>(-6.f * lo, -6.f * hi));
}

// ------------------------------------------------------------------ the kernel

template <int DT, int DP, int PACK, int RP>
__global__ void __launch_bounds__(kT4Threads, 1)
    tree_attn4(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ T4Args T) {
    using C = T4Cfg<DP, PACK, RP>;
    using Sh = T4Shared<DP, PACK, RP>;
    extern __shared__ uint8_t t4_raw[];
    Sh &sh = *reinterpret_cast<Sh *>((reinterpret_cast<uintptr_t>(t4_raw) + 1023) & ~(uintptr_t)1023);
    const TaArgs &A = T.a;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    constexpr int kCols = C::kCols, kStages = C::kStages, kW = C::kW;
    constexpr float kLift = 7.f;  // weights up to 2^15: those 2^-29 below the maximum are still normal in float16

    if (threadIdx.x == 0) {
        for (int i = 0; i < kTaSlots; ++i) {
            mbar_init(&sh.seg_full[i], 1);
            mbar_init(&sh.path_full[i], 1);
            mbar_init(&sh.seg_free[i], 4 + 2);
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_free[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.k_full[i], 4);
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 4);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.o_free, 4);
        mbar_init(&sh.meet, 4);
        mbar_init(&sh.done, 1);
        sh.abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&tm_q);
    }
    // the rows of Q past the last one stay 0
    for (int i = threadIdx.x; i < (int)sizeof(sh.q) / 16; i += kT4Threads)
        reinterpret_cast<uint4 *>(sh.q)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    if (warp == kT4WarpMma) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    pdl_trigger();
    pdl_wait();
    Walk<kTaSplitKeys> w;
    if (warp == kT4WarpPlan) w.fetch(A, 0);
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
        return __all_sync(0xFFFFFFFFu, ta_wait(bar, parity & 1u, abort, A.tries)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(reinterpret_cast<unsigned long long *>(bar));
    };
    // segment k, or nothing when the wait for it ran out
    auto take = [&](uint64_t *bars, int k) -> const SegSlot * {
        return wait(&bars[k % kTaSlots], (uint32_t)(k / kTaSlots)) ? &sh.seg[k % kTaSlots] : nullptr;
    };

    if (warp == kT4WarpPlan) {  // ------------------------------------------- scheduling
        ta_schedule<kTaSplitKeys>(A, w, sh.incl, sh.seg, sh.seg_full, sh.path_full, sh.seg_free, u_first, u_last, run,
                                  abort);
    } else if (warp == kT4WarpLoad) {  // ------------------------------------- loads
        const int recs = kTaKeys >> T.block_shift;           // blocks of a head's tile
        const int nb = PACK * recs, ahead = 32 / nb;         // copies of a tile, tiles whose pages are fetched at once
        const int mine = lane % nb, slot = mine / recs, rec = mine % recs;
        uint32_t stage = 0, fill = 0;
        int seg_no = 0;
        bool ok = true;
        for (; ok; ++seg_no) {
            const SegSlot *sp = take(sh.seg_full, seg_no);
            if (!sp || sp->s.n == 0) break;
            const Seg s = sp->s;
            arrive(&sh.seg_free[seg_no % kTaSlots]);
            const int qb = seg_no % kTaSlots;
            if (seg_no >= kTaSlots && !wait(&sh.q_free[qb], (uint32_t)(seg_no / kTaSlots - 1))) break;
            if (elect_one()) {
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
            const int *row = A.table + s.b * A.row_b + head * A.row_h;
            const uint8_t *from = T.data + head * T.head_st;
            // the first position of this lane's block in tile i, and whether a node sees any of it
            auto block_pos = [&](int i) -> int { return s.g.tile(i) * kTaKeys + (rec << T.block_shift); };
            auto block_seen = [&](int j) -> bool {
                return head < T.heads && j < s.g.end && (s.g.wlo - j < T.block || j < A.sinks);
            };
            auto fetch = [&](int i0) -> int {  // the page of this lane's block in tile i0 + lane / nb
                const int i = i0 + lane / nb;
                if (i >= i_end) return 0;
                const int j = block_pos(i);
                if (!block_seen(j)) return 0;
                int p = __ldcg(row + (j >> A.page_shift));
                if ((unsigned)p >= (unsigned)A.num_pages) {
                    flag(A.status, SPEC_DEV_BAD_PAGE);
                    p = 0;
                }
                return p;
            };
            int base = s.i0, now = fetch(base), next = fetch(base + ahead);
            for (int i = s.i0; i < i_end; ++i) {
                if (i == base + ahead) {
                    base = i;
                    now = next;
                    next = fetch(base + ahead);
                }
                if (fill > 0 && !wait(&sh.empty[stage], fill - 1)) {
                    ok = false;
                    break;
                }
                const int j = block_pos(i);
                const bool load = lane / nb == i - base && block_seen(j);
                const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, load);
                if (elect_one()) mbar_expect_tx(&sh.full[stage], (uint32_t)(__popc(lanes) * T.bytes));
                __syncwarp();
                if (load)
                    bulk_g2s(sh.tile[stage] + mine * T.bytes,
                             from + now * T.page_st + ((j & (A.page - 1)) >> T.block_shift) * T.bytes,
                             (uint32_t)T.bytes, &sh.full[stage]);
                __syncwarp();
                if (++stage == kStages) stage = 0, ++fill;
            }
        }
        // every copy has landed before the CTA may exit
        for (uint32_t x = 0; x < (uint32_t)kStages; ++x) {
            const uint32_t n = fill + (x < stage ? 1u : 0u);
            if (n > 0) mbar_wait_bounded(&sh.full[x], (n - 1) & 1u, kTaWaitNs);
        }
        for (int x = 0; x < kTaSlots; ++x) {
            const int n = (seg_no + kTaSlots - 1 - x) / kTaSlots;
            if (n > 0) mbar_wait_bounded(&sh.q_full[x], (uint32_t)(n - 1) & 1u, kTaWaitNs);
        }
        __syncwarp();
    } else if (warp == kT4WarpMma) {  // -------------------------------------- products
        constexpr uint32_t kIdS = (ta_idesc<DT>(RP, false)), kIdO = ta_idesc<SPEC_DTYPE_F16>(kCols, true);
        const uint64_t q_desc = umma_desc_sw128(smem_u32(sh.q[0]));
        const uint64_t w_desc = p_desc<C::kRowP, C::kSwizzle>(smem_u32(sh.p[0]));
        const int steps = T.C / 16;
        int s_seg = 0, s_left = 0, v_seg = 0, v_left = 0;
        bool fresh = false, ok = true;
        auto scores = [&](uint32_t e) -> bool {
            const uint32_t buf = e & 1u, use = e >> 1;
            if (s_left == 0) {
                if (!take(sh.seg_full, s_seg)) return false;
                s_left = __shfl_sync(0xFFFFFFFFu, sh.seg[s_seg % kTaSlots].s.n, 0);
                if (!wait(&sh.q_full[s_seg % kTaSlots], (uint32_t)(s_seg / kTaSlots))) return false;
                ++s_seg;
            }
            const int qb = (s_seg - 1) % kTaSlots;
            if (!wait(&sh.k_full[buf], use)) return false;
            if (use > 0 && !wait(&sh.s_free[buf], use - 1)) return false;
            tc_fence_after();
            --s_left;
            if (elect_one()) {
#pragma unroll
                for (int x = 0; x < PACK; ++x) {
                    const uint64_t qd = q_desc + (uint64_t)((qb * C::kQ + x * RP * DP * 2) / 16);
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)
                        if (k < steps)
                            mma_ts(tmem + kT4S + buf * kT4Buf + (uint32_t)(x * RP),
                                   tmem + kT4K + buf * kT4Buf + (uint32_t)(x * DP / 2 + k * 8),
                                   qd + (uint64_t)((k >> 2) * (RP * 128 / 16) + (k & 3) * 2), kIdS, k > 0 ? 1u : 0u);
                }
                umma_commit(&sh.s_full[buf]);
                if (s_left == 0) umma_commit(&sh.q_free[qb]);
            }
            __syncwarp();
            return true;
        };
        auto values = [&](uint32_t e) -> bool {
            const uint32_t buf = e & 1u, use = e >> 1;
            if (v_left == 0) {
                v_left = __shfl_sync(0xFFFFFFFFu, sh.seg[v_seg % kTaSlots].s.n, 0);
                if (v_seg > 0 && !wait(&sh.o_free, (uint32_t)(v_seg - 1))) return false;
                ++v_seg;
                fresh = true;
            }
            if (!wait(&sh.v_full[buf], use) || !wait(&sh.p_full[buf], use)) return false;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTaKeys / 16; ++k)
                    mma_ts(tmem + kT4O, tmem + kT4V + buf * kT4Buf + (uint32_t)(k * 8),
                           w_desc + (uint64_t)((buf * (uint32_t)(kTaKeys * C::kRowP) + k * 16 * C::kRowP) / 16), kIdO,
                           fresh && k == 0 ? 0u : 1u);
                umma_commit(&sh.pv_done[buf]);
            }
            __syncwarp();
            fresh = false;
            if (--v_left == 0) arrive(&sh.seg_free[(v_seg - 1) % kTaSlots]);
            return true;
        };
        // the next tile's scores go before a tile's values, whose weights take longer
        if (tiles > 0) ok = scores(0);
        for (uint32_t e = 0; e < tiles && ok; ++e) {
            if (e + 1 < tiles) ok = scores(e + 1);
            ok = ok && values(e);
        }
        // every MMA has finished before the TMEM is freed
        if (elect_one()) umma_commit(&sh.done);
        mbar_wait_bounded(&sh.done, 0u, kTaWaitNs);
        __syncwarp();
    } else if (warp >= 8) {  // ------------------------------------------------ V
        const int quad = warp & 3, slot = quad * 32 / DP, ch = (quad * 32 + lane) % DP;
        const bool works = slot < PACK && ch - lane < T.C;  // the warp's lanes alike
        const int g = ch >> 5, block_mask = T.block - 1;
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + kT4V;
        const int head_off = slot * ((kTaKeys >> T.block_shift) * T.bytes);
        for (uint32_t e = 0, stage = 0, fill = 0; e < tiles; ++e) {
            if (!wait(&sh.full[stage], fill)) break;
            const uint8_t *tile = sh.tile[stage] + head_off;
            uint4 *scale = sh.scale[quad], *bias = sh.bias[quad];
            if (works) {  // scales of keys 4 lane .. 4 lane + 3
                const int t = 4 * lane;
                const uint32_t x = *reinterpret_cast<const uint32_t *>(
                    tile + (t >> T.block_shift) * T.bytes + T.block * (T.C + T.groups + g) + (t & block_mask));
                const uint2 a = unpack_scale<SPEC_DTYPE_F16>(scale_of(x & 255u), scale_of((x >> 8) & 255u));
                const uint2 b = unpack_scale<SPEC_DTYPE_F16>(scale_of((x >> 16) & 255u), scale_of(x >> 24));
                __syncwarp();
                reinterpret_cast<uint2 *>(scale)[lane] = make_uint2(a.x, b.x);
                reinterpret_cast<uint2 *>(bias)[lane] = make_uint2(a.y, b.y);
                __syncwarp();
            }
            if (e >= 2 && !wait(&sh.pv_done[e & 1u], (e >> 1) - 1)) break;
            if (works) {
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = (h * 8 + i) * 8;
                        const uint32_t x = *reinterpret_cast<const uint32_t *>(
                            tile + (t >> T.block_shift) * T.bytes + T.block * (T.C >> 1) +
                            (((t & block_mask) >> 3) * T.C + ch) * 4);
                        const uint4 s = scale[h * 8 + i], b = bias[h * 8 + i];
                        v[4 * i] = unpack_pair<SPEC_DTYPE_F16>(x, 0, s.x, b.x);
                        v[4 * i + 1] = unpack_pair<SPEC_DTYPE_F16>(x, 1, s.y, b.y);
                        v[4 * i + 2] = unpack_pair<SPEC_DTYPE_F16>(x, 2, s.z, b.z);
                        v[4 * i + 3] = unpack_pair<SPEC_DTYPE_F16>(x, 3, s.w, b.w);
                    }
                    tmem_store(to + (e & 1u) * kT4Buf + (uint32_t)(h * 32), v);
                }
                tmem_wait_store();
                tc_fence_before();
            }
            arrive(&sh.empty[stage]);
            arrive(&sh.v_full[e & 1u]);
            if (++stage == (uint32_t)kStages) stage = 0, ++fill;
        }
    } else if (warp >= 4) {  // ------------------------------------------------ K
        const int quad = warp & 3, key = quad * 32 + lane;
        const uint32_t to = tmem + ((uint32_t)(quad * 32) << 16) + kT4K;
        const int t = key & (T.block - 1), recs = kTaKeys >> T.block_shift;
        const int code_off = (key >> T.block_shift) * T.bytes + ((t >> 3) * T.groups * 8 + (t & 7)) * 16;
        const int scale_off = (key >> T.block_shift) * T.bytes + T.block * T.C + t;
        for (uint32_t e = 0, stage = 0, fill = 0; e < tiles; ++e) {
            if (!wait(&sh.full[stage], fill)) break;
            if (e >= 2 && !wait(&sh.s_full[e & 1u], (e >> 1) - 1)) break;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < PACK * DP / 64; ++x) {  // 64 channels of a head at a time
                const int slot = x / (DP / 64), g0 = x % (DP / 64) * 2;
                const uint8_t *tile = sh.tile[stage] + slot * recs * T.bytes;
                uint32_t k[32];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int g = g0 + i < T.groups ? g0 + i : 0;  // (past the last group: not multiplied)
                    const uint4 c = *reinterpret_cast<const uint4 *>(tile + code_off + g * 128);
                    const float f = scale_of(tile[scale_off + g * T.block]);
                    const uint2 s = unpack_scale<DT>(f, f);
                    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int z = 0; z < 4; ++z) k[16 * i + 4 * y + z] = unpack_pair<DT>(word[y], z, s.x, s.y);
                }
                tmem_store(to + (e & 1u) * kT4Buf + (uint32_t)(x * 32), k);
            }
            tmem_wait_store();
            tc_fence_before();
            arrive(&sh.empty[stage]);
            arrive(&sh.k_full[e & 1u]);
            if (++stage == (uint32_t)kStages) stage = 0, ++fill;
        }
    } else {  // ---------------------------------------------------------------- softmax
        const int key = warp * 32 + lane;  // of a tile; and the channel (of a slot) in O
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const int slot = warp * 32 / DP, ch = (warp * 32 + lane) % DP;
        const int rows_used = A.np * A.G, rows_cta = PACK * rows_used;
        // a quarter of the keys' scale was multiplied in float16
        const float scale = A.scale_log2 * (DT == SPEC_DTYPE_F16 ? 4.f : 1.f);
        const int sinks = A.window ? A.sinks : 0;
        float *m = sh.m[warp], *f = sh.f[warp];
        uint32_t e = 0, meeting = 0;
        int seg_no = 0;
        bool ok = true;
        // Waits for all four warps; whether a thread of any says so.  (Bounded like every wait: a
        // warp that has given up is not waited for for ever, as it would be at a hardware barrier.)
        auto any = [&](bool x) -> bool {
            const bool mine = __any_sync(0xFFFFFFFFu, x);
            int4 *votes = &sh.votes[meeting & 1u];
            if (lane == 0) reinterpret_cast<volatile int *>(votes)[warp] = mine;
            arrive(&sh.meet);
            ok = ok && wait(&sh.meet, meeting++);
            const volatile int *v = reinterpret_cast<const volatile int *>(votes);
            return (v[0] | v[1] | v[2] | v[3]) != 0;
        };
        for (; ok; ++seg_no) {
            const SegSlot *sp = take(sh.path_full, seg_no);
            if (!sp || sp->s.n == 0) break;
            const Seg s = sp->s;
            const Geo &g = s.g;
            // positions from `whole` on (to g.c) are seen by all nodes
            const int whole = A.window ? max(g.wlo, min(g.c, g.c + g.cnt - A.window)) : 0;
            float2 l[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) l[i] = make_float2(0.f, 0.f);
            for (int i = lane; i < kCols; i += 32) m[i] = -FLT_MAX;
            __syncwarp();
            for (int t = 0; t < s.n && ok; ++t, ++e) {
                const int j0 = g.tile(s.i0 + t) * kTaKeys;
                const uint32_t buf = e & 1u, use = e >> 1;
                const bool all = g.c - j0 >= kTaKeys && (j0 >= whole || sinks - j0 >= kTaKeys);
                unsigned long long seen = ~0ull;  // the rows of a head that see this key
                if (!all) {
                    const int j = j0 + key;
                    seen = 0ull;
                    if (j < g.end) {
                        const unsigned long long one = A.G >= 64 ? ~0ull : (1ull << A.G) - 1ull;
#pragma unroll 1
                        for (int n = 0; n < A.np; ++n) {
                            const int node = s.node0 + n;
                            if (node >= g.cnt) break;
                            const bool yes = j < g.c ? j >= sp->low[node] || j < sinks
                                                     : ((sp->path[node] >> (j - g.c)) & 1ull) != 0;
                            if (yes) seen |= one << (n * A.G);
                        }
                    }
                }
                ok = wait(&sh.s_full[buf], use);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < kCols / kW; ++h) {
                    const int c0 = h * kW;  // first column
                    float2 z[kW / 2];
                    auto scores = [&](uint32_t (&x)[kW]) {  // -inf where they are not seen
                        tmem_load(tmem + lanes + kT4S + buf * kT4Buf + (uint32_t)c0, x);
                        if (!all) {
#pragma unroll
                            for (int i = 0; i < kW; ++i)
                                if (!((seen >> ((c0 + i) % RP)) & 1ull)) x[i] = 0xFF800000u;
                            __syncwarp();
                        }
                    };
                    auto shift = [&](const uint32_t (&x)[kW]) -> float {  // scaled, less the references; the largest
                        const float2 c2 = make_float2(scale, scale);
                        float mx = -INFINITY;
#pragma unroll
                        for (int i = 0; i < kW; i += 4) {
                            const float4 r = *reinterpret_cast<const float4 *>(m + c0 + i);
                            z[i / 2] = fma2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2,
                                            make_float2(-r.x, -r.y));
                            z[i / 2 + 1] = fma2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), c2,
                                                make_float2(-r.z, -r.w));
                            mx = fmaxf(mx, fmaxf(fmaxf(z[i / 2].x, z[i / 2].y), fmaxf(z[i / 2 + 1].x, z[i / 2 + 1].y)));
                        }
                        return mx;
                    };
                    float largest;
                    {
                        uint32_t x[kW];
                        scores(x);
                        largest = shift(x);
                    }
                    const bool grown = any(largest > kLift + kTaGrow);
                    if (!ok) break;
                    if (grown) {
                        // new references: the columns' maxima over the four warps' keys
                        uint32_t x[kW];
                        scores(x);
                        float mine = -INFINITY;
#pragma unroll
                        for (int i = 0; i < kW; ++i) {
                            float y = __uint_as_float(x[i]);
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, o));
                            if (lane == i) mine = y;
                        }
                        if (lane < kW) sh.top[warp][c0 + lane] = mine;
                        any(false);
                        if (!ok) break;
                        if (lane < kW) {
                            float y = fmaxf(fmaxf(sh.top[0][c0 + lane], sh.top[1][c0 + lane]),
                                            fmaxf(sh.top[2][c0 + lane], sh.top[3][c0 + lane])) * scale;
                            const float old = m[c0 + lane];
                            y = y > old + kLift ? y - kLift : old;
                            f[c0 + lane] = ex2(old - y);
                            m[c0 + lane] = y;
                        }
                        __syncwarp();
                        shift(x);
#pragma unroll
                        for (int i = 0; i < kW / 2; ++i) {
                            const float2 y = *reinterpret_cast<const float2 *>(f + c0 + 2 * i);
                            l[c0 / 2 + i] = make_float2(l[c0 / 2 + i].x * y.x, l[c0 / 2 + i].y * y.y);
                        }
                        if (t > 0) {  // O holds the tiles before this one
                            ok = wait(&sh.pv_done[buf ^ 1u], (e - 1) >> 1);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int d = 0; d < kW; d += 16) {
                                uint32_t o[16];
                                tmem_load(tmem + lanes + kT4O + (uint32_t)(c0 + d), o);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f[c0 + d + i]);
                                tmem_store(tmem + lanes + kT4O + (uint32_t)(c0 + d), o);
                            }
                            tmem_wait_store();
                        }
                    }
                    if (h == kCols / kW - 1) {
                        tc_fence_before();
                        arrive(&sh.s_free[buf]);
                    }
                    if (h == 0 && e >= 2) {  // the weights of the tile before the last are through
                        ok = wait(&sh.pv_done[buf], use - 1);
                        if (!ok) break;
                    }
                    uint8_t *to = sh.p[buf] + key * C::kRowP;
                    constexpr int kSwap = C::kRowP / 16 - 1;
                    const int swap = C::kRowP == 128 ? key & 7 : C::kRowP == 64 ? (key >> 1) & 3 : (key >> 2) & 1;
                    static_assert(kSwap == 7 || kSwap == 3 || kSwap == 1, "bytes of a key's weights");
#pragma unroll
                    for (int i = 0; i < kW; i += 8) {
                        uint32_t p[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float2 w2 = make_float2(ex2(z[i / 2 + y].x), ex2(z[i / 2 + y].y));
                            l[(c0 + i) / 2 + y] = add2(l[(c0 + i) / 2 + y], w2);
                            // rounded to float16 for the product; the sum takes them unrounded, and the
                            // errors, 2^-12 each, average out
                            p[y] = pack2<SPEC_DTYPE_F16>(w2.x, w2.y);
                        }
                        *reinterpret_cast<uint4 *>(to + ((((c0 + i) / 8) ^ swap) * 16)) =
                            make_uint4(p[0], p[1], p[2], p[3]);
                    }
                }
                if (!ok) break;
                fence_proxy_async();
                tc_fence_before();
                arrive(&sh.p_full[buf]);
            }
            if (!ok) break;
            arrive(&sh.seg_free[seg_no % kTaSlots]);

            // ---- the segment's result: sums over the warp's keys, a column to a lane (two where there are 64)
            constexpr int kPerLane = kCols == 64 ? 2 : 1;
            float *part = reinterpret_cast<float *>(l);
#pragma unroll
            for (int o = 16, n = kCols; o > 0; o >>= 1) {
                if (n > kPerLane) {  // lanes o apart take half of the columns each
                    n >>= 1;
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i) {
                        if (i >= n) break;
                        const bool up = (lane & o) != 0;
                        const float give = up ? part[i] : part[i + n];
                        part[i] = (up ? part[i + n] : part[i]) + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                    }
                } else {
                    part[0] += __shfl_xor_sync(0xFFFFFFFFu, part[0], o);
                }
            }
            // lane bits from the top choose the upper halves: with 16 columns lanes 2 i and 2 i + 1 hold column i,
            // with 32 lane i column i, with 64 lane i columns 2 i and 2 i + 1
            if (kCols == 16) {
                if ((lane & 1) == 0) sh.sum[warp][lane >> 1] = part[0];
            } else {
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) sh.sum[warp][lane * kPerLane + i] = part[i];
            }
            any(false);
            const uint32_t last = e - 1;
            ok = ok && wait(&sh.pv_done[last & 1u], last >> 1);
            if (!ok) break;
            tc_fence_after();
            const bool whole_item = s.n == g.nt;
            const long long place = (long long)blockIdx.x * 2 + (s.i0 == 0 ? 1 : 0);  // a cut item's part
            for (int c = warp * 32 + lane; c < kCols; c += 128) {  // a thread per row: its sum's reciprocal and lse
                const float total = sh.sum[0][c] + sh.sum[1][c] + sh.sum[2][c] + sh.sum[3][c];
                const int r = c % RP, local = r / A.G, node = s.node0 + local, hk = s.hk * PACK + c / RP;
                const bool exists = r < rows_used && node < A.N && hk < T.heads, valid = exists && node < g.cnt;
                float ref = sh.m[0][c];
                if (total != total) ref = fmaxf(ref, 0.f);  // the row's part must not pass for empty
                sh.top[0][c] = 4.f / total;                 // (O is a quarter of itself)
                if (exists) {
                    if (whole_item) {
                        const long long orow = ((long long)s.b * A.N + node) * A.Hq + hk * A.G + (r - local * A.G);
                        if (A.lse) A.lse[orow] = ta_lse(valid, ref, total);
                    } else {
                        A.part_ml[place * rows_cta + (c / RP) * rows_used + r] =
                            valid ? make_float2(ref, total) : make_float2(-INFINITY, 0.f);
                    }
                }
            }
            any(false);
            if (!ok) break;
            const int hk = s.hk * PACK + slot;
            if (slot < PACK && hk < T.heads && ch - lane < A.D) {
                constexpr int kO = RP < 32 ? RP : 32;
                int local = 0, in_group = 0;
#pragma unroll 1
                for (int c0 = 0; c0 < rows_used; c0 += kO) {
                    uint32_t o[kO];
                    __syncwarp();
                    tmem_load(tmem + lanes + kT4O + (uint32_t)(slot * RP + c0), o);
#pragma unroll
                    for (int i = 0; i < kO; ++i) {
                        const int node = s.node0 + local;
                        if (c0 + i < rows_used && node < A.N && ch < A.D) {
                            const bool valid = node < g.cnt;
                            const float y = __uint_as_float(o[i]);
                            if (whole_item) {
                                const long long orow = ((long long)s.b * A.N + node) * A.Hq + hk * A.G + in_group;
                                A.out[orow * A.D + ch] =
                                    valid ? (uint16_t)pack2<DT>(y * sh.top[0][slot * RP + c0 + i], 0.f) : (uint16_t)0;
                            } else if (valid) {
                                A.part_o[(place * rows_cta + slot * rows_used + c0 + i) * A.D + ch] = 4.f * y;
                            }
                        }
                        if (++in_group == A.G) in_group = 0, ++local;
                    }
                }
            }
            tc_fence_before();
            arrive(&sh.o_free);
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
                for (long long i = r0 * A.D / 8 + threadIdx.x; i < r1 * A.D / 8; i += 128)
                    o[i] = make_uint4(0u, 0u, 0u, 0u);
                if (A.lse)
#pragma unroll 1
                    for (long long i = r0 + threadIdx.x; i < r1; i += 128) A.lse[i] = -INFINITY;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kT4WarpMma) {
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
    // two heads to a pack while their rows fit 64 columns, since one head of 64 leaves half of V's lanes empty
    r.pack = r.dp == 64 && heads > 1 && N * G <= 32 ? 2 : 1;
    const int most = r.pack == 2 ? 32 : 64, fit = most / G;
    const int tiles = (N + fit - 1) / fit;
    r.np = (N + tiles - 1) / tiles;
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
    static bool ready[64] = {};
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(tree_attn4<DT, DP, PACK, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess)
            return SPEC_ERR_CUDA;
        ready[dev] = true;
    }
    const spec_status_t st =
        launch_pdl(tree_attn4<DT, DP, PACK, RP>, dim3((unsigned)ctas), dim3(kT4Threads), smem, s, q, T);
    if (st != SPEC_OK) return st;
    constexpr int rows = 256 / kTaJoinLanes;
    const int used = T.a.np * T.a.G, cta = PACK * used;
    return launch_pdl(tree_attn_join<DT>, dim3((unsigned)ctas, (unsigned)((cta + rows - 1) / rows)), dim3(256), 0, s,
                      T.a, used, cta, PACK == 2 ? (int)kTaSplitHeads : (int)kTaSplitKeys);
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
        ((uintptr_t)q & 15) || ((uintptr_t)out & 15) || window < 0 || sinks < 0 || !(scale > 0.f) ||
        !(scale < 3.0e38f) || (per_head != 0 && per_head != 1))
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
    A.scale_log2 = scale * 1.44269504089f;
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
