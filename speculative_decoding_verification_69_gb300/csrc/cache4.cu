// cache4.cu -- writing, reading, committing, copying and forking the 4-bit cache.
//
// A block of 8 tokens is what shares bytes (a value's word holds 8 tokens of a
// channel), so the movers work on such blocks: a thread owns 8 channels of one
// head and of one block of 8 tokens, which makes every access 4, 16 or 32
// contiguous bytes and a block's words belong to one thread.  The four threads
// of a group of 32 channels lie side by side in a warp.
#include "cache4.cuh"

namespace sv {

struct Move4Args {
    Pool4 P;
    const int *table, *len, *count;
    const uint4 *k_in, *v_in;   // append
    uint4 *k_out, *v_out;       // read
    long long sb, sn, sh;       // of k_in and v_in, in 16-byte vectors
    int N, max_pages, B;
    uint32_t *status;
};

// The 8 tokens of block i of request b: where they lie, and which of them are
// among its m tokens from position n0 on.  False: the block has none, or no page.
struct Block8 {
    uint8_t *at;      // its page and head 0, layer 0
    int tok;          // its first token's place in the page
    int n;            // that token's number among the request's (may be negative)
    int t0, t1;       // its tokens [t0, t1) are meant
};
__device__ __forceinline__ bool block8(const Move4Args &A, int b, int i, int n0, int m, bool report, Block8 &x) {
    const long long first = ((long long)n0 >> 3) + i;         // the block's number in the sequence
    const long long pos = first << 3, n = pos - n0;
    if (n >= m || m <= 0) return false;  // (without tokens a block that begins before n0 has none either)
    x.n = (int)n;
    x.t0 = n < 0 ? (int)-n : 0;
    x.t1 = (int)min(8ll, m - n);
    const long long place = pos >> A.P.page_shift;
    if (place >= A.max_pages) {
        if (report) flag(A.status, SPEC_DEV_BAD_LEN);
        return false;
    }
    const int p = A.table[(long long)b * A.max_pages + place];
    if ((unsigned)p >= (unsigned)A.P.num_pages) {
        if (report) flag(A.status, SPEC_DEV_BAD_PAGE);
        return false;
    }
    x.at = A.P.data + p * A.P.page_st;
    x.tok = (int)(pos & (A.P.page - 1));
    return true;
}

template <int DT> __device__ __forceinline__ void widen(uint4 x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = unpack16<DT>(w[e]);
        f[2 * e] = y.x, f[2 * e + 1] = y.y;
    }
}

// The scale byte of a group that holds what is not finite, or out of the codes' range, and the codes of a
// thread's 8 channels in it, 4 bits each.  (Out of line: it would be half of the kernel's code.)
template <int DT> __device__ __noinline__ uint2 quantise8_any(uint4 x, uint32_t lanes) {
    float f[8], top = 0.f;
    widen<DT>(x, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));  // (of those that are numbers, infinities among them)
    top = fmaxf(top, __shfl_xor_sync(lanes, top, 1));
    const uint32_t byte = scale_byte(fmaxf(top, __shfl_xor_sync(lanes, top, 2)));
    const float s = scale_of(byte);
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) codes |= code_of(f[e], s) << (4 * e);
    return make_uint2(byte, codes);
}

// Codes of a thread's 8 channels, each handed to `put`, and the scale byte of their group of 32,
// which the four threads of the group find together.  Magnitudes are compared as whole numbers, which
// order alike, NaN above all.  Returns whether all are finite.
template <int DT, class F>
__device__ __forceinline__ bool quantise8(uint4 x, uint32_t lanes, uint32_t &byte, F &&put) {
    constexpr uint32_t kInf = DT == SPEC_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
    auto magnitude = [](uint32_t w) { return w & 0x7FFF7FFFu; };
    uint32_t m = __vmaxu2(__vmaxu2(magnitude(x.x), magnitude(x.y)), __vmaxu2(magnitude(x.z), magnitude(x.w)));
    m = __vmaxu2(m, __shfl_xor_sync(lanes, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(lanes, m, 2));
    m = max(m & 0xFFFFu, m >> 16);
    byte = scale_byte(unpack16<DT>(m).x);
    if (m < kInf && byte < 255u) {
        float f[8];
        widen<DT>(x, f);
        const float s = scale_of(byte), inv = near_reciprocal(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) put(e, code_sum(f[e], s, inv) & 15u);
        return true;
    }
    const uint2 y = quantise8_any<DT>(x, lanes);
    byte = y.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) put(e, (y.y >> (4 * e)) & 15u);
    return m < kInf;
}

// The words of a block's keys in one group, from thread j of its four holding word j of the 8 tokens to
// holding word a of token 2 j + b at 2 a + b, or back.
__device__ __forceinline__ void exchange(uint32_t (&w)[8], int j, uint32_t lanes) {
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {
        const bool up = (j & o) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if ((i >> 1) & o) continue;
            const uint32_t give = up ? w[i] : w[i + 2 * o];
            const uint32_t got = __shfl_xor_sync(lanes, give, o);
            if (up) w[i] = got;
            else w[i + 2 * o] = got;
        }
    }
}

// New keys and values into the pages.  Grid (blocks of 8 tokens, requests), block (columns of
// 8 channels, token blocks).  55 us for 32752 tokens of 8 heads of 128, 3.1 TB/s of the 170 MB (92 us with divisions,
// and with 4-byte stores of the keys).  A thread loads its 16 vectors, then quantises: its 109 registers leave two CTAs
// to an SM, too few warps (23 % of those that fit) to load while others compute, so neither HBM (31 %) nor the
// issue slots (50 %, the integer pipe 45 %) are full, and warps wait for loads and shuffles.  A step of 9 tokens for 8
// requests is a launch, 6.6 us.
template <int DT> __global__ void __launch_bounds__(256) sv_append4(const __grid_constant__ Move4Args A) {
    pdl_trigger();
    pdl_wait();
    const Pool4 &P = A.P;
    const int b = blockIdx.y, n0 = A.len[b], m = A.count ? max(0, min(A.count[b], A.N)) : A.N;
    if (n0 < 0) {
        if (threadIdx.x == 0 && threadIdx.y == 0) flag(A.status, SPEC_DEV_BAD_LEN);
        return;
    }
    Block8 x;
    if (!block8(A, b, blockIdx.x * blockDim.y + threadIdx.y, n0, m, threadIdx.x == 0, x)) return;
    const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
    const uint32_t group_lanes = 0xFu << (lane & 28);  // (rows of threads are multiples of 4 wide)
    const int per = P.C >> 3;
    for (int c = threadIdx.x; c < P.heads * per; c += blockDim.x) {
        const int h = c / per, d8 = c - h * per, g = d8 >> 2;
        uint8_t *to = x.at + h * P.head;
        const bool real = d8 * 8 < P.D;
        const long long from = (long long)b * A.sb + x.n * A.sn + h * A.sh + d8;
        uint4 k[8], v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            k[t] = v[t] = make_uint4(0u, 0u, 0u, 0u);
            if (real && t >= x.t0 && t < x.t1) {
                k[t] = ld_stream_v4(A.k_in + from + t * A.sn);
                v[t] = ld_stream_v4(A.v_in + from + t * A.sn);
            }
        }
        uint4 *words = reinterpret_cast<uint4 *>(to + value4(P, x.tok, d8 * 8));
        uint32_t w[8] = {};
        if (x.t1 - x.t0 < 8) {  // the block's other tokens stay
            const uint4 a = words[0], z = words[1];
            uint32_t keep = 0;
#pragma unroll
            for (int t = 0; t < 8; ++t)
                if (t < x.t0 || t >= x.t1) keep |= 15u << bit4(t);
            w[0] = a.x & keep, w[1] = a.y & keep, w[2] = a.z & keep, w[3] = a.w & keep;
            w[4] = z.x & keep, w[5] = z.y & keep, w[6] = z.z & keep, w[7] = z.w & keep;
        }
        bool finite = true;
        const bool whole = x.t1 - x.t0 == 8;
        uint32_t kw[8] = {}, bytes[2][2] = {};  // words of the keys; scales of keys and values, a byte for each token
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t < x.t0 || t >= x.t1) continue;
            uint32_t byte;
            finite = quantise8<DT>(k[t], group_lanes, byte, [&](int e, uint32_t c) { kw[t] |= c << bit4(e); }) && finite;
            bytes[0][t >> 2] |= byte << (8 * (t & 3));
            finite = quantise8<DT>(v[t], group_lanes, byte, [&](int e, uint32_t c) { w[e] |= c << bit4(t); }) && finite;
            bytes[1][t >> 2] |= byte << (8 * (t & 3));
        }
        uint8_t *codes = to + key4(P, x.tok, g);
        if (whole) {
            // each of a group's four threads writes two tokens: 32 bytes, not eight times 4 beside other threads'
            const int j = d8 & 3;
            exchange(kw, j, group_lanes);
            uint4 *two = reinterpret_cast<uint4 *>(codes) + 2 * j;
            two[0] = make_uint4(kw[0], kw[2], kw[4], kw[6]);
            two[1] = make_uint4(kw[1], kw[3], kw[5], kw[7]);
            if (j < 2)
                *reinterpret_cast<uint2 *>(to + scale4(P, x.tok, g, j == 1)) =
                    j == 1 ? make_uint2(bytes[1][0], bytes[1][1]) : make_uint2(bytes[0][0], bytes[0][1]);
        } else {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (t < x.t0 || t >= x.t1) continue;
                *reinterpret_cast<uint32_t *>(codes + t * 16 + (d8 & 3) * 4) = kw[t];
                if ((d8 & 3) < 2)
                    to[scale4(P, x.tok + t, g, (d8 & 3) == 1)] =
                        (uint8_t)((d8 & 3) == 1 ? bytes[1][t >> 2] >> (8 * (t & 3)) : bytes[0][t >> 2] >> (8 * (t & 3)));
            }
        }
        words[0] = make_uint4(w[0], w[1], w[2], w[3]);
        words[1] = make_uint4(w[4], w[5], w[6], w[7]);
        if (!finite) flag(A.status, SPEC_DEV_BAD_VALUE);
    }
}

// The numbers of a 4-bit cache.  Grid (blocks of 8 tokens, requests, layers), block as above.  35 us for the 170 MB of
// 32752 tokens of 8 heads of 128, 4.8 TB/s; 78 us for 64 requests of 32 tokens in 36 layers, the same rate.  Codes are
// converted one by one, which takes 62 % of the integer pipe with two CTAs to an SM (94 registers); HBM is busy for 38 to
// 55 % of the time.
template <int DT> __global__ void __launch_bounds__(256) sv_read4(const __grid_constant__ Move4Args A) {
    pdl_trigger();
    pdl_wait();
    const Pool4 &P = A.P;
    const int b = blockIdx.y, m = A.count ? max(0, min(A.count[b], A.N)) : A.N;
    int n0 = A.len[b];
    const bool bad = n0 < 0;
    if (bad) {
        if (threadIdx.x == 0 && threadIdx.y == 0) flag(A.status, SPEC_DEV_BAD_LEN);
        n0 = 0;
    }
    const int i = blockIdx.x * blockDim.y + threadIdx.y;
    Block8 x;
    const bool there = block8(A, b, i, n0, bad ? 0 : m, threadIdx.x == 0 && blockIdx.z == 0, x);
    // rows of this block, there or not
    const long long first = (((long long)n0 >> 3) + i) * 8 - n0;
    const int t0 = first < 0 ? (int)-first : 0, t1 = (int)min(8ll, A.N - first);
    if (t1 <= t0) return;
    const int per = P.C >> 3, vecs = P.D >> 3;
    const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
    const uint32_t group_lanes = 0xFu << (lane & 28);
    for (int c = threadIdx.x; c < P.heads * per; c += blockDim.x) {
        const int h = c / per, d8 = c - h * per, g = d8 >> 2;
        uint32_t kw[8], vw[8], ks[8], vs[8];
        if (there) {
            const uint8_t *from = x.at + blockIdx.z * P.layer + h * P.head;
            const uint4 *words = reinterpret_cast<const uint4 *>(from + value4(P, x.tok, d8 * 8));
            const uint4 *two = reinterpret_cast<const uint4 *>(from + key4(P, x.tok, g)) + 2 * (d8 & 3);
            const uint4 a = words[0], z = words[1], y0 = two[0], y1 = two[1];
            const uint2 sk = *reinterpret_cast<const uint2 *>(from + scale4(P, x.tok, g, false));
            const uint2 sv = *reinterpret_cast<const uint2 *>(from + scale4(P, x.tok, g, true));
            vw[0] = a.x, vw[1] = a.y, vw[2] = a.z, vw[3] = a.w, vw[4] = z.x, vw[5] = z.y, vw[6] = z.z, vw[7] = z.w;
            kw[0] = y0.x, kw[2] = y0.y, kw[4] = y0.z, kw[6] = y0.w, kw[1] = y1.x, kw[3] = y1.y, kw[5] = y1.z, kw[7] = y1.w;
            exchange(kw, d8 & 3, group_lanes);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                ks[t] = ((t < 4 ? sk.x : sk.y) >> (8 * (t & 3))) & 255u;
                vs[t] = ((t < 4 ? sv.x : sv.y) >> (8 * (t & 3))) & 255u;
            }
        }
        if (d8 >= vecs) continue;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t < t0 || t >= t1) continue;
            uint32_t k[4] = {}, v[4] = {};
            if (there && t >= x.t0 && t < x.t1) {
                const float s = scale_of(ks[t]), u = scale_of(vs[t]);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    auto num = [](uint32_t w, int bit, float y) { return ((float)((w >> bit) & 15u) - 8.f) * y; };
                    k[e / 2] = pack16<DT>(num(kw[t], bit4(e), s), num(kw[t], bit4(e + 1), s));
                    v[e / 2] = pack16<DT>(num(vw[e], bit4(t), u), num(vw[e + 1], bit4(t), u));
                }
            }
            const long long row = ((long long)blockIdx.z * A.B + b) * A.N + first + t;
            const long long to = (row * P.heads + h) * vecs + d8;
            A.k_out[to] = make_uint4(k[0], k[1], k[2], k[3]);
            A.v_out[to] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

// Accepted nodes moved behind their root.  Grid (requests, shares of the layers and heads): a CTA finds the
// request's path and the places of its pieces once, then a warp takes a layer and head at a time.
// All that moves is read before anything is written: the keys' codes and all scales into
// registers, the values' words (which hold other tokens' codes too) into shared memory, where a
// lane takes four channels' codes from node to place in the order of the path (place <= node, so no
// code is overwritten before it is read), and writes the words back that changed.  28.7 us for 64 requests of 32
// nodes, 36 layers of 8 heads (a thread per channel took 77), 46 MB from HBM: bound by latency (HBM 20 %, issue slots
// 16 %), since a warp reads a layer and head only when it has written the one before.
constexpr int kC4Warps = 8, kC4Blocks = SPEC_MAX_TREE / 8 + 1, kC4Pieces = SPEC_MAX_TREE * 4;
struct Piece4 {  // 16 bytes of codes of a moved key, and the scales beside them: offsets from a layer's head
    long long src, dst;
    int src_scale, dst_scale;  // from those: of the key; the value's lies `groups` blocks on
};
__global__ void __launch_bounds__(kC4Warps * 32) sv_commit4(Pool4 P, Pool ids, const int *table, const int *len,
                                                            const int *nodes, const int *accept, int *new_len, int N,
                                                            int max_pages, uint32_t *status) {
    // places as page * page_size + token
    __shared__ long long s_src[SPEC_MAX_TREE], s_dst[SPEC_MAX_TREE], s_block[kC4Blocks];
    __shared__ Piece4 pieces[kC4Pieces];
    __shared__ uint4 words[kC4Warps][kC4Blocks][32];
    __shared__ int s_n, s_move[SPEC_MAX_TREE], s_last;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const bool first = blockIdx.y == 0;
    const int a = commit_path(ids, table, len, nodes, accept, b, N, max_pages, s_src, s_dst, &s_n, status, first);
    const int n0 = len[b], n8 = n0 & 7;
    if (first && new_len && tid == 0) new_len[b] = commit_len(n0, a);
    if (a <= 0 || !nodes) return;
    if (tid == 0) s_last = 0;
    __syncthreads();
    if (tid < a) {  // the blocks and bits that node tid's codes move between
        const int node = nodes[(long long)b * N + tid], from = n8 + node, to = n8 + 1 + tid;
        s_move[tid] = (from >> 3) | bit4(from & 7) << 8 | (to >> 3) << 16 | bit4(to & 7) << 24;
        atomicMax(&s_last, node);  // (a path need not be in order)
    }
    if (tid < kC4Blocks) {  // the blocks of 8 tokens from the root's on; -1: no page, so nothing moves from or to it
        const long long pos = ((long long)(n0 >> 3) + tid) << 3, place = pos >> P.page_shift;
        const int p = place < max_pages ? table[(long long)b * max_pages + place] : -1;
        s_block[tid] = (unsigned)p < (unsigned)P.num_pages
                           ? (long long)p * P.page_st + value4(P, (int)(pos & (P.page - 1)), 0)
                           : -1ll;
    }
    const int count = a * P.groups;
    for (int x = tid; x < count; x += kC4Warps * 32) {
        const int i = x / P.groups, g = x - i * P.groups;
        Piece4 y;
        auto place = [&](long long id, long long &at, int &scale) {
            const int tok = (int)(id & (P.page - 1)), key = key4(P, tok, g);
            at = (id >> P.page_shift) * P.page_st + key;
            scale = scale4(P, tok, g, false) - key;
        };
        place(s_src[i], y.src, y.src_scale);
        place(s_dst[i], y.dst, y.dst_scale);
        pieces[x] = y;
    }
    __syncthreads();
    const int blocks = ((n8 + s_last) >> 3) + 1, value_scale = P.groups * P.block;
    uint4(&w)[kC4Blocks][32] = words[tid >> 5];
    for (int item = blockIdx.y * kC4Warps + (tid >> 5); item < P.layers * P.heads; item += gridDim.y * kC4Warps) {
        uint8_t *base = P.data + item / P.heads * P.layer + item % P.heads * P.head;
        const bool mine = lane * 4 < P.C;
        if (mine) {
#pragma unroll
            for (int i = 0; i < kC4Blocks; ++i) {
                if (i >= blocks) break;
                w[i][lane] = s_block[i] >= 0 ? *reinterpret_cast<const uint4 *>(base + s_block[i] + lane * 16)
                                             : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        constexpr int kMost = kC4Pieces / 32;
        uint4 code[kMost];
        uint8_t sk[kMost], sv[kMost];
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            if (u * 32 >= count) break;
            if (u * 32 + lane < count) {
                const Piece4 &y = pieces[u * 32 + lane];
                const uint8_t *from = base + y.src;
                code[u] = *reinterpret_cast<const uint4 *>(from);
                sk[u] = from[y.src_scale];
                sv[u] = from[y.src_scale + value_scale];
            }
        }
        __syncwarp();
        if (mine) {
            uint32_t changed = 0;
            for (int i = 0; i < a; ++i) {
                const int move = s_move[i], from = move & 255, to = (move >> 16) & 255;
                const int right = (move >> 8) & 255, left = move >> 24;
                if (from == to && right == left) continue;
                const uint4 x = w[from][lane];
                uint4 y = w[to][lane];
                const uint32_t keep = ~(15u << left);
                y.x = (y.x & keep) | ((x.x >> right) & 15u) << left;
                y.y = (y.y & keep) | ((x.y >> right) & 15u) << left;
                y.z = (y.z & keep) | ((x.z >> right) & 15u) << left;
                y.w = (y.w & keep) | ((x.w >> right) & 15u) << left;
                w[to][lane] = y;
                changed |= 1u << to;
            }
            for (int i = 0; i < blocks; ++i)
                if ((changed >> i) & 1u) *reinterpret_cast<uint4 *>(base + s_block[i] + lane * 16) = w[i][lane];
        }
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            if (u * 32 >= count) break;
            if (u * 32 + lane < count) {
                const Piece4 &y = pieces[u * 32 + lane];
                if (y.src == y.dst) continue;
                uint8_t *to = base + y.dst;
                *reinterpret_cast<uint4 *>(to) = code[u];
                to[y.dst_scale] = sk[u];
                to[y.dst_scale + value_scale] = sv[u];
            }
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------ host

spec_status_t make_pool4(const spec_pages4_t *p, Pool4 &P) {
    if (!p || !p->data) return SPEC_ERR_INVALID_ARG;
    const size_t bytes = spec_cache4_page_bytes(p->page_size, p->head_dim);
    if (p->layers < 1 || p->layers > 65535 || p->num_pages < 1 || p->num_pages == INT_MAX || bytes == 0 ||
        p->heads < 1 || p->heads > 1024 || ((uintptr_t)p->data & 15))
        return SPEC_ERR_INVALID_ARG;
    const long long st[3] = {p->layer_stride, p->page_stride, p->head_stride};
    const int extent[3] = {p->layers, p->num_pages, p->heads};
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || st[i] % 16) return SPEC_ERR_INVALID_ARG;
        if (extent[i] == 1) continue;
        __int128 reach = bytes;  // no two pages and heads may share a place
        for (int j = 0; j < 3; ++j)
            if (j != i && st[j] <= st[i]) reach += (__int128)(extent[j] - 1) * st[j];
        if (st[i] < reach) return SPEC_ERR_INVALID_ARG;
    }
    P.data = static_cast<uint8_t *>(p->data);
    P.layer = p->layer_stride;
    P.page_st = p->page_stride;
    P.head = p->head_stride;
    P.layers = p->layers;
    P.num_pages = p->num_pages;
    P.page = p->page_size;
    P.page_shift = 0;
    while ((1 << P.page_shift) < P.page) ++P.page_shift;
    P.heads = p->heads;
    P.D = p->head_dim;
    P.C = (p->head_dim + 31) / 32 * 32;
    P.groups = P.C / 32;
    P.block = P.page < 128 ? P.page : 128;
    P.bytes = P.block * P.C / 16 * 17;
    return SPEC_OK;
}

// The pool for copies of whole pages: a page and head as rows ("tokens") of 272 bytes, of which "keys" are
// the first 9 vectors and "values" the last 9.  (The middle one is both, and copied twice alike.)
static Pool copy_pool(const Pool4 &P) {
    Pool Q = {};
    Q.k = reinterpret_cast<uint4 *>(P.data);
    Q.v = Q.k + 8;
    Q.layer = P.layer / 16;
    Q.page_st = P.page_st / 16;
    Q.token = 17;
    Q.head = P.head / 16;
    Q.layers = P.layers;
    Q.num_pages = P.num_pages;
    Q.page = P.page / P.block * P.bytes / 272;
    Q.vecs = 9;
    Q.cols = P.heads * 9;
    return Q;
}

static bool dtype16(int dt) { return dt == SPEC_DTYPE_BF16 || dt == SPEC_DTYPE_F16; }

// Threads over the columns of 8 channels, a multiple of 4 of them, and over blocks of 8 tokens.
static dim3 block4_shape(const Pool4 &P) {
    const int cols = P.heads * (P.C / 8), x = cols < 256 ? cols : 256;
    return dim3((unsigned)x, (unsigned)(256 / x));
}

} // namespace sv

extern "C" {

size_t spec_cache4_page_bytes(int page_size, int head_dim) {
    if (page_size < 8 || page_size > (1 << 20) || (page_size & (page_size - 1)) || head_dim < 8 || head_dim % 8 ||
        head_dim > SPEC_MAX_HEAD_DIM)
        return 0;
    return (size_t)page_size * ((head_dim + 31) / 32 * 32) / 16 * 17;
}

spec_status_t spec_cache4_append(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *cache_len,
                                 const void *k_new, const void *v_new, spec_dtype_t dtype, long long new_stride_b,
                                 long long new_stride_n, long long new_stride_h, const int32_t *count, int B, int N,
                                 int max_pages, uint32_t *dev_status, void *stream) {
    sv::Move4Args A = {};
    const spec_status_t st = sv::make_pool4(pages, A.P);
    if (st != SPEC_OK) return st;
    if (!sv::dtype16(dtype)) return SPEC_ERR_UNSUPPORTED;
    if (A.P.layers != 1 || !page_table || !cache_len || !k_new || !v_new || ((uintptr_t)k_new & 15) ||
        ((uintptr_t)v_new & 15) || new_stride_b < 0 || new_stride_n < 0 || new_stride_h < 0 || new_stride_b % 8 ||
        new_stride_n % 8 || new_stride_h % 8 || B < 1 || B >= (1 << 16) || N < 1 || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    A.table = page_table;
    A.len = cache_len;
    A.count = count;
    A.k_in = static_cast<const uint4 *>(k_new);
    A.v_in = static_cast<const uint4 *>(v_new);
    A.sb = new_stride_b / 8;
    A.sn = new_stride_n / 8;
    A.sh = new_stride_h / 8;
    A.B = B;
    A.N = N;
    A.max_pages = max_pages;
    A.status = dev_status;
    const dim3 block = sv::block4_shape(A.P);
    const unsigned blocks = (unsigned)(N / 8) + 2u;  // that N tokens may touch
    const dim3 grid((blocks + block.y - 1) / block.y, (unsigned)B);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_DTYPE_BF16 ? sv::launch_pdl(sv::sv_append4<SPEC_DTYPE_BF16>, grid, block, 0, s, A)
                                    : sv::launch_pdl(sv::sv_append4<SPEC_DTYPE_F16>, grid, block, 0, s, A);
}

spec_status_t spec_cache4_read(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *start,
                               const int32_t *count, void *k, void *v, spec_dtype_t dtype, int B, int N,
                               int max_pages, uint32_t *dev_status, void *stream) {
    sv::Move4Args A = {};
    const spec_status_t st = sv::make_pool4(pages, A.P);
    if (st != SPEC_OK) return st;
    if (!sv::dtype16(dtype)) return SPEC_ERR_UNSUPPORTED;
    if (!page_table || !start || !k || !v || ((uintptr_t)k & 15) || ((uintptr_t)v & 15) || B < 1 || B >= (1 << 16) ||
        N < 1 || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    A.table = page_table;
    A.len = start;
    A.count = count;
    A.k_out = static_cast<uint4 *>(k);
    A.v_out = static_cast<uint4 *>(v);
    A.B = B;
    A.N = N;
    A.max_pages = max_pages;
    A.status = dev_status;
    const dim3 block = sv::block4_shape(A.P);
    const unsigned blocks = (unsigned)(N / 8) + 2u;
    const dim3 grid((blocks + block.y - 1) / block.y, (unsigned)B, (unsigned)A.P.layers);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_DTYPE_BF16 ? sv::launch_pdl(sv::sv_read4<SPEC_DTYPE_BF16>, grid, block, 0, s, A)
                                    : sv::launch_pdl(sv::sv_read4<SPEC_DTYPE_F16>, grid, block, 0, s, A);
}

spec_status_t spec_cache4_commit(const spec_pages4_t *pages, const int32_t *page_table, const int32_t *cache_len,
                                 const int32_t *out_nodes, const int32_t *accept_len, int32_t *new_len, int B, int N,
                                 int max_pages, uint32_t *dev_status, void *stream) {
    sv::Pool4 P;
    const spec_status_t st = sv::make_pool4(pages, P);
    if (st != SPEC_OK) return st;
    if (!page_table || !cache_len || !accept_len || !new_len || B < 1 || B >= (1 << 16) || N < 1 ||
        N > SPEC_MAX_TREE || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    sv::Pool ids = {};  // in which a place's offset is its number
    ids.page_st = P.page;
    ids.token = 1;
    ids.num_pages = P.num_pages;
    ids.page = P.page;
    ids.page_shift = P.page_shift;
    const bool in_place = new_len == cache_len;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (out_nodes || !in_place) {
        int dev = 0, sms = 0;
        if (!sv::current_device(dev, sms)) return SPEC_ERR_CUDA;
        // about four CTAs to an SM: more would find the paths anew
        const long long shares = ((long long)P.layers * P.heads + sv::kC4Warps - 1) / sv::kC4Warps, fit = 4 * sms / B + 1;
        const unsigned each = out_nodes ? (unsigned)(shares < fit ? shares : fit) : 1u;
        const spec_status_t r = sv::launch_pdl(sv::sv_commit4, dim3((unsigned)B, each),
                                               dim3(sv::kC4Warps * 32), 0, s, P, ids, page_table, cache_len,
                                               out_nodes, accept_len, in_place ? (int *)nullptr : new_len, N,
                                               max_pages, dev_status);
        if (r != SPEC_OK || !in_place) return r;
    }
    return sv::launch_commit_len(ids, page_table, new_len, out_nodes, accept_len, B, N, max_pages, dev_status, s);
}

spec_status_t spec_cache4_copy(const spec_pages4_t *pages, const int32_t *src_pages, const int32_t *dst_pages, int n,
                               uint32_t *dev_status, void *stream) {
    sv::Pool4 P;
    const spec_status_t st = sv::make_pool4(pages, P);
    if (st != SPEC_OK) return st;
    if (!src_pages || !dst_pages || n < 1) return SPEC_ERR_INVALID_ARG;
    return sv::launch_copy(sv::copy_pool(P), src_pages, dst_pages, nullptr, n, dev_status,
                           static_cast<cudaStream_t>(stream));
}

spec_status_t spec_cache4_fork(const spec_pages4_t *pages, int32_t *page_table, int32_t *page_count,
                               int32_t *page_ref, int32_t *cache_len, const int32_t *src, const int32_t *dst, int F,
                               int slots, int max_pages, void *workspace, size_t workspace_bytes,
                               uint32_t *dev_status, void *stream) {
    sv::Pool4 P;
    const spec_status_t st = sv::make_pool4(pages, P);
    if (st != SPEC_OK) return st;
    if (!page_table || !page_count || !page_ref || !cache_len || !src || !dst || F < 1 || F > SPEC_MAX_SLOTS ||
        slots < 1 || slots > SPEC_MAX_SLOTS || max_pages < 1)
        return SPEC_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < spec_cache_fork_workspace_bytes(F))
        return SPEC_ERR_WORKSPACE;
    const sv::Pool Q = sv::copy_pool(P);
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
    A.whole = Q.page;
    A.status = dev_status;
    return sv::launch_fork(A, Q, static_cast<cudaStream_t>(stream));
}

} // extern "C"
