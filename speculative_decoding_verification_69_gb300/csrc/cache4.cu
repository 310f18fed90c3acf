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
    if (n >= m) return false;
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

// Largest magnitude of a group: over a thread's 8 channels and the four threads of the group.
__device__ __forceinline__ float group_max(const float (&f)[8], uint32_t mask) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    m = fmaxf(m, __shfl_xor_sync(mask, m, 1));
    return fmaxf(m, __shfl_xor_sync(mask, m, 2));
}
template <int DT> __device__ __forceinline__ void widen(uint4 x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = unpack16<DT>(w[e]);
        f[2 * e] = y.x, f[2 * e + 1] = y.y;
    }
}

// New keys and values into the pages.  Grid (blocks of 8 tokens, requests), block (columns of
// 8 channels, token blocks).
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
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t < x.t0 || t >= x.t1) continue;
            float f[8];
            widen<DT>(k[t], f);
            uint32_t byte = scale_byte(group_max(f, group_lanes)), word = 0;
            float s = scale_of(byte);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                word |= code_of(f[e], s) << bit4(e);
                finite = finite && fabsf(f[e]) < INFINITY;
            }
            *reinterpret_cast<uint32_t *>(to + key4(P, x.tok + t, g) + (d8 & 3) * 4) = word;
            if ((d8 & 3) == 0) to[scale4(P, x.tok + t, g, false)] = (uint8_t)byte;
            widen<DT>(v[t], f);
            byte = scale_byte(group_max(f, group_lanes));
            s = scale_of(byte);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] |= code_of(f[e], s) << bit4(t);
                finite = finite && fabsf(f[e]) < INFINITY;
            }
            if ((d8 & 3) == 0) to[scale4(P, x.tok + t, g, true)] = (uint8_t)byte;
        }
        words[0] = make_uint4(w[0], w[1], w[2], w[3]);
        words[1] = make_uint4(w[4], w[5], w[6], w[7]);
        if (!finite) flag(A.status, SPEC_DEV_BAD_VALUE);
    }
}

// The numbers of a 4-bit cache.  Grid (blocks of 8 tokens, requests, layers), block as above.
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
    for (int c = threadIdx.x; c < P.heads * per; c += blockDim.x) {
        const int h = c / per, d8 = c - h * per, g = d8 >> 2;
        if (d8 >= vecs) continue;
        uint32_t kw[8], vw[8], ks[8], vs[8];
        if (there) {
            const uint8_t *from = x.at + blockIdx.z * P.layer + h * P.head;
            const uint4 *words = reinterpret_cast<const uint4 *>(from + value4(P, x.tok, d8 * 8));
            const uint4 a = words[0], z = words[1];
            vw[0] = a.x, vw[1] = a.y, vw[2] = a.z, vw[3] = a.w, vw[4] = z.x, vw[5] = z.y, vw[6] = z.z, vw[7] = z.w;
            const uint2 sk = *reinterpret_cast<const uint2 *>(from + scale4(P, x.tok, g, false));
            const uint2 sv = *reinterpret_cast<const uint2 *>(from + scale4(P, x.tok, g, true));
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                kw[t] = *reinterpret_cast<const uint32_t *>(from + key4(P, x.tok + t, g) + (d8 & 3) * 4);
                ks[t] = ((t < 4 ? sk.x : sk.y) >> (8 * (t & 3))) & 255u;
                vs[t] = ((t < 4 ? sv.x : sv.y) >> (8 * (t & 3))) & 255u;
            }
        }
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

// Accepted nodes moved behind their root.  Grid (requests, layers x heads), 128 threads.
// All that moves is read before anything is written: the keys' codes and all scales into
// registers, the values' words (which hold other tokens' codes too) into shared memory, where a
// thread takes one channel's codes from node to place in the order of the path (place <= node, so no
// code is overwritten before it is read), and writes the words back that changed.
constexpr int kC4Threads = 128, kC4Blocks = SPEC_MAX_TREE / 8 + 1;
__global__ void __launch_bounds__(kC4Threads) sv_commit4(Pool4 P, Pool ids, const int *table, const int *len,
                                                         const int *nodes, const int *accept, int *new_len, int N,
                                                         int max_pages, uint32_t *status) {
    // places as page * page_size + token
    __shared__ long long s_src[SPEC_MAX_TREE], s_dst[SPEC_MAX_TREE];
    __shared__ uint32_t words[kC4Blocks][kC4Threads];
    __shared__ int s_n, s_node[SPEC_MAX_TREE];
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x, tid = threadIdx.x;
    const bool first = blockIdx.y == 0;
    const int a = commit_path(ids, table, len, nodes, accept, b, N, max_pages, s_src, s_dst, &s_n, status, first);
    const int n0 = len[b];
    if (first && new_len && tid == 0) new_len[b] = commit_len(n0, a);
    if (a <= 0 || !nodes) return;
    if (tid < a) s_node[tid] = nodes[(long long)b * N + tid];
    uint8_t *base = P.data + (blockIdx.y / P.heads) * P.layer + (blockIdx.y % P.heads) * P.head;
    auto page_of = [&](long long id) { return base + (id >> P.page_shift) * P.page_st; };
    auto tok_of = [&](long long id) { return (int)(id & (P.page - 1)); };
    __syncthreads();
    // the blocks of 8 tokens from the root's to the last node's (a path need not be in order)
    int last = 0;
    for (int i = 0; i < a; ++i) last = max(last, s_node[i]);
    const int n8 = n0 & 7, blocks = ((n8 + last) >> 3) + 1;
    auto block_at = [&](int i) -> uint8_t * {  // nullptr: no page, so nothing moves from or to it
        const long long pos = ((long long)(n0 >> 3) + i) << 3, place = pos >> P.page_shift;
        const int p = place < max_pages ? table[(long long)b * max_pages + place] : -1;
        if ((unsigned)p >= (unsigned)P.num_pages) return nullptr;
        return base + p * P.page_st + value4(P, (int)(pos & (P.page - 1)), tid);
    };
    if (tid < P.C) {
#pragma unroll
        for (int i = 0; i < kC4Blocks; ++i) {
            if (i >= blocks) break;
            const uint8_t *w = block_at(i);
            words[i][tid] = w ? *reinterpret_cast<const uint32_t *>(w) : 0u;
        }
    }
    constexpr int kMost = (SPEC_MAX_TREE * 4 + kC4Threads - 1) / kC4Threads;
    uint4 code[kMost];
    uint8_t sk[kMost], sv[kMost];
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int x = u * kC4Threads + tid, i = x / P.groups, g = x - i * P.groups;
        if (i < a && s_src[i] != s_dst[i]) {
            const uint8_t *from = page_of(s_src[i]);
            const int t = tok_of(s_src[i]);
            code[u] = *reinterpret_cast<const uint4 *>(from + key4(P, t, g));
            sk[u] = from[scale4(P, t, g, false)];
            sv[u] = from[scale4(P, t, g, true)];
        }
    }
    if (tid < P.C) {
        uint32_t changed = 0;
        for (int i = 0; i < a; ++i) {
            const int from = n8 + s_node[i], to = n8 + 1 + i;
            if (from == to) continue;
            const uint32_t c = (words[from >> 3][tid] >> bit4(from & 7)) & 15u;
            uint32_t &w = words[to >> 3][tid];
            w = (w & ~(15u << bit4(to & 7))) | (c << bit4(to & 7));
            changed |= 1u << (to >> 3);
        }
        for (int i = 0; i < blocks; ++i)
            if ((changed >> i) & 1u) *reinterpret_cast<uint32_t *>(block_at(i)) = words[i][tid];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int x = u * kC4Threads + tid, i = x / P.groups, g = x - i * P.groups;
        if (i < a && s_src[i] != s_dst[i]) {
            uint8_t *to = page_of(s_dst[i]);
            const int t = tok_of(s_dst[i]);
            *reinterpret_cast<uint4 *>(to + key4(P, t, g)) = code[u];
            to[scale4(P, t, g, false)] = sk[u];
            to[scale4(P, t, g, true)] = sv[u];
        }
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
        N > SPEC_MAX_TREE || max_pages < 1 || (long long)P.layers * P.heads > 65535)
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
        const unsigned each = out_nodes ? (unsigned)(P.layers * P.heads) : 1u;
        const spec_status_t r = sv::launch_pdl(sv::sv_commit4, dim3((unsigned)B, each), dim3(sv::kC4Threads), 0, s, P,
                                               ids, page_table, cache_len, out_nodes, accept_len,
                                               in_place ? (int *)nullptr : new_len, N, max_pages, dev_status);
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
