// tree_attn4.cu -- attention of drafted trees over a 4-bit paged cache.
//
// First form: a warp per row, a key at a time, with the running maximum and sum
// of the softmax.
#include "cache4.cuh"

namespace sv {

struct T4Args {
    Pool4 P;
    const uint16_t *q;
    long long qb, qn, qh;
    const int *table, *len, *parent, *node_count;
    long long row_b, row_h;  // strides of the table's rows
    int B, N, Hq, G, max_pages, window, sinks;
    float scale_log2;
    uint16_t *out;
    float *lse;
    uint32_t *status;
};

template <int DT> __global__ void __launch_bounds__(256) tree_attn4_rows(const __grid_constant__ T4Args A) {
    pdl_trigger();
    pdl_wait();
    const Pool4 &P = A.P;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (long long)A.B * A.N * A.Hq) return;
    const int hq = (int)(row % A.Hq), n = (int)(row / A.Hq % A.N), b = (int)(row / A.Hq / A.N), h = hq / A.G;
    const long long cap = min((long long)A.max_pages << P.page_shift, (1ll << 31) - 256);
    int cnt = A.node_count ? max(0, min(A.node_count[b], A.N)) : A.N;
    int c = A.len[b];
    if (c < 0 || c > cap - cnt) {
        if (lane == 0) flag(A.status, SPEC_DEV_BAD_LEN);
        c = (int)max(0ll, min((long long)c, cap));
        cnt = (int)min((long long)cnt, cap - c);
    }
    uint16_t *out = A.out + row * P.D;
    if (n >= cnt) {
        for (int d = lane; d < P.D; d += 32) out[d] = 0;
        if (A.lse && lane == 0) A.lse[row] = -INFINITY;
        return;
    }
    unsigned long long path = 0;
    int depth = 0;
    for (int m = n;;) {
        path |= 1ull << m;
        if (m == 0) break;
        const int up = A.parent ? A.parent[(long long)b * A.N + m] : m - 1;
        if ((unsigned)up >= (unsigned)m) {
            if (lane == 0) flag(A.status, SPEC_DEV_BAD_TREE);
            break;
        }
        m = up;
        ++depth;
    }
    const int low = A.window ? max(0, c + depth + 1 - A.window) : 0, sinks = A.window ? A.sinks : 0;
    const int *table = A.table + b * A.row_b + h * A.row_h;
    const uint16_t *q = A.q + b * A.qb + n * A.qn + hq * A.qh;
    float qf[4], o[4] = {};
    for (int g = 0; g < 4; ++g) {
        const int d = g * 32 + lane;
        qf[g] = d < P.D ? unpack16<DT>(q[d]).x : 0.f;
    }
    float m = -INFINITY, l = 0.f;
    int place = 0;  // along the path
    for (int j = 0; j < c + cnt; ++j) {
        if (j < c) {
            if (j < low && j >= sinks) continue;
        } else {
            if (!((path >> (j - c)) & 1ull)) continue;
            const int at = c + place++;
            if (at < low && at >= sinks) continue;
        }
        int p = table[j >> P.page_shift];
        if ((unsigned)p >= (unsigned)P.num_pages) {
            if (lane == 0) flag(A.status, SPEC_DEV_BAD_PAGE);
            p = 0;
        }
        const int tok = j & (P.page - 1);
        const uint8_t *x = P.data + p * P.page_st + h * P.head;
        float s = 0.f;
        for (int g = 0; g < P.groups; ++g) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(x + key4(P, tok, g) + (lane >> 3) * 4);
            s = fmaf(qf[g], ((float)((w >> bit4(lane & 7)) & 15u) - 8.f) * scale_of(x[scale4(P, tok, g, false)]), s);
        }
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, i);
        s *= A.scale_log2;
        if (s == -INFINITY) {
            m = fmaxf(m, -FLT_MAX);  // seen, weight 0
            continue;
        }
        const float top = fmaxf(m, s), f = m == -INFINITY ? 0.f : ex2(m - top), e = ex2(s - top);
        m = top;
        l = fmaf(l, f, e);
        for (int g = 0; g < P.groups; ++g) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(x + value4(P, tok, g * 32 + lane));
            const float v = ((float)((w >> bit4(tok & 7)) & 15u) - 8.f) * scale_of(x[scale4(P, tok, g, true)]);
            o[g] = fmaf(o[g], f, e * v);
        }
    }
    for (int g = 0; g < P.groups; ++g) {
        const int d = g * 32 + lane;
        if (d < P.D) out[d] = (uint16_t)pack16<DT>(o[g] / l, 0.f);
    }
    if (A.lse && lane == 0) A.lse[row] = l > 0.f ? 0.69314718056f * (m + log2f(l)) : __uint_as_float(0x7FFFFFFFu);
}

} // namespace sv

extern "C" {

size_t spec_tree_attention4_workspace_bytes(int B, int N, int Hq, int heads, int head_dim) {
    if (B < 1 || B >= (1 << 16) || N < 1 || N > SPEC_MAX_TREE || heads < 1 || heads > 1024 || Hq < heads ||
        Hq % heads || Hq / heads > 64 || head_dim < 8 || head_dim % 8 || head_dim > SPEC_MAX_HEAD_DIM)
        return 0;
    return 256;
}

spec_status_t spec_tree_attention4(const void *q, spec_dtype_t dtype, long long q_stride_b, long long q_stride_n,
                                   long long q_stride_h, const spec_pages4_t *pages, const int32_t *page_table,
                                   int per_head, const int32_t *cache_len, const int32_t *parent,
                                   const int32_t *node_count, int B, int N, int Hq, int max_pages, float scale,
                                   int window, int sinks, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, uint32_t *dev_status, void *stream) {
    sv::T4Args A = {};
    const spec_status_t st = sv::make_pool4(pages, A.P);
    if (st != SPEC_OK) return st;
    if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    const int D = pages->head_dim, H = pages->heads;
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
    A.q = static_cast<const uint16_t *>(q);
    A.qb = q_stride_b;
    A.qn = q_stride_n;
    A.qh = q_stride_h;
    A.table = page_table;
    A.len = cache_len;
    A.parent = parent;
    A.node_count = node_count;
    A.row_b = (long long)max_pages * (per_head ? H : 1);
    A.row_h = per_head ? max_pages : 0;
    A.B = B;
    A.N = N;
    A.Hq = Hq;
    A.G = Hq / H;
    A.max_pages = max_pages;
    A.window = window;
    A.sinks = sinks;
    A.scale_log2 = scale * 1.44269504089f;
    A.out = static_cast<uint16_t *>(out);
    A.lse = lse;
    A.status = dev_status;
    const unsigned ctas = (unsigned)(((long long)B * N * Hq + 7) / 8);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_DTYPE_BF16
               ? sv::launch_pdl(sv::tree_attn4_rows<SPEC_DTYPE_BF16>, dim3(ctas), dim3(256), 0, s, A)
               : sv::launch_pdl(sv::tree_attn4_rows<SPEC_DTYPE_F16>, dim3(ctas), dim3(256), 0, s, A);
}

} // extern "C"
