// tree_attn.cu -- attention of drafted trees over a paged key/value cache.
#include <cuda_fp16.h>

#include "spec_cache.h"
#include "sv_cache.cuh"

namespace sv {

template <int DT> __device__ __forceinline__ float to_float(uint16_t x);
template <> __device__ __forceinline__ float to_float<SPEC_DTYPE_BF16>(uint16_t x) {
    return __uint_as_float((uint32_t)x << 16);
}
template <> __device__ __forceinline__ float to_float<SPEC_DTYPE_F16>(uint16_t x) {
    return __half2float(__ushort_as_half(x));
}
template <int DT> __device__ __forceinline__ uint16_t from_float(float x);
template <> __device__ __forceinline__ uint16_t from_float<SPEC_DTYPE_BF16>(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <> __device__ __forceinline__ uint16_t from_float<SPEC_DTYPE_F16>(float x) {
    return __half_as_ushort(__float2half_rn(x));
}

struct AttnArgs {
    const uint16_t *q;
    long long qb, qn, qh;
    Pool P;  // strides in elements here
    const int *table, *len, *parent, *node_count;
    int B, N, Hq, D, max_pages, window, sinks;
    float scale_log2;
    uint16_t *out;
    float *lse;
    uint32_t *status;
};

// One warp per (request, node, query head): lanes share the head dimension, the
// keys one after another with the running maximum and sum of a softmax.
template <int DT>
__global__ void __launch_bounds__(32) sv_tree_attn(AttnArgs A) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x;
    const int h = blockIdx.x % A.Hq, n = blockIdx.x / A.Hq, b = blockIdx.y;
    const int G = A.Hq / (A.P.cols / A.P.vecs), hk = h / G;
    const int cap = (int)min((long long)A.max_pages << A.P.page_shift, 0x7FFFFFFFll);
    int cnt = A.node_count ? max(0, min(A.node_count[b], A.N)) : A.N;
    int c = A.len[b];
    if (c < 0 || c > cap - cnt) {
        if (lane == 0) flag(A.status, SPEC_DEV_BAD_LEN);
        c = max(0, min(c, cap));
        cnt = min(cnt, cap - c);
    }
    uint16_t *o = A.out + (((long long)b * A.N + n) * A.Hq + h) * A.D;
    float *l_out = A.lse ? A.lse + ((long long)b * A.N + n) * A.Hq + h : nullptr;
    if (n >= cnt) {
        for (int d = lane; d < A.D; d += 32) o[d] = 0;
        if (lane == 0 && l_out) *l_out = -INFINITY;
        return;
    }
    // the path, as a mask of nodes and their depths
    const int *par = A.parent ? A.parent + (long long)b * A.N : nullptr;
    auto up = [&](int m) -> int {
        const int p = par ? par[m] : m - 1;
        if (m > 0 && (unsigned)p >= (unsigned)m) {
            flag(A.status, SPEC_DEV_BAD_TREE);
            return -1;
        }
        return m > 0 ? p : -1;
    };
    unsigned long long anc = 0;
    int depth = -1;
    for (int m = n; m >= 0; m = up(m)) {
        anc |= 1ull << m;
        ++depth;
    }
    float q[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint16_t *qp = A.q + b * A.qb + n * A.qn + h * A.qh;
#pragma unroll
    for (int u = 0; u < 4; ++u) q[u] = lane + 32 * u < A.D ? to_float<DT>(qp[lane + 32 * u]) : 0.f;
    const uint16_t *kp = reinterpret_cast<const uint16_t *>(A.P.k), *vp = reinterpret_cast<const uint16_t *>(A.P.v);
    float m_run = -INFINITY, l_run = 0.f;
    const int tip = c + depth;
    const int low = A.window ? max(0, tip - A.window + 1) : 0;
    int up_depth = depth;
    (void)up_depth;
    for (int j = 0; j < c + cnt; ++j) {
        int place = j;
        if (j >= c) {
            if (!((anc >> (j - c)) & 1ull)) continue;
            place = c + __popcll(anc & ((2ull << (j - c)) - 1ull)) - 1;
        }
        if (place < low && place >= A.sinks) {
            if (j < c) j = min(low, c) - 1;
            continue;
        }
        int p = A.table[(long long)b * A.max_pages + (j >> A.P.page_shift)];
        if ((unsigned)p >= (unsigned)A.P.num_pages) {
            if (lane == 0) flag(A.status, SPEC_DEV_BAD_PAGE);
            p = 0;
        }
        const long long at = p * A.P.page_st + (j & (A.P.page - 1)) * A.P.token + hk * A.P.head;
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (lane + 32 * u < A.D) s = fmaf(q[u], to_float<DT>(kp[at + lane + 32 * u]), s);
        s = warp_sum(s) * A.scale_log2;
        const float m_new = fmaxf(m_run, s), corr = exp2f(m_run - m_new), e = exp2f(s - m_new);
        m_run = m_new;
        l_run = fmaf(l_run, corr, e);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (lane + 32 * u < A.D) acc[u] = fmaf(acc[u], corr, e * to_float<DT>(vp[at + lane + 32 * u]));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (lane + 32 * u < A.D) o[lane + 32 * u] = from_float<DT>(acc[u] / l_run);
    if (lane == 0 && l_out) *l_out = 0.69314718056f * (m_run + log2f(l_run));
}

} // namespace sv

extern "C" {

size_t spec_tree_attention_workspace_bytes(int B, int N, int Hq, int heads, int head_dim) {
    if (B < 1 || B >= (1 << 16) || N < 1 || N > SPEC_MAX_TREE || heads < 1 || heads > 1024 || Hq < heads ||
        Hq % heads || Hq / heads > 64 || head_dim < 8 || head_dim % 8 || head_dim > SPEC_MAX_HEAD_DIM)
        return 0;
    return 256;
}

spec_status_t spec_tree_attention(const void *q, long long q_stride_b, long long q_stride_n,
                                  long long q_stride_h, const spec_pages_t *pages,
                                  const int32_t *page_table, const int32_t *cache_len,
                                  const int32_t *parent, const int32_t *node_count, int B, int N,
                                  int Hq, int max_pages, float scale, int window, int sinks,
                                  void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  uint32_t *dev_status, void *stream) {
    sv::AttnArgs A = {};
    const spec_status_t st = sv::make_pool(pages, A.P);
    if (st != SPEC_OK) return st;
    if (pages->dtype != SPEC_DTYPE_BF16 && pages->dtype != SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
    const size_t need = spec_tree_attention_workspace_bytes(B, N, Hq, pages->heads, pages->head_dim);
    if (!q || !page_table || !cache_len || !out || need == 0 || pages->layers != 1 || max_pages < 1 ||
        ((uintptr_t)q & 15) || ((uintptr_t)out & 15) || q_stride_b < 0 || q_stride_n < 0 || q_stride_h < 0 ||
        q_stride_b % 8 || q_stride_n % 8 || q_stride_h % 8 || window < 0 || sinks < 0 || !(scale > 0.f) ||
        !(scale < 3.0e38f))
        return SPEC_ERR_INVALID_ARG;
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need) return SPEC_ERR_WORKSPACE;
    A.P.page_st = pages->page_stride;
    A.P.token = pages->token_stride;
    A.P.head = pages->head_stride;
    A.q = static_cast<const uint16_t *>(q);
    A.qb = q_stride_b;
    A.qn = q_stride_n;
    A.qh = q_stride_h;
    A.table = page_table;
    A.len = cache_len;
    A.parent = parent;
    A.node_count = node_count;
    A.B = B;
    A.N = N;
    A.Hq = Hq;
    A.D = pages->head_dim;
    A.max_pages = max_pages;
    A.window = window;
    A.sinks = sinks;
    A.scale_log2 = scale * 1.44269504089f;
    A.out = static_cast<uint16_t *>(out);
    A.lse = lse;
    A.status = dev_status;
    return sv::launch_pdl(pages->dtype == SPEC_DTYPE_BF16 ? sv::sv_tree_attn<SPEC_DTYPE_BF16>
                                                          : sv::sv_tree_attn<SPEC_DTYPE_F16>,
                          dim3((unsigned)N * Hq, (unsigned)B), dim3(32), 0, static_cast<cudaStream_t>(stream), A);
}

} // extern "C"
