// sv_cache.cuh -- what the kernels of the paged cache share: the pool of pages
// as 16-byte vectors, status flags, and launches that overlap the end of the
// kernel before them.
#pragma once
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

__device__ __forceinline__ void flag(uint32_t *status, uint32_t bits) {
    if (status) atomicOr(status, bits);
}

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
