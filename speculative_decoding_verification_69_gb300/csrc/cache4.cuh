// cache4.cuh -- the format of the 4-bit cache (spec_cache.h) on the device.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sv_cache.cuh"

namespace sv {

// A 4-bit pool.  Strides in bytes.
struct Pool4 {
    uint8_t *data;
    long long layer, page_st, head;
    int layers, num_pages, page, page_shift, heads, D;
    int C;        // channels kept: D rounded up to 32
    int block;    // tokens of a block
    int bytes;    // of a block
    int groups;   // of 32 channels
};

spec_status_t make_pool4(const spec_pages4_t *p, Pool4 &P);

// Byte offsets inside a page and head.
__device__ __forceinline__ int block4(const Pool4 &P, int tok) { return tok / P.block * P.bytes; }
__device__ __forceinline__ int key4(const Pool4 &P, int tok, int group) {  // 16 bytes
    const int t = tok & (P.block - 1);
    return block4(P, tok) + (((t >> 3) * P.groups + group) * 8 + (t & 7)) * 16;
}
__device__ __forceinline__ int value4(const Pool4 &P, int tok, int d) {  // 4 bytes: 8 tokens
    const int t = tok & (P.block - 1);
    return block4(P, tok) + P.block * (P.C >> 1) + ((t >> 3) * P.C + d) * 4;
}
__device__ __forceinline__ int scale4(const Pool4 &P, int tok, int group, bool values) {
    const int t = tok & (P.block - 1);
    return block4(P, tok) + P.block * (P.C + (values ? P.groups : 0) + group) + t;
}

// The bit of code i in its word.
__device__ __forceinline__ int bit4(int i) { return 4 * (i >> 1) + 16 * (i & 1); }

// (1 + m/8) 2^(e-19) of the byte 8 e + m: its bits are a float's exponent and upper mantissa.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float((byte + ((127u - 19u) << 3)) << 20);
}
// x / d for inv near 1 / d: one residual correction of the quotient (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  Where x / d has few bits it is exact.
__device__ __forceinline__ float quotient(float x, float d, float inv) {
    const float y = x * inv;
    return fmaf(fmaf(-d, y, x), inv, y);
}
// The byte of the scale nearest to amax / 7 (ties to even), of the smallest or largest one beyond
// the ends.  The true quotient of a number of 11 bits is no nearer to the middle between
// two scales than 2^-13 of it, unless it is one, and then it has few bits.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t b = __float_as_uint(amax < INFINITY ? quotient(amax, 7.f, 1.f / 7.f) : amax);
    const int r = (int)((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - ((127 - 19) << 3);
    return (uint32_t)max(0, min(r, 255));
}
// The code of x, which is finite, |x| / s within 7.5: the low four bits of the sum.  inv: 1 / s to 2^-22.
// Ties are exact (see quotient); all other quotients of a number of 11 bits and one of 4 are 2^-12 or
// more from a tie.  Adding 1.5 * 2^23 (+ 8) rounds to a whole number, ties to even.
__device__ __forceinline__ uint32_t code_sum(float x, float s, float inv) {
    return __float_as_uint(quotient(x, s, inv) + (12582912.f + 8.f));
}
__device__ __forceinline__ float near_reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The same for any x: NaN gives 0, and what is out of range the end of it.
__device__ __forceinline__ uint32_t code_of(float x, float s) {
    return (uint32_t)(max(-8, min(__float2int_rn(__fdiv_rn(x, s)), 7)) + 8);  // (NaN converts to 0)
}

template <int DT> __device__ __forceinline__ float2 unpack16(uint32_t x) {
    if (DT == SPEC_DTYPE_BF16) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}
template <int DT> __device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (DT == SPEC_DTYPE_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&x);
    }
    const __half2 x = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}

} // namespace sv
