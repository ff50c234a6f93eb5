// kv_cache.cuh -- the paged key-value cache as the kernels see it.
//
// Slot j of a sequence is row j % page_size of page page_table[j / page_size]; the
// address of a row is 64-bit arithmetic throughout (pools pass 4 GiB).
//
// What these kernels read may have been written by the kernel just before them, beside whose
// end they start (griddepcontrol.wait orders the two), so nothing is read through the
// non-coherent path.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "wq_device.cuh"

namespace wq {

// x / d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery, 1994, with
// the 33-bit multiplier split as 2^32 + mul).
struct FastDiv {
    uint32_t d, mul, shift;
    __device__ __forceinline__ uint32_t div(uint32_t x) const {
        return (__umulhi(x, mul) + x) >> shift;
    }
};

inline FastDiv make_fast_div(uint32_t d) {
    FastDiv f{d, 0u, 0u};
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
    return f;
}

struct KvView {
    char *k, *v;
    long long page_stride, head_stride, token_stride;  // in bytes
    FastDiv page_size;
    int n_pages, max_pages, n_heads, head_dim, dtype;
    const int32_t *page_table;  // [n_seq][max_pages]

    // Byte offset of head h's row of slot j in both pools, or -1 for a page out of range.
    __device__ __forceinline__ long long row(int s, int h, int j) const {
        const uint32_t p = page_size.div((uint32_t)j);
        const int page = page_table[(long long)s * max_pages + p];
        if ((unsigned)page >= (unsigned)n_pages) return -1;
        return (long long)page * page_stride + (long long)h * head_stride +
               (long long)(j - (int)(p * page_size.d)) * token_stride;
    }
};

// Element types of the cache.
template <int DT> struct KvType;
template <> struct KvType<kBF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float get(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ T put(float x) { return __float2bfloat16_rn(x); }
};
template <> struct KvType<kF16> {
    using T = __half;
    static __device__ __forceinline__ float get(T x) { return __half2float(x); }
    static __device__ __forceinline__ T put(float x) { return __float2half_rn(x); }
};
template <> struct KvType<kF32> {
    using T = float;
    static __device__ __forceinline__ float get(T x) { return x; }
    static __device__ __forceinline__ T put(float x) { return x; }
};

}  // namespace wq
