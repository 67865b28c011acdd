// Shared by the paged cache's kernels: where a token lies, and the attention of one row.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace titans {

constexpr unsigned kStatusMissingPage = 16u;

struct CacheArgs {
    int d, B, H, Hkv;
    int page_shift;  // log2 of the page's tokens
    int num_pages, max_pages;
    long T;
    void *pk, *pv;             // [num_pages, Hkv, page, d] bf16 or e4m3
    float *k_scale, *v_scale;  // [num_pages, Hkv, page], e4m3 only
    const int *table, *starts, *counts;
    unsigned* status;
};

// Valid tokens of sequence b in a call.
__device__ __forceinline__ int cache_count(const CacheArgs& a, int b) {
    return a.counts ? (int)min((long)max(a.counts[b], 0), a.T) : (int)a.T;
}

// Row of the pool ([num_pages * Hkv * page] rows of d values) that holds position `pos` of sequence b for
// key/value head h; -1 where the page is missing.
__device__ __forceinline__ long cache_row(const CacheArgs& a, int b, int h, long pos) {
    const long index = pos >> a.page_shift;
    if (pos < 0 || index >= a.max_pages) return -1;
    const int page = a.table[(long)b * a.max_pages + index];
    if ((unsigned)page >= (unsigned)a.num_pages) return -1;
    return (((long)page * a.Hkv + h) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

// The lower (UPPER: upper) two of four e4m3 values as fp16, exactly.
template <bool UPPER>
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t four) {
    uint32_t y;
    if constexpr (UPPER)
        asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(y) : "r"(four));
    else
        asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(y) : "r"(four));
    return y;
}
template <bool UPPER>
__device__ __forceinline__ float2 e4m3_to_float2(uint32_t four) {
    const uint32_t h = e4m3_to_half2<UPPER>(four);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace titans
