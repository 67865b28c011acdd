// Shared by the attention kernels of the paged cache: which keys a row sees, and a row taken key by key.
#pragma once
#include "cache.h"

namespace titans {

// Positions that the page table has room for, below 2^31.
__device__ __forceinline__ int capacity(const CacheArgs& c) { return c.max_pages << c.page_shift; }

// The keys that the row at position p sees, as far as the table has room for them: j < sink_end, or begin <= j < end.
struct Seen {
    int begin, end, sink_end;
    __device__ bool operator()(int key) const { return key < end && (key >= begin || key < sink_end); }
};
__device__ __forceinline__ Seen seen_by(const AttendArgs& a, long p) {
    const long cap = capacity(a.c), begin = a.window ? max(0L, p - a.window + 1) : 0L;
    return {(int)min(begin, cap), (int)max(0L, min(p + 1, cap)), (int)min((long)min(a.sinks, capacity(a.c)), begin)};
}
// The keys that some row at positions p0..p1 sees: the widest of all bounds.
__device__ __forceinline__ Seen seen_by_any(const AttendArgs& a, long p0, long p1) {
    const Seen lo = seen_by(a, max(p0, 0L)), hi = seen_by(a, p1);
    return {lo.begin, hi.end, hi.sink_end};
}

// The tiles of KEYS keys that those keys lie in: 0..head-1 and from tail on, `count` together.
struct Tiles {
    int head, tail, count;
    __device__ int operator[](int i) const { return i < head ? i : tail + i - head; }
};
template <int KEYS>
__device__ __forceinline__ Tiles tiles_of(const Seen& s) {
    const int end = (s.end + KEYS - 1) / KEYS, tail = min(s.begin / KEYS, end);
    const int head = min(tail, (min(s.sink_end, s.end) + KEYS - 1) / KEYS);
    return {head, tail, head + end - tail};
}

// N consecutive values of a row of the pool.
template <int N, bool E4M3>
__device__ __forceinline__ void load_row(const void* pool, const float* scales, long row, int col, int D, float (&x)[N]) {
    if constexpr (E4M3) {
        const float s = scales[row];
        const uint8_t* p = static_cast<const uint8_t*>(pool) + row * D + col;
        uint32_t u;  // two or four of them
        if constexpr (N == 4)
            u = *reinterpret_cast<const uint32_t*>(p);
        else
            u = *reinterpret_cast<const uint16_t*>(p);
        const float2 f = e4m3_to_float2<false>(u);
        x[0] = f.x * s, x[1] = f.y * s;
        if constexpr (N == 4) {
            const float2 g = e4m3_to_float2<true>(u);
            x[2] = g.x * s, x[3] = g.y * s;
        }
    } else {
        const __nv_bfloat162* p =
            reinterpret_cast<const __nv_bfloat162*>(static_cast<const __nv_bfloat16*>(pool) + row * D + col);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = __bfloat1622float2(p[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// One row by one warp, key by key, over tiles first..last-1: m (log2 units), l and D / 32 columns a lane.
template <int D, bool E4M3, int KEYS>
__device__ __noinline__ void attend_row(const AttendArgs& a, int b, int hk, const __nv_bfloat16* q, long p, Tiles tiles,
                                        int first, int last, float& m, float& l, float (&acc)[D / 32]) {
    constexpr int N = D / 32;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 31;
    const Seen s = seen_by(a, p);
    float qr[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        qr[i] = __bfloat162float(q[lane * N + i]) * (a.scale * 1.44269504f);
        acc[i] = 0.f;
    }
    m = -INFINITY, l = 0.f;
    for (int i = first; i < last; ++i) {
        const int j0 = tiles[i] * KEYS;
        for (int j = j0; j < min(j0 + KEYS, s.end); ++j) {
            if (!s(j)) continue;
            const long at = cache_row(c, b, hk, j);
            if (at < 0) continue;
            float x[N], z = 0.f;
            load_row<N, E4M3>(c.pk, c.k_scale, at, lane * N, D, x);
#pragma unroll
            for (int i = 0; i < N; ++i) z = fmaf(qr[i], x[i], z);
#pragma unroll
            for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
            const float top = fmaxf(m, z);
            if (top == -INFINITY && z == z) continue;
            const float keep = m == top ? 1.f : exp2f(m - top), w = exp2f(z - top);
            m = top;
            l = l * keep + w;
            load_row<N, E4M3>(c.pv, c.v_scale, at, lane * N, D, x);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(w, x[i], acc[i] * keep);
        }
    }
}

}  // namespace titans
