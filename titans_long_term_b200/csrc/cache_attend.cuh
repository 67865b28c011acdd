// Shared by the attention kernels of the paged cache: which keys a row sees, and a row taken key by key.
#pragma once
#include "cache.h"

namespace titans {

// The keys that the row at position p sees: j < sink_end, or begin <= j <= p.
struct Seen {
    long begin, sink_end;
};
__device__ __forceinline__ Seen seen_by(const AttendArgs& a, long p) {
    const long begin = a.window ? max(0L, p - a.window + 1) : 0L;
    return {begin, min((long)a.sinks, begin)};
}

// The tiles of KEYS keys that rows at positions p0..p1 see: 0..head-1 and tail..end-1.
struct Tiles {
    int head, tail, count;
    __device__ int operator[](int i) const { return i < head ? i : tail + i - head; }
};
template <int KEYS>
__device__ __forceinline__ Tiles tiles_of(const AttendArgs& a, long p0, long p1) {
    Tiles t{0, 0, 0};
    if (p1 < 0) return t;
    const long end = p1 / KEYS + 1;
    t.tail = (int)(seen_by(a, max(p0, 0L)).begin / KEYS);
    // the last row has the widest view of the sinks: those before its own window
    t.head = (int)min((long)t.tail, (seen_by(a, p1).sink_end + KEYS - 1) / KEYS);
    t.count = t.head + (int)end - t.tail;
    return t;
}

// N consecutive values of a row of the pool.
template <int N, bool E4M3>
__device__ __forceinline__ void load_row(const void* pool, const float* scales, long row, int col, int D, float (&x)[N]) {
    if constexpr (E4M3) {
        const float s = scales[row];
        const uint16_t* p = reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(pool) + row * D + col);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = e4m3x2_to_float2(p[i]);
            x[2 * i] = f.x * s;
            x[2 * i + 1] = f.y * s;
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
        const long j0 = (long)tiles[i] * KEYS;
        for (long j = j0; j < j0 + KEYS && j <= p; ++j) {
            if (j >= s.sink_end && j < s.begin) continue;
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
