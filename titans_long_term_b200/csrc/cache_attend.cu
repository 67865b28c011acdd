// Attention of a chunk of new tokens over the paged cache.
//
// Row (b, h, t) stands at position p = starts[b] + t and takes the softmax of scale q.k over the keys that it
// sees, in one pass over them with a running maximum and sum. One warp has a row, d/32 columns a lane.
#include "cache.h"

namespace titans {
namespace {

// The keys that the row at position p sees: j < first_end, or j in [begin, p].
struct Seen {
    long first_end, begin;
};
__device__ __forceinline__ Seen seen_by(const AttendArgs& a, long p) {
    const long begin = a.window ? max(0L, p - a.window + 1) : 0L;
    return {min((long)a.sinks, begin), begin};
}

// 4 or 2 consecutive values of a row of the pool.
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

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) attend_rows_kernel(AttendArgs a) {
    constexpr int N = D / 32;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 31;
    const long row = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long)c.B * c.H * c.T) return;
    const long unit = row / c.T;
    const int t = (int)(row - unit * c.T), b = (int)(unit / c.H), h = (int)(unit % c.H), hk = h / (c.H / c.Hkv);
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row * D + lane * N;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + row * D + lane * N;
    float acc[N] = {}, m = -INFINITY, l = 0.f;
    if (t < cache_count(c, b)) {
        const long p = (long)c.starts[b] + t;
        const Seen s = seen_by(a, p);
        float qr[N];
#pragma unroll
        for (int i = 0; i < N; ++i) qr[i] = __bfloat162float(q[i]) * a.scale;
        for (long j = s.first_end > 0 ? 0 : s.begin; j <= p; ++j) {
            if (j == s.first_end && j < s.begin) j = s.begin;
            const long at = cache_row(c, b, hk, j);
            if (at < 0) {
                if (lane == 0) atomicOr(c.status, kStatusMissingPage);
                continue;
            }
            float x[N], z = 0.f;
            load_row<N, E4M3>(c.pk, c.k_scale, at, lane * N, D, x);
#pragma unroll
            for (int i = 0; i < N; ++i) z = fmaf(qr[i], x[i], z);
#pragma unroll
            for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
            const float top = fmaxf(m, z);
            if (top == -INFINITY && z == z) continue;
            const float keep = m == top ? 1.f : expf(m - top), w = expf(z - top);
            m = top;
            l = l * keep + w;
            load_row<N, E4M3>(c.pv, c.v_scale, at, lane * N, D, x);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(w, x[i], acc[i] * keep);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = __float2bfloat16(acc[i] * inv);
}

}  // namespace

cudaError_t launch_cache_attend(const AttendArgs& a, bool e4m3, cudaStream_t st) {
    const unsigned grid = (unsigned)(((long)a.c.B * a.c.H * a.c.T + 3) / 4);
    auto* kernel = a.c.d == 64 ? (e4m3 ? attend_rows_kernel<64, true> : attend_rows_kernel<64, false>)
                               : (e4m3 ? attend_rows_kernel<128, true> : attend_rows_kernel<128, false>);
    kernel<<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace titans
