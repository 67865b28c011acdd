// Gated delta rule, token by token: A = exp(g) W, e = beta (v - A k), W = A + e k^T, y = W q.
//
// The rows of W are independent of one another (row i sees v_i, and k, q, g, beta as a whole), so a
// warp takes eight rows into registers and walks the tokens; nothing is shared between warps. Both
// products a token needs are taken from the state before the write,
//   y_i = exp(g) (W q)_i + e_i (k . q),
// so one pass over the row gives the two dot products and a second one updates it.
//
// Eight lanes hold a row, 4 consecutive floats of every 32: a warp reads and writes the state in
// 128-byte runs, and a dot product needs three shuffles. For one token (titans_delta_step) the state
// is read once and written once, which is what the call cannot do without; it is bound by that: 1024 units of d = 128
// (134 MB) take 24.4 us, 5.5 TB/s, 0.84 of a copy's rate. 16 units of d = 64 take 4.3 us, a launch and one round trip.
#include <cuda_bf16.h>

#include "delta.h"

namespace titans {
namespace {

constexpr int kRows = 2;               // rows of a lane
constexpr int kWarpRows = 4 * kRows;   // four row groups of eight lanes

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

// Sum over the eight lanes of a row, in every one of them.
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x;
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}

template <int D, typename Tok>
__global__ void __launch_bounds__(64) delta_tokens_kernel(DeltaArgs a) {
    constexpr int N4 = D / 32;  // float4 of a lane and row
    const int lane = threadIdx.x & 31;
    const long warp = (long)blockIdx.x * 2 + (threadIdx.x >> 5);
    const long unit = warp / (D / kWarpRows);
    const int row0 = (int)(warp % (D / kWarpRows)) * kWarpRows + (lane >> 3) * kRows;
    const int col = (lane & 7) * 4;
    const long b = unit / a.H, key_head = b * a.Hk + (unit % a.H) / (a.H / a.Hk);
    const long len = a.lengths ? min((long)max(a.lengths[b], 0), a.T) : a.T;
    const Tok* k = static_cast<const Tok*>(a.k) + key_head * a.T * D + col;
    const Tok* q = static_cast<const Tok*>(a.q) + key_head * a.T * D + col;
    const Tok* v = static_cast<const Tok*>(a.v) + unit * a.T * D + row0;
    const Tok* attn = a.attn ? static_cast<const Tok*>(a.attn) + unit * a.T * D + row0 : nullptr;
    Tok* y = static_cast<Tok*>(a.y) + unit * a.T * D + row0;
    const float* g = a.g + unit * a.T;
    const float* beta = a.beta + unit * a.T;
    float* W = a.W + unit * D * D + (long)row0 * D + col;

    float4 w[kRows][N4];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < N4; ++i) w[r][i] = load4(W + r * D + 32 * i);

    for (long t = 0; t < len; ++t, k += D, q += D, v += D, y += D) {
        float4 kt[N4], qt[N4];
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            kt[i] = load4(k + 32 * i);
            qt[i] = load4(q + 32 * i);
        }
        const float decay = expf(g[t]), bt = beta[t];
        float vt[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) vt[r] = to_float(v[r]);
        float kq = 0.f, kw[kRows] = {}, qw[kRows] = {};
#pragma unroll
        for (int i = 0; i < N4; ++i) {
            kq = dot4(kt[i], qt[i], kq);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                // decay first: an infinite g (decay 0) leaves nothing of W, whatever it held in finite numbers
                w[r][i].x *= decay, w[r][i].y *= decay, w[r][i].z *= decay, w[r][i].w *= decay;
                kw[r] = dot4(w[r][i], kt[i], kw[r]);
                qw[r] = dot4(w[r][i], qt[i], qw[r]);
            }
        }
        kq = row_sum(kq);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float e = bt * (vt[r] - row_sum(kw[r]));
            float o = fmaf(e, kq, row_sum(qw[r]));
#pragma unroll
            for (int i = 0; i < N4; ++i) {
                w[r][i].x = fmaf(e, kt[i].x, w[r][i].x);
                w[r][i].y = fmaf(e, kt[i].y, w[r][i].y);
                w[r][i].z = fmaf(e, kt[i].z, w[r][i].z);
                w[r][i].w = fmaf(e, kt[i].w, w[r][i].w);
            }
            if ((lane & 7) == 0) {
                if (attn) o = to_float(attn[t * D + r]) / (1.f + expf(-o));
                store(y + r, o);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int i = 0; i < N4; ++i) *reinterpret_cast<float4*>(W + r * D + 32 * i) = w[r][i];
    for (long t = len; t < a.T; ++t, y += D)
        if ((lane & 7) == 0)
            for (int r = 0; r < kRows; ++r) store(y + r, 0.f);
}

template <int D>
cudaError_t launch(const DeltaArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((long)a.B * a.H * (D / kWarpRows) / 2);
    if (a.bf16)
        delta_tokens_kernel<D, __nv_bfloat16><<<grid, 64, 0, st>>>(a);
    else
        delta_tokens_kernel<D, float><<<grid, 64, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_tokens(const DeltaArgs& a, cudaStream_t st) {
    return a.d == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace titans
