// Shared by the gated delta rule's chunked kernels.
//
// A chunk has C = 64 tokens with cumulative log decays G, gamma = exp(G), D_ij = exp(G_i - G_j) (j <= i):
//   M   = strictly lower part of D o K K^T      (how write j shows in the residual of token i)
//   N   solves (I + M beta) N = M               (strictly lower, so X - N beta X inverts I + M beta)
//   P   = lower part of D o Q K^T
//   X   = V - gamma K W0^T,  eps = X - N (beta X),  E = beta eps     (the chunk's writes)
//   Y   = gamma Q W0^T + P E,  W = gamma_C W0 + (l E)^T K,  l_j = exp(G_C - G_j)
//
// Matrix products run on the tensor cores (mma.sync m16n8k16, fp16 operands, fp32 sums) with operands
// split into fp16 pieces, x = s (hi + lo), where s is a power of two that puts the largest |x| of the row or
// tile at 2^14..2^15. hi + lo hold 22 bits of every value down to 2^-16 of the largest one, and below
// that an absolute error of 2^-39 of it; a bf16 value is one piece exactly down to 2^-28 of the largest.
// Three products (hi hi, hi lo, lo hi) therefore stand for an fp32 one, two where one side is exact: bf16
// pieces would need six and three for the same 22 bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "delta.h"
#include "ptx.cuh"

namespace titans {

constexpr int kC = 64;  // tokens of a chunk

// What the first kernel leaves of a chunk for the others, in the workspace.
struct DeltaChunk {
    __half N[2][kC * kC];  // pieces hi, lo; rows of 128 bytes, swizzled as swz<64>(), only in_lower_blocks()
    __half P[2][kC * kC];
    float gamma[kC], rest[kC], beta[kC];  // exp(G_i), exp(G_C - G_i), beta_i
    float k_scale, q_scale;               // powers of two that the tiles of K and Q are multiplied by
    float k_inv, q_inv, n_inv, p_inv;     // 1 / the scales
    float ghi[kC], glo[kC];               // G_i as two floats
    int zeros[kC];                        // decays of 0 (g < -104) up to token i, which G leaves out
    float from[kC], to[3][48];            // decays from the end of the block of 16 before token i's to i, and from token
                                          // j to the end of blocks 0, 1 and 2: their product is D_ij between blocks
    float pad[170];
};
static_assert(sizeof(DeltaChunk) % 1024 == 0, "chunks stay 1 KiB aligned");

// Whether 16-byte block i of the pieces of such a tile lies on or below the diagonal in blocks of 16 x 16. The others are neither
// written nor read.
__device__ __forceinline__ bool in_lower_blocks(int i) {
    const int row = (i >> 3) & (kC - 1), block = (i & 7) ^ (row & 7);
    return block >> 1 <= row >> 4;
}

// exp(G_i - G_j) for j <= i, 0 where a decay of 0 lies between.
__device__ __forceinline__ float decay_between(const float* ghi, const float* glo, const int* zeros, int i, int j) {
    return zeros[i] == zeros[j] ? expf((ghi[i] - ghi[j]) + (glo[i] - glo[j])) : 0.f;
}

// Power of two that brings `top` to [2^14, 2^15), and its inverse. At most 2^114, for tops below 2^-100.
__device__ __forceinline__ float pow2_scale(float top, float& inv) {
    const int e = max(__float_as_int(top) >> 23, 27) - 127;  // top >= 0: no sign bit
    inv = __int_as_float((e - 14 + 127) << 23);
    return __int_as_float((14 - e + 127) << 23);
}

// A row of a [rows][D] fp16 tile has D / 8 blocks of 16 bytes; block c of row r lies at c ^ (r & 7), so that the
// eight rows of an 8x8 matrix fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int block) {
    return (uint32_t)(row * D * 2 + ((block ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragments of a [rows][D] tile at `base` for two n-tiles (16 of n) and 16 of k, as b0, b1 of the first and
// b0, b1 of the second: n along the tile's rows (k contiguous) ...
template <int D>
__device__ __forceinline__ void frag_b(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
    const int m = lane >> 3;
    ldsm4(r, base + swz<D>(n0 + (lane & 7) + (m >> 1) * 8, (k0 >> 3) + (m & 1)));
}
// ... or k along the tile's rows (n contiguous).
template <int D>
__device__ __forceinline__ void frag_bt(uint32_t (&r)[4], uint32_t base, int n0, int k0, int lane) {
    const int m = lane >> 3;
    ldsm4t(r, base + swz<D>(k0 + (lane & 7) + (m & 1) * 8, (n0 >> 3) + (m >> 1)));
}
// The 16 x 16 fragment of A: m along the tile's rows ...
template <int D>
__device__ __forceinline__ void frag_a(uint32_t (&r)[4], uint32_t base, int m0, int k0, int lane) {
    const int m = lane >> 3;
    ldsm4(r, base + swz<D>(m0 + (lane & 7) + (m & 1) * 8, (k0 >> 3) + (m >> 1)));
}
// ... or k along them.
template <int D>
__device__ __forceinline__ void frag_at(uint32_t (&r)[4], uint32_t base, int m0, int k0, int lane) {
    const int m = lane >> 3;
    ldsm4t(r, base + swz<D>(k0 + (lane & 7) + (m >> 1) * 8, (m0 >> 3) + (m & 1)));
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// hi and lo of two scaled values.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = half2_bits(h);
    lo = half2_bits(__floats2half2_rn(x - f.x, y - f.y));
}
__device__ __forceinline__ uint32_t pack_half2(float x, float y) { return half2_bits(__floats2half2_rn(x, y)); }

// An accumulator of 16 rows: t[n-tile][0, 1] belong to row lane / 4, [2, 3] to row lane / 4 + 8, columns
// 8 n-tile + 2 (lane % 4) + 0, 1. Two neighbouring n-tiles, packed, are an A fragment of 16 of k.

// The largest |x| of both rows, in each of their four lanes.
template <int NT>
__device__ __forceinline__ void row_tops(const float (&t)[NT][4], float& top0, float& top1) {
    top0 = top1 = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        top0 = fmaxf(top0, fmaxf(fabsf(t[i][0]), fabsf(t[i][1])));
        top1 = fmaxf(top1, fmaxf(fabsf(t[i][2]), fabsf(t[i][3])));
    }
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
        top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, s));
        top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, s));
    }
}
// Pieces of n-tiles 2 kt and 2 kt + 1 as A fragments, the rows multiplied by s0 and s1.
template <int NT>
__device__ __forceinline__ void split_a(const float (&t)[NT][4], int kt, float s0, float s1, uint32_t (&hi)[4],
                                        uint32_t (&lo)[4]) {
    split2(t[2 * kt][0] * s0, t[2 * kt][1] * s0, hi[0], lo[0]);
    split2(t[2 * kt][2] * s1, t[2 * kt][3] * s1, hi[1], lo[1]);
    split2(t[2 * kt + 1][0] * s0, t[2 * kt + 1][1] * s0, hi[2], lo[2]);
    split2(t[2 * kt + 1][2] * s1, t[2 * kt + 1][3] * s1, hi[3], lo[3]);
}

// Eight consecutive token values as floats.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// Eight token values as they lie in memory.
template <typename Tok>
struct Block8;
template <>
struct Block8<__nv_bfloat16> {
    uint4 u;
    __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ void clear() { u = make_uint4(0, 0, 0, 0); }
    __device__ void get(float (&x)[8]) const { unpack8(u, x); }
};
template <>
struct Block8<float> {
    float v[8];
    __device__ void load(const float* p) { load8(p, v); }
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[i];
    }
};

// Eight values, scaled, into one 16-byte block of the tile's hi piece (and of its lo piece, LO bytes further).
template <int PIECES>
__device__ __forceinline__ void put8(uint32_t addr, uint32_t lo_offset, const float (&x)[8], float s) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(x[2 * i] * s, x[2 * i + 1] * s, h[i], l[i]);
    st_shared_v4(addr, h[0], h[1], h[2], h[3]);
    if constexpr (PIECES == 2) st_shared_v4(addr + lo_offset, l[0], l[1], l[2], l[3]);
}

// acc += A B for one n-tile, over the pieces: hi hi, lo hi, hi lo where there are such.
template <int NA, int NB>
__device__ __forceinline__ void mma_all(float (&acc)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][2]) {
    mma16816(acc, a[0], b[0][0], b[0][1]);
    if constexpr (NA == 2) mma16816(acc, a[1], b[0][0], b[0][1]);
    if constexpr (NB == 2) mma16816(acc, a[0], b[1][0], b[1][1]);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int s = 16; s; s >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s));
    return x;
}
__device__ __forceinline__ double warp_prefix(double x, int lane) {
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, s);
        if (lane >= s) x += y;
    }
    return x;
}

// f(integral constant) for 0 .. N - 1.
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
    if constexpr (N > 0) {
        unrolled<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ long delta_length(const DeltaArgs& a, long b) {
    return a.lengths ? min((long)max(a.lengths[b], 0), a.T) : a.T;
}
__device__ __forceinline__ long delta_key_head(const DeltaArgs& a, long unit) {
    return unit / a.H * a.Hk + (unit % a.H) / (a.H / a.Hk);
}

}  // namespace titans
