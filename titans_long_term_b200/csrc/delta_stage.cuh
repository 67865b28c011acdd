// Stages of the two serial kernels of the chunked gated delta rule and the warps that fill them.
#pragma once
#include "delta_common.cuh"

namespace titans {

constexpr int kProducers = 128;

// One chunk in shared memory: pieces of K, Q, N, P (P of them PP), values or their adjoints as floats.
template <int D, int RW, int NP, int PP>
struct Stage {
    static constexpr int kVLd = RW + 4;  // floats between V's rows: lanes of a fragment hit 32 banks
    __half k[NP][kC * D], q[NP][kC * D];
    __half n[2][kC * kC], p[PP][kC * kC];
    float v[kC * kVLd];
    float gamma[kC], rest[kC], beta[kC];
    float scal[8];  // k_scale, q_scale, k_inv, q_inv, n_inv, p_inv
    float pad[56];
};

// acc[.] += A B over 16 of k for two n-tiles; the pieces of A are hi, lo and those of B b[0], b[1]: hi hi, lo hi and,
// where B has a second piece, hi lo.
template <int NB>
__device__ __forceinline__ void mma_pieces(float (&acc0)[4], float (&acc1)[4], const uint32_t (&hi)[4],
                                           const uint32_t (&lo)[4], const uint32_t (&b)[NB][4]) {
    mma16816(acc0, hi, b[0][0], b[0][1]);
    mma16816(acc1, hi, b[0][2], b[0][3]);
    mma16816(acc0, lo, b[0][0], b[0][1]);
    mma16816(acc1, lo, b[0][2], b[0][3]);
    if constexpr (NB == 2) {
        mma16816(acc0, hi, b[1][0], b[1][1]);
        mma16816(acc1, hi, b[1][2], b[1][3]);
    }
}

// Thread p of the producers brings chunk r, whose tokens start at t0 and of which n count, into stage s. k, q: rows of the
// key head; v: the CTA's columns of V or dY. WITH_Q: Q and P too.
template <int D, int RW, typename Tok, int PP, bool WITH_Q>
__device__ __forceinline__ void fill_stage(Stage<D, RW, sizeof(Tok) == 4 ? 2 : 1, PP>& s, const DeltaChunk& r,
                                           const Tok* k, const Tok* q, const Tok* v, long t0, int n, int p) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, VEC = kC * D / 8 / kProducers, VV = kC * RW / 8 / kProducers;
    constexpr int BATCH = sizeof(Tok) == 4 ? 2 : 4;  // blocks of eight values in flight
    float x[BATCH][8];
    const float ks = r.k_scale, qs = r.q_scale;
    for (int i = p; i < (int)sizeof(r.N) / 16; i += kProducers)
        cp_async16(smem_u32(s.n) + i * 16, reinterpret_cast<const uint4*>(r.N) + i);
    if constexpr (WITH_Q)
        for (int i = p; i < PP * kC * kC / 8; i += kProducers)
            cp_async16(smem_u32(s.p) + i * 16, reinterpret_cast<const uint4*>(r.P) + i);
    for (int i = p; i < 3 * kC / 4; i += kProducers)
        cp_async16(smem_u32(s.gamma) + i * 16, reinterpret_cast<const uint4*>(r.gamma) + i);
    if (p < 6) s.scal[p] = (&r.k_scale)[p];
#pragma unroll
    for (int w = 0; w < (WITH_Q ? 2 : 1); ++w) {
        const Tok* src = (w ? q : k) + t0 * D;
        const uint32_t base = smem_u32(w ? s.q : s.k);
#pragma unroll
        for (int i0 = 0; i0 < VEC; i0 += BATCH) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int block = (i0 + i) * kProducers + p;
                if (block / (D / 8) < n) {
                    load8(src + (long)block * 8, x[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int block = (i0 + i) * kProducers + p;
                put8<NP>(base + swz<D>(block / (D / 8), block % (D / 8)), kC * D * 2, x[i], w ? qs : ks);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VV; ++i) {
        const int block = i * kProducers + p, row = block / (RW / 8), col = block % (RW / 8) * 8;
        if (row < n) {
            load8(v + (t0 + row) * D + col, x[0]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[0][j] = 0.f;
        }
        store8(s.v + row * (RW + 4) + col, x[0]);
    }
    cp_async_wait_all();
}

}  // namespace titans
