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

// acc[.] += A B over 16 of k for n-tiles 2 J0 .. 2 J1 - 1. The pieces of A are hi, lo (NA = 1: hi only) and those of B the NB tiles
// PIECE bytes apart: hi hi, lo hi and, where B has a second piece, hi lo. All tiles take one piece product before the next one, so that a
// tile's next product does not wait for its last. fragment(f, j, piece) loads the fragments of n-tiles 2 j, 2 j + 1.
template <int NA, int NB, int J0, int J1, int NT, typename Fragment>
__device__ __forceinline__ void mma_row(float (&acc)[NT][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                        Fragment fragment) {
    uint32_t f[J1 - J0][4];
#pragma unroll
    for (int j = J0; j < J1; ++j) fragment(f[j - J0], j, 0);
#pragma unroll
    for (int e = 0; e < NA; ++e)
#pragma unroll
        for (int j = J0; j < J1; ++j) {
            mma16816(acc[2 * j], e ? lo : hi, f[j - J0][0], f[j - J0][1]);
            mma16816(acc[2 * j + 1], e ? lo : hi, f[j - J0][2], f[j - J0][3]);
        }
    if constexpr (NB == 2) {
#pragma unroll
        for (int j = J0; j < J1; ++j) fragment(f[j - J0], j, 1);
#pragma unroll
        for (int j = J0; j < J1; ++j) {
            mma16816(acc[2 * j], hi, f[j - J0][0], f[j - J0][1]);
            mma16816(acc[2 * j + 1], hi, f[j - J0][2], f[j - J0][3]);
        }
    }
}
// The same for k-step KT of a lower triangular 64 x 64 tile of B, whose zero blocks are left out: LOWER: n-tiles from
// the k-step on, else up to it.
template <int KT, bool LOWER, int NA, int NB, typename Fragment>
__device__ __forceinline__ void mma_triangle(float (&acc)[8][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                             Fragment fragment) {
    mma_row<NA, NB, LOWER ? KT : 0, LOWER ? 4 : KT + 1>(acc, hi, lo, fragment);
}
// w[row][.] = decay w[row][.] + sum over the 64 tokens of t[row][token] B[token][.]; t's two rows are scaled by s0, s1 on the way
// and the products by i0, i1. B: NB pieces of a [64][D] tile at `tile`.
template <int D, int NB>
__device__ __forceinline__ void add_outer(float (&w)[D / 8][4], float decay, const float (&t)[8][4], float s0, float s1,
                                          float i0, float i1, uint32_t tile, int lane) {
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) split_a<8>(t, kt, s0, s1, hi[kt], lo[kt]);
#pragma unroll
    for (int half = 0; half < D / 64; ++half) {
        float acc[8][4] = {};
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
            mma_row<2, NB, 0, 4>(acc, hi[kt], lo[kt], [&](uint32_t(&f)[4], int j, int e) {
                frag_bt<D>(f, tile + e * kC * D * 2, half * 64 + j * 16, kt * 16, lane);
            });
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float(&u)[4] = w[half * 8 + j];
            u[0] = fmaf(u[0], decay, acc[j][0] * i0), u[1] = fmaf(u[1], decay, acc[j][1] * i0);
            u[2] = fmaf(u[2], decay, acc[j][2] * i1), u[3] = fmaf(u[3], decay, acc[j][3] * i1);
        }
    }
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

// What thread p of the producers brings of a chunk: K, the CTA's columns of V (or dY) and, WITH_Q, Q and P too. The tokens are
// fetched into registers while the chunks before are still in work: one round trip to memory a chunk, which nothing waits for.
template <int D, int RW, typename Tok, int PP, bool WITH_Q>
struct Producer {
    static constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, VEC = kC * D / 8 / kProducers, VV = kC * RW / 8 / kProducers;
    Block8<Tok> k[VEC], q[WITH_Q ? VEC : 1], v[VV];

    // Tokens t0 .. t0 + n - 1 (n <= 64, the rest zeros); kp, qp: rows of the key head, vp: the CTA's columns.
    __device__ __forceinline__ void fetch(const Tok* kp, const Tok* qp, const Tok* vp, long t0, int n, int p) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int block = i * kProducers + p;
            if (block / (D / 8) < n) {
                k[i].load(kp + t0 * D + (long)block * 8);
                if constexpr (WITH_Q) q[i].load(qp + t0 * D + (long)block * 8);
            } else {
                k[i].clear();
                if constexpr (WITH_Q) q[i].clear();
            }
        }
#pragma unroll
        for (int i = 0; i < VV; ++i) {
            const int block = i * kProducers + p, row = block / (RW / 8), col = block % (RW / 8) * 8;
            if (row < n)
                v[i].load(vp + (t0 + row) * D + col);
            else
                v[i].clear();
        }
    }
    // The fetched tokens and record r into stage s.
    __device__ __forceinline__ void store(Stage<D, RW, NP, PP>& s, const DeltaChunk& r, int p) {
        for (int i = p; i < (int)sizeof(r.N) / 16; i += kProducers)
            if (in_lower_blocks(i)) cp_async16(smem_u32(s.n) + i * 16, reinterpret_cast<const uint4*>(r.N) + i);
        if constexpr (WITH_Q)
            for (int i = p; i < PP * kC * kC / 8; i += kProducers)
                if (in_lower_blocks(i)) cp_async16(smem_u32(s.p) + i * 16, reinterpret_cast<const uint4*>(r.P) + i);
        for (int i = p; i < 3 * kC / 4; i += kProducers)
            cp_async16(smem_u32(s.gamma) + i * 16, reinterpret_cast<const uint4*>(r.gamma) + i);
        if (p < 6) s.scal[p] = (&r.k_scale)[p];
        const float ks = r.k_scale, qs = r.q_scale;
        float x[8];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int block = i * kProducers + p;
            const uint32_t at = swz<D>(block / (D / 8), block % (D / 8));
            k[i].get(x);
            put8<NP>(smem_u32(s.k) + at, kC * D * 2, x, ks);
            if constexpr (WITH_Q) {
                q[i].get(x);
                put8<NP>(smem_u32(s.q) + at, kC * D * 2, x, qs);
            }
        }
#pragma unroll
        for (int i = 0; i < VV; ++i) {
            const int block = i * kProducers + p, row = block / (RW / 8), col = block % (RW / 8) * 8;
            v[i].get(x);
            store8(s.v + row * (RW + 4) + col, x);
        }
        cp_async_wait_all();
    }
};

}  // namespace titans
