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

// Two warps share sixteen rows of a state: each has half of its columns in registers and, within a chunk, half of the
// tokens. What they tell one another goes through shared memory in the layout of the registers, a lane to the same lane of
// the other warp.
template <int D, int NP>
struct Exchange {
    float4 part[2][4][32];  // partial sums over the writer's columns, for the reader's tokens; [1], once read, takes
                            // fragments of one half of the tokens that the other one needs
    uint4 outer[2][4][32];  // fragments of the outer product's left side: 2 k-steps x (hi, lo) of each half of the tokens
    uint4 w[NP][D / 16][32], e[NP][4][32];  // for the output warp: the state's and the writes' fragments
    float2 inv[32], outer_inv[2][32], w_inv[2][32], e_inv[2][32];  // inverse scales of a lane's two rows
};
__device__ __forceinline__ uint4 as_uint4(const uint32_t (&x)[4]) { return make_uint4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void from_uint4(uint32_t (&x)[4], uint4 u) { x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w; }

// w[row][.] = decay w[row][.] + sum over 32 tokens of t[row][token] B[token][.] for the columns col0 .. of a half: the two k-steps'
// fragments hi, lo, tokens from tok0 on; the products times f0, f1. B: NB pieces of a [64][D] tile at `tile`.
template <int D, int NB>
__device__ __forceinline__ void add_outer(float (&w)[D / 16][4], float decay, const uint32_t (&hi)[2][4],
                                          const uint32_t (&lo)[2][4], float f0, float f1, uint32_t tile, int col0,
                                          int tok0, int lane) {
    float acc[D / 16][4] = {};
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
        mma_row<2, NB, 0, D / 32>(acc, hi[kt], lo[kt], [&](uint32_t(&f)[4], int j, int e) {
            frag_bt<D>(f, tile + e * kC * D * 2, col0 + j * 16, tok0 + kt * 16, lane);
        });
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        w[j][0] = fmaf(w[j][0], decay, acc[j][0] * f0), w[j][1] = fmaf(w[j][1], decay, acc[j][1] * f0);
        w[j][2] = fmaf(w[j][2], decay, acc[j][2] * f1), w[j][3] = fmaf(w[j][3], decay, acc[j][3] * f1);
    }
}
// Splits t (the own tokens, 2 k-steps) into fragments hi, lo, which, where it is `needed`, also go to the other warp; inv: their
// rows' inverse scales.
__device__ __forceinline__ void share(const float (&t)[4][4], uint32_t (&hi)[2][4], uint32_t (&lo)[2][4], float2& inv,
                                      uint4 (&to)[4][32], float2 (&to_inv)[32], int lane, bool needed = true) {
    float top0, top1;
    row_tops<4>(t, top0, top1);
    const float s0 = pow2_scale(top0, inv.x), s1 = pow2_scale(top1, inv.y);
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
        split_a<4>(t, kt, s0, s1, hi[kt], lo[kt]);
        if (needed) to[2 * kt][lane] = as_uint4(hi[kt]), to[2 * kt + 1][lane] = as_uint4(lo[kt]);
    }
    if (needed) to_inv[lane] = inv;
}
// What the other warp shared.
__device__ __forceinline__ void shared_by(uint32_t (&hi)[2][4], uint32_t (&lo)[2][4], float2& inv,
                                          const uint4 (&from)[4][32], const float2 (&from_inv)[32], int lane) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) from_uint4(hi[kt], from[2 * kt][lane]), from_uint4(lo[kt], from[2 * kt + 1][lane]);
    inv = from_inv[lane];
}
// The outer product of both halves of the tokens: this warp's t and, through `ex`, the other one's. `pair` is the two
// warps' barrier.
template <int D, int NB, typename Pair>
__device__ __forceinline__ void add_outer_both(float (&w)[D / 16][4], float decay, const float (&t)[4][4], float factor,
                                               uint4 (&ex)[2][4][32], float2 (&ex_inv)[2][32], uint32_t tile, int half,
                                               int lane, Pair pair) {
    uint32_t hi[2][4], lo[2][4];
    float2 inv;
    share(t, hi, lo, inv, ex[half], ex_inv[half], lane);
    const int col0 = half * (D / 2);
    add_outer<D, NB>(w, decay, hi, lo, inv.x * factor, inv.y * factor, tile, col0, half * 32, lane);
    pair();
    shared_by(hi, lo, inv, ex[half ^ 1], ex_inv[half ^ 1], lane);
    add_outer<D, NB>(w, 1.f, hi, lo, inv.x * factor, inv.y * factor, tile, col0, 32 - half * 32, lane);
}

// The state's sixteen rows times the tokens of K (tile): out, the own half of the tokens. inv: inverse scales of this warp's half of
// the columns; keep(kt, hi, lo) sees the fragments of its k-step kt.
template <int D, int NP, typename Pair, typename Keep>
__device__ __forceinline__ void times_tokens(float (&out)[4][4], const float (&w)[D / 16][4], float2& inv, uint32_t tile,
                                             float4 (&ex)[2][4][32], int half, int lane, Pair pair, Keep keep) {
    float top0, top1;
    row_tops<D / 16>(w, top0, top1);
    const float s0 = pow2_scale(top0, inv.x), s1 = pow2_scale(top1, inv.y);
    float x[8][4] = {};
#pragma unroll
    for (int kt = 0; kt < D / 32; ++kt) {
        uint32_t hi[4], lo[4];
        split_a<D / 16>(w, kt, s0, s1, hi, lo);
        mma_row<2, NP, 0, 4>(x, hi, lo, [&](uint32_t(&f)[4], int j, int e) {  // n-tiles in the order own, other half
            frag_b<D>(f, tile + e * kC * D * 2, ((j + 2 * half) & 3) * 16, half * (D / 2) + kt * 16, lane);
        });
        keep(kt, hi, lo);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ex[half][i][lane] = make_float4(x[4 + i][0] * inv.x, x[4 + i][1] * inv.x, x[4 + i][2] * inv.y, x[4 + i][3] * inv.y);
    pair();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 u = ex[half ^ 1][i][lane];
        out[i][0] = fmaf(x[i][0], inv.x, u.x), out[i][1] = fmaf(x[i][1], inv.x, u.y);
        out[i][2] = fmaf(x[i][2], inv.y, u.z), out[i][3] = fmaf(x[i][3], inv.y, u.w);
    }
}

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
