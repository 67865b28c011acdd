// Gated delta rule, backward: the adjoint's way back through the chunks.
//
// With A the adjoint of a chunk's final state, and the names of delta_common.cuh,
//   dE = P^T dY + l K A^T,  dR = dE - N^T (beta dE)   (dR: adjoint of beta X, so dV = beta dR)
//   A <- gamma_C A + (gamma dY)^T Q - (beta gamma dR)^T K
// which runs over rows of A as the forward runs over rows of W: the same pairs of warps with sixteen rows each in
// registers, half of the columns and of the tokens a warp, the same stages and producers (delta_stage.cuh), chunks in
// falling order. Here the first half's dE and dR need the second half's dY and beta dE. It leaves A and dR of each
// chunk for the tokens' gradients, which do not depend on one another.
// Bound like the forward by the chain of a chunk: 128 units of 64 chunks, d = 64, take 246 us, 3.8 us a chunk, with the issue slots 40 %
// busy and HBM 8 %.
#include "delta_stage.cuh"

namespace titans {
namespace {

constexpr int kFull = 0, kFree = 2, kPair = 4;  // named barriers

struct Swap {
    float4 part[2][4][32];                // partial sums of A K^T; [0], once read, beta dE of the second half
    uint4 outer[2][2][4][32], dy[4][32];  // left sides of the outer products (gamma dY; beta gamma dR); dY of the second half
    float2 inv[32], outer_inv[2][2][32], dy_inv[32];
};

template <int D, int RW, typename Tok>
__global__ void __launch_bounds__(RW * 4 + kProducers, 1)
    delta_adjoint_kernel(DeltaArgs a, const DeltaChunk* recs, int chunks, DeltaGrads g) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, kChain = RW / 8, kThreads = kChain * 32 + kProducers;
    static_assert(RW <= 64, "barriers");
    using S = Stage<D, RW, NP, 2>;
    extern __shared__ __align__(1024) unsigned char smem[];
    S* stages = reinterpret_cast<S*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kSlices = D / RW;
    const long unit = blockIdx.x / kSlices;
    const int row_base = (int)(blockIdx.x % kSlices) * RW;
    const long len = delta_length(a, unit / a.H);
    const int used = (int)((len + kC - 1) / kC);
    const DeltaChunk* rec = recs + unit * chunks;

    if (warp >= kChain) {  // ------------------------------------------- producers
        const int p = tid - kChain * 32;
        const Tok* k = static_cast<const Tok*>(a.k) + delta_key_head(a, unit) * a.T * D;
        const Tok* q = static_cast<const Tok*>(a.q) + delta_key_head(a, unit) * a.T * D;
        const Tok* dy = static_cast<const Tok*>(g.dy) + unit * a.T * D + row_base;
        Producer<D, RW, Tok, 2, true> next;
        auto fetch = [&](int c) { next.fetch(k, q, dy, (long)c * kC, (int)min((long)kC, len - (long)c * kC), p); };
        if (used > 0) fetch(used - 1);
        for (int c = used - 1, i = 0; c >= 0; --c, ++i) {
            if (i >= 2) bar_sync(kFree + (i & 1), kThreads);
            next.store(stages[i & 1], rec[c], p);
            bar_arrive(kFull + (i & 1), kThreads);
            if (c > 0) fetch(c - 1);
        }
        return;
    }
    // --------------------------------------------------------------------- the adjoint: a pair of warps for sixteen rows
    const int group = warp >> 1, half = warp & 1, tok0 = 32 * half, col0 = half * (D / 2), col2 = 2 * (lane & 3);
    Swap& ex = reinterpret_cast<Swap*>(smem + 2 * sizeof(S))[group];
    auto pair = [&] { bar_sync(kPair + group, 64); };
    const int row = row_base + group * 16 + (lane >> 2);
    float w[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        float2 u = make_float2(0.f, 0.f), z = u;
        if (g.dW) {
            const float* src = g.dW + (unit * D + row) * D + col0 + col2;
            u = *reinterpret_cast<const float2*>(src + 8 * i);
            z = *reinterpret_cast<const float2*>(src + 8 * D + 8 * i);
        }
        w[i][0] = u.x, w[i][1] = u.y, w[i][2] = z.x, w[i][3] = z.y;
    }
    auto write = [&](float* matrix) {
        float* o = matrix + row * D + col0 + col2;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            *reinterpret_cast<float2*>(o + 8 * t) = make_float2(w[t][0], w[t][1]);
            *reinterpret_cast<float2*>(o + 8 * D + 8 * t) = make_float2(w[t][2], w[t][3]);
        }
    };
    for (int c = used - 1, i = 0; c >= 0; --c, ++i) {
        S& s = stages[i & 1];
        write(g.adj + (unit * chunks + c) * D * D);
        bar_sync(kFull + (i & 1), kThreads);
        const uint32_t ks = smem_u32(s.k), qs = smem_u32(s.q), ns = smem_u32(s.n), ps = smem_u32(s.p);
        const float k_inv = s.scal[2], q_inv = s.scal[3], n_inv = s.scal[4], p_inv = s.scal[5];
        const float* vs = s.v + group * 16 + (lane >> 2);
        // dY^T of the own tokens (row: value, column: token) and gamma dY^T as fragments
        float v[4][4];
        uint32_t y_hi[2][4], y_lo[2][4], o_hi[2][4], o_lo[2][4];
        float2 y_inv, o_inv;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float* v0 = vs + (tok0 + 8 * t + col2) * S::kVLd;
            v[t][0] = v0[0], v[t][1] = v0[S::kVLd], v[t][2] = v0[8], v[t][3] = v0[S::kVLd + 8];
        }
        share(v, y_hi, y_lo, y_inv, ex.dy, ex.dy_inv, lane, half == 1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok0 + 8 * t + col2);
            v[t][0] *= gm.x, v[t][1] *= gm.y, v[t][2] *= gm.x, v[t][3] *= gm.y;
        }
        share(v, o_hi, o_lo, o_inv, ex.outer[0][half], ex.outer_inv[0][half], lane);
        float x[4][4];  // A K^T, then dE^T, then dR^T of the own tokens
        float2 inv;
        times_tokens<D, NP>(x, w, inv, ks, ex.part, half, lane, pair,
                            [](int, const uint32_t(&)[4], const uint32_t(&)[4]) {});
        // A <- gamma_C A + (gamma dY)^T Q
        add_outer<D, NP>(w, s.gamma[kC - 1], o_hi, o_lo, o_inv.x * q_inv, o_inv.y * q_inv, qs, col0, tok0, lane);
        shared_by(o_hi, o_lo, o_inv, ex.outer[0][half ^ 1], ex.outer_inv[0][half ^ 1], lane);
        add_outer<D, NP>(w, 1.f, o_hi, o_lo, o_inv.x * q_inv, o_inv.y * q_inv, qs, col0, 32 - tok0, lane);
        // acc[.] += t B for the own tokens' columns of a lower triangular tile, t the own tokens or (first half) the others
        auto own = [&](float(&acc)[4][4], const uint32_t(&hi)[2][4], const uint32_t(&lo)[2][4], uint32_t tile) {
            auto from = [&](int k) {
                return [=](uint32_t(&f)[4], int j, int e) {
                    frag_bt<kC>(f, tile + e * kC * kC * 2, tok0 + j * 16, tok0 + k * 16, lane);
                };
            };
            mma_row<2, 2, 0, 1>(acc, hi[0], lo[0], from(0));
            mma_row<2, 2, 0, 2>(acc, hi[1], lo[1], from(1));
        };
        auto cross = [&](float(&acc)[4][4], const uint32_t(&hi)[2][4], const uint32_t(&lo)[2][4], uint32_t tile) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
                mma_row<2, 2, 0, 2>(acc, hi[kt], lo[kt], [&](uint32_t(&f)[4], int j, int e) {
                    frag_bt<kC>(f, tile + e * kC * kC * 2, j * 16, 32 + kt * 16, lane);
                });
        };
        auto add = [&](const float(&acc)[4][4], float f0, float f1) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[t][0] = fmaf(acc[t][0], f0, x[t][0]), x[t][1] = fmaf(acc[t][1], f0, x[t][1]);
                x[t][2] = fmaf(acc[t][2], f1, x[t][2]), x[t][3] = fmaf(acc[t][3], f1, x[t][3]);
            }
        };
        {  // dE^T = l (A K^T) + dY^T P
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 l = *reinterpret_cast<const float2*>(s.rest + tok0 + 8 * t + col2);
                x[t][0] *= l.x * k_inv, x[t][1] *= l.y * k_inv, x[t][2] *= l.x * k_inv, x[t][3] *= l.y * k_inv;
            }
            float acc[4][4] = {};
            own(acc, y_hi, y_lo, ps);
            add(acc, y_inv.x * p_inv, y_inv.y * p_inv);
            if (half == 0) {
                float far[4][4] = {};
                shared_by(y_hi, y_lo, y_inv, ex.dy, ex.dy_inv, lane);
                cross(far, y_hi, y_lo, ps);
                add(far, y_inv.x * p_inv, y_inv.y * p_inv);
            }
        }
        {  // dR^T = dE^T - (beta dE)^T N
            uint4(&other)[4][32] = reinterpret_cast<uint4(&)[4][32]>(ex.part[0]);
            float r[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok0 + 8 * t + col2);
                r[t][0] = bt.x * x[t][0], r[t][1] = bt.y * x[t][1], r[t][2] = bt.x * x[t][2], r[t][3] = bt.y * x[t][3];
            }
            share(r, y_hi, y_lo, y_inv, other, ex.inv, lane, half == 1);
            float acc[4][4] = {};
            own(acc, y_hi, y_lo, ns);
            add(acc, -y_inv.x * n_inv, -y_inv.y * n_inv);
            pair();
            if (half == 0) {
                float far[4][4] = {};
                shared_by(y_hi, y_lo, y_inv, other, ex.inv, lane);
                cross(far, y_hi, y_lo, ns);
                add(far, -y_inv.x * n_inv, -y_inv.y * n_inv);
            }
        }
        float* o = g.dr + ((unit * chunks + c) * kC + tok0) * D + row;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int tok = tok0 + 8 * t + col2;
            const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok);
            const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[(long)(8 * t + col2 + (e & 1)) * D + (e >> 1) * 8] = x[t][e];
            x[t][0] *= bt.x * gm.x, x[t][1] *= bt.y * gm.y, x[t][2] *= bt.x * gm.x, x[t][3] *= bt.y * gm.y;
        }
        // A <- A - (beta gamma dR)^T K
        add_outer_both<D, NP>(w, 1.f, x, -k_inv, ex.outer[1], ex.outer_inv[1], ks, half, lane, pair);
        if (c >= 2) bar_arrive(kFree + (i & 1), kThreads);
    }
    write(g.dW0 + unit * D * D);
}

template <int D, int RW, typename Tok>
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaGrads& g, cudaStream_t st) {
    constexpr size_t bytes = 2 * sizeof(Stage<D, RW, sizeof(Tok) == 4 ? 2 : 1, 2>) + RW / 16 * sizeof(Swap);
    static_assert(bytes <= 227 * 1024, "two stages and the exchanges fit an SM");
    auto* kernel = delta_adjoint_kernel<D, RW, Tok>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long)a.B * a.H * (D / RW)), RW * 4 + kProducers, bytes, st>>>(
        a, static_cast<const DeltaChunk*>(recs), (int)((a.T + kC - 1) / kC), g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_adjoint(const DeltaArgs& a, const void* chunks, const DeltaGrads& g, cudaStream_t st) {
    if (a.d == 64)
        return a.bf16 ? launch<64, 64, __nv_bfloat16>(a, chunks, g, st) : launch<64, 32, float>(a, chunks, g, st);
    return a.bf16 ? launch<128, 32, __nv_bfloat16>(a, chunks, g, st) : launch<128, 16, float>(a, chunks, g, st);
}

}  // namespace titans
