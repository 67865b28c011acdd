// Gated delta rule, backward: the adjoint's way back through the chunks.
//
// With A the adjoint of a chunk's final state, and the names of delta_common.cuh,
//   dE = P^T dY + l K A^T,  dR = dE - N^T (beta dE)   (dR: adjoint of beta X, so dV = beta dR)
//   A <- gamma_C A + (gamma dY)^T Q - (beta gamma dR)^T K
// which runs over rows of A as the forward runs over rows of W: the same sixteen rows a warp in registers, the
// same stages and producers (delta_stage.cuh), chunks in falling order. It leaves A and dR of each chunk for
// the tokens' gradients, which do not depend on one another.
#include "delta_stage.cuh"

namespace titans {
namespace {

template <int D, int RW, typename Tok>
__global__ void __launch_bounds__(RW * 2 + kProducers, 1)
    delta_adjoint_kernel(DeltaArgs a, const DeltaChunk* recs, int chunks, DeltaGrads g) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, NW = RW / 16, kThreads = NW * 32 + kProducers;
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
    // barriers 1, 2: stage filled; 3, 4: stage free

    if (warp >= NW) {  // ------------------------------------------------ producers
        const int p = tid - NW * 32;
        const Tok* k = static_cast<const Tok*>(a.k) + delta_key_head(a, unit) * a.T * D;
        const Tok* q = static_cast<const Tok*>(a.q) + delta_key_head(a, unit) * a.T * D;
        const Tok* dy = static_cast<const Tok*>(g.dy) + unit * a.T * D + row_base;
        Producer<D, RW, Tok, 2, true> next;
        auto fetch = [&](int c) { next.fetch(k, q, dy, (long)c * kC, (int)min((long)kC, len - (long)c * kC), p); };
        if (used > 0) fetch(used - 1);
        for (int c = used - 1, i = 0; c >= 0; --c, ++i) {
            if (i >= 2) bar_sync(3 + (i & 1), kThreads);
            next.store(stages[i & 1], rec[c], p);
            bar_arrive(1 + (i & 1), kThreads);
            if (c > 0) fetch(c - 1);
        }
        return;
    }
    // --------------------------------------------------------------------- sixteen rows of the adjoint a warp
    const int row = row_base + warp * 16 + (lane >> 2), col2 = 2 * (lane & 3);
    float w[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        float2 u = make_float2(0.f, 0.f), z = u;
        if (g.dW) {
            const float* src = g.dW + (unit * D + row) * D + col2;
            u = *reinterpret_cast<const float2*>(src + 8 * i);
            z = *reinterpret_cast<const float2*>(src + 8 * D + 8 * i);
        }
        w[i][0] = u.x, w[i][1] = u.y, w[i][2] = z.x, w[i][3] = z.y;
    }
    for (int c = used - 1, i = 0; c >= 0; --c, ++i) {
        S& s = stages[i & 1];
        {
            float* o = g.adj + ((unit * chunks + c) * D + row) * D + col2;
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
                *reinterpret_cast<float2*>(o + 8 * t) = make_float2(w[t][0], w[t][1]);
                *reinterpret_cast<float2*>(o + 8 * D + 8 * t) = make_float2(w[t][2], w[t][3]);
            }
        }
        bar_sync(1 + (i & 1), kThreads);
        const uint32_t ks = smem_u32(s.k), qs = smem_u32(s.q), ns = smem_u32(s.n), ps = smem_u32(s.p);
        const float k_inv = s.scal[2], q_inv = s.scal[3], n_inv = s.scal[4], p_inv = s.scal[5];
        const float* vs = s.v + warp * 16 + (lane >> 2);
        float x[8][4] = {};  // (A K^T), then dE^T, then dR^T
        float i0, i1;
        {
            float top0, top1;
            row_tops<D / 8>(w, top0, top1);
            const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
#pragma unroll
            for (int kt = 0; kt < D / 16; ++kt) {
                uint32_t hi[4], lo[4];
                split_a<D / 8>(w, kt, s0, s1, hi, lo);
                mma_row<2, NP, 0, 4>(x, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                    frag_b<D>(f, ks + e * kC * D * 2, j * 16, kt * 16, lane);
                });
            }
        }
        {  // dE^T = l (A K^T) + dY^T P
            float v[8][4], acc[8][4] = {};
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int tok = 8 * t + col2;
                const float* v0 = vs + tok * S::kVLd;
                v[t][0] = v0[0], v[t][1] = v0[S::kVLd], v[t][2] = v0[8], v[t][3] = v0[S::kVLd + 8];
                const float2 l = *reinterpret_cast<const float2*>(s.rest + tok);
                x[t][0] *= l.x * k_inv * i0, x[t][1] *= l.y * k_inv * i0;
                x[t][2] *= l.x * k_inv * i1, x[t][3] *= l.y * k_inv * i1;
            }
            float top0, top1;
            row_tops<8>(v, top0, top1);
            const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
            unrolled<4>([&](auto kt) {  // P_ij, i >= j
                uint32_t hi[4], lo[4];
                split_a<8>(v, kt, s0, s1, hi, lo);
                mma_triangle<kt, false, 2, 2>(acc, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                    frag_bt<kC>(f, ps + e * kC * kC * 2, j * 16, kt * 16, lane);
                });
            });
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                x[t][0] += acc[t][0] * i0 * p_inv, x[t][1] += acc[t][1] * i0 * p_inv;
                x[t][2] += acc[t][2] * i1 * p_inv, x[t][3] += acc[t][3] * i1 * p_inv;
            }
            // A <- gamma_C A + (gamma dY)^T Q
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 gm = *reinterpret_cast<const float2*>(s.gamma + 8 * t + col2);
                v[t][0] *= gm.x, v[t][1] *= gm.y, v[t][2] *= gm.x, v[t][3] *= gm.y;
            }
            row_tops<8>(v, top0, top1);
            const float r0 = pow2_scale(top0, i0), r1 = pow2_scale(top1, i1);
            add_outer<D, NP>(w, s.gamma[kC - 1], v, r0, r1, i0 * q_inv, i1 * q_inv, qs, lane);
        }
        {  // dR^T = dE^T - (beta dE)^T N
            float r[8][4], acc[8][4] = {};
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + 8 * t + col2);
                r[t][0] = bt.x * x[t][0], r[t][1] = bt.y * x[t][1], r[t][2] = bt.x * x[t][2], r[t][3] = bt.y * x[t][3];
            }
            float top0, top1;
            row_tops<8>(r, top0, top1);
            const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
            unrolled<4>([&](auto kt) {  // N_ij, i > j
                uint32_t hi[4], lo[4];
                split_a<8>(r, kt, s0, s1, hi, lo);
                mma_triangle<kt, false, 2, 2>(acc, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                    frag_bt<kC>(f, ns + e * kC * kC * 2, j * 16, kt * 16, lane);
                });
            });
            float* o = g.dr + (unit * chunks + c) * kC * D + row;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int tok = 8 * t + col2;
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok);
                const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok);
                x[t][0] -= acc[t][0] * i0 * n_inv, x[t][1] -= acc[t][1] * i0 * n_inv;
                x[t][2] -= acc[t][2] * i1 * n_inv, x[t][3] -= acc[t][3] * i1 * n_inv;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[(long)(tok + (e & 1)) * D + (e >> 1) * 8] = x[t][e];
                x[t][0] *= bt.x * gm.x, x[t][1] *= bt.y * gm.y, x[t][2] *= bt.x * gm.x, x[t][3] *= bt.y * gm.y;
            }
        }
        {  // A <- A - (beta gamma dR)^T K
            float top0, top1;
            row_tops<8>(x, top0, top1);
            const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
            add_outer<D, NP>(w, 1.f, x, s0, s1, -k_inv * i0, -k_inv * i1, ks, lane);
        }
        if (c >= 2) bar_arrive(3 + (i & 1), kThreads);
    }
    float* o = g.dW0 + (unit * D + row) * D + col2;
#pragma unroll
    for (int t = 0; t < D / 8; ++t) {
        *reinterpret_cast<float2*>(o + 8 * t) = make_float2(w[t][0], w[t][1]);
        *reinterpret_cast<float2*>(o + 8 * D + 8 * t) = make_float2(w[t][2], w[t][3]);
    }
}

template <int D, int RW, typename Tok>
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaGrads& g, cudaStream_t st) {
    constexpr size_t bytes = 2 * sizeof(Stage<D, RW, sizeof(Tok) == 4 ? 2 : 1, 2>);
    static_assert(bytes <= 227 * 1024, "two stages fit an SM");
    auto* kernel = delta_adjoint_kernel<D, RW, Tok>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long)a.B * a.H * (D / RW)), RW * 2 + kProducers, bytes, st>>>(
        a, static_cast<const DeltaChunk*>(recs), (int)((a.T + kC - 1) / kC), g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_adjoint(const DeltaArgs& a, const void* chunks, const DeltaGrads& g, cudaStream_t st) {
    if (a.d == 64)
        return a.bf16 ? launch<64, 64, __nv_bfloat16>(a, chunks, g, st) : launch<64, 64, float>(a, chunks, g, st);
    return a.bf16 ? launch<128, 64, __nv_bfloat16>(a, chunks, g, st) : launch<128, 32, float>(a, chunks, g, st);
}

}  // namespace titans
