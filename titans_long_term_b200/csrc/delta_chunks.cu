// Gated delta rule, second kernel of the chunked path: the state's way through the chunks, and y.
//
// What is serial is the state: each chunk's writes need it (X = V - gamma K W0^T). Rows of W are independent, so
// a warp keeps sixteen of them in registers as the accumulator of its tensor-core products, which is also the layout
// of their next A operand: per chunk it takes W0 K^T and W0 Q^T, E^T from N, P E, and adds (l E)^T K to W, without
// exchanging anything with other warps and without W ever leaving registers. A CTA has 64 rows (32 in
// fp32 mode at d = 128), four or two such warps, and four producer warps that bring the next chunk's K, Q, V, N
// and P into a second stage of shared memory meanwhile, the tokens split into fp16 pieces on the way.
//
// The serial chain bounds it: with few units most SMs have one warp per tensor core, which runs
// 448 (d = 64) or 816 (d = 128) m16n8k16 products per chunk one after another.
#include "delta_stage.cuh"

namespace titans {
namespace {

template <int D, int RW, typename Tok, bool STATES>
__global__ void __launch_bounds__(RW * 2 + kProducers, 1)
    delta_chunks_kernel(DeltaArgs a, const DeltaChunk* recs, int chunks, DeltaStates st) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, NW = RW / 16, kThreads = NW * 32 + kProducers;
    using S = Stage<D, RW, NP, NP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    S* stages = reinterpret_cast<S*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kSlices = D / RW;
    const long unit = blockIdx.x / kSlices;
    const int row_base = (int)(blockIdx.x % kSlices) * RW;
    const long b = unit / a.H, len = delta_length(a, b);
    const int used = (int)((len + kC - 1) / kC);
    const DeltaChunk* rec = recs + unit * chunks;
    // barriers 1, 2: stage filled; 3, 4: stage free

    if (warp >= NW) {  // ------------------------------------------------ producers
        const int p = tid - NW * 32;
        const Tok* k = static_cast<const Tok*>(a.k) + delta_key_head(a, unit) * a.T * D;
        const Tok* q = static_cast<const Tok*>(a.q) + delta_key_head(a, unit) * a.T * D;
        const Tok* v = static_cast<const Tok*>(a.v) + unit * a.T * D + row_base;
        Producer<D, RW, Tok, NP, !STATES> next;
        auto fetch = [&](int c) { next.fetch(k, q, v, (long)c * kC, (int)min((long)kC, len - (long)c * kC), p); };
        if (used > 0) fetch(0);
        for (int c = 0; c < used; ++c) {
            if (c >= 2) bar_sync(3 + (c & 1), kThreads);
            next.store(stages[c & 1], rec[c], p);
            bar_arrive(1 + (c & 1), kThreads);
            if (c + 1 < used) fetch(c + 1);
        }
    } else {  // --------------------------------------------------------- sixteen rows of the state a warp
        const int row = row_base + warp * 16 + (lane >> 2), col2 = 2 * (lane & 3);
        float w[D / 8][4];
        float* W = a.W + unit * D * D + (long)row * D + col2;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const float2 u = *reinterpret_cast<const float2*>(W + 8 * i);
            const float2 z = *reinterpret_cast<const float2*>(W + 8 * D + 8 * i);
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = z.x, w[i][3] = z.y;
        }
        for (int c = 0; c < used; ++c) {
            S& s = stages[c & 1];
            if constexpr (STATES) {
                float* o = st.states + ((unit * chunks + c) * D + row) * D + col2;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    *reinterpret_cast<float2*>(o + 8 * i) = make_float2(w[i][0], w[i][1]);
                    *reinterpret_cast<float2*>(o + 8 * D + 8 * i) = make_float2(w[i][2], w[i][3]);
                }
            }
            bar_sync(1 + (c & 1), kThreads);
            const uint32_t ks = smem_u32(s.k), qs = smem_u32(s.q), ns = smem_u32(s.n), ps = smem_u32(s.p);
            const float k_inv = s.scal[2], q_inv = s.scal[3], n_inv = s.scal[4], p_inv = s.scal[5];
            float* vs = s.v + warp * 16 + (lane >> 2);
            // W0 K^T and W0 Q^T
            float x[8][4] = {}, y[STATES ? 1 : 8][4] = {};
            float i0, i1;  // inverse scales of the two rows
            {
                float top0, top1;
                row_tops<D / 8>(w, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
#pragma unroll
                for (int kt = 0; kt < D / 16; ++kt) {
                    uint32_t hi[4], lo[4];
                    split_a<D / 8>(w, kt, s0, s1, hi, lo);
                    auto from = [&](uint32_t tile) {
                        return [=](uint32_t(&f)[4], int j, int e) { frag_b<D>(f, tile + e * kC * D * 2, j * 16, kt * 16, lane); };
                    };
                    mma_row<2, NP, 0, 4>(x, hi, lo, from(ks));
                    // y is rounded to the tokens' type: 11 bits of W are enough for bf16
                    if constexpr (!STATES) mma_row<NP, NP, 0, 4>(y, hi, lo, from(qs));
                }
            }
            // X^T = V^T - gamma W0 K^T (row: value, column: token), and Y's share of W0
            float r[8][4];  // beta X
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int tok = 8 * t + col2;
                const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok);
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok);
                const float* v0 = vs + tok * S::kVLd;
                x[t][0] = v0[0] - gm.x * k_inv * (x[t][0] * i0);
                x[t][1] = v0[S::kVLd] - gm.y * k_inv * (x[t][1] * i0);
                x[t][2] = v0[8] - gm.x * k_inv * (x[t][2] * i1);
                x[t][3] = v0[S::kVLd + 8] - gm.y * k_inv * (x[t][3] * i1);
                r[t][0] = bt.x * x[t][0], r[t][1] = bt.y * x[t][1];
                r[t][2] = bt.x * x[t][2], r[t][3] = bt.y * x[t][3];
                if constexpr (!STATES) {
                    y[t][0] *= gm.x * q_inv * i0, y[t][1] *= gm.y * q_inv * i0;
                    y[t][2] *= gm.x * q_inv * i1, y[t][3] *= gm.y * q_inv * i1;
                }
            }
            // eps^T = X^T - (beta X)^T N^T; N is strictly lower: tokens 16 j + .. see those up to them
            {
                float top0, top1;
                row_tops<8>(r, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
                float acc[8][4] = {};
                unrolled<4>([&](auto kt) {
                    uint32_t hi[4], lo[4];
                    split_a<8>(r, kt, s0, s1, hi, lo);
                    mma_triangle<kt, true, 2, 2>(acc, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                        frag_b<kC>(f, ns + e * kC * kC * 2, j * 16, kt * 16, lane);
                    });
                });
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    x[t][0] -= acc[t][0] * i0 * n_inv, x[t][1] -= acc[t][1] * i0 * n_inv;
                    x[t][2] -= acc[t][2] * i1 * n_inv, x[t][3] -= acc[t][3] * i1 * n_inv;
                }
            }
            if constexpr (STATES) {
                float* o = st.eps + ((unit * chunks + c) * kC) * D + row;
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[(long)(8 * t + col2 + (e & 1)) * D + (e >> 1) * 8] = x[t][e];
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {  // E = beta eps
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + 8 * t + col2);
                x[t][0] *= bt.x, x[t][1] *= bt.y, x[t][2] *= bt.x, x[t][3] *= bt.y;
            }
            if constexpr (!STATES) {  // Y^T += E^T P^T
                float top0, top1;
                row_tops<8>(x, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
                float acc[8][4] = {};
                unrolled<4>([&](auto kt) {
                    uint32_t hi[4], lo[4];
                    split_a<8>(x, kt, s0, s1, hi, lo);
                    mma_triangle<kt, true, NP, NP>(acc, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                        frag_b<kC>(f, ps + e * kC * kC * 2, j * 16, kt * 16, lane);
                    });
                });
#pragma unroll
                for (int t = 0; t < 8; ++t) {  // into V's place, whose columns only this warp reads
                    float* v0 = vs + (8 * t + col2) * S::kVLd;
                    v0[0] = y[t][0] + acc[t][0] * i0 * p_inv;
                    v0[S::kVLd] = y[t][1] + acc[t][1] * i0 * p_inv;
                    v0[8] = y[t][2] + acc[t][2] * i1 * p_inv;
                    v0[S::kVLd + 8] = y[t][3] + acc[t][3] * i1 * p_inv;
                }
            }
            // W = gamma_C W + (l E)^T K
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 l = *reinterpret_cast<const float2*>(s.rest + 8 * t + col2);
                x[t][0] *= l.x, x[t][1] *= l.y, x[t][2] *= l.x, x[t][3] *= l.y;
            }
            {
                float top0, top1;
                row_tops<8>(x, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
                add_outer<D, NP>(w, s.gamma[kC - 1], x, s0, s1, i0 * k_inv, i1 * k_inv, ks, lane);
            }
            if constexpr (!STATES) {  // two lanes a token: 32 or 64 bytes of its row
                __syncwarp();
                const long t0 = (long)c * kC;
                const int n = (int)min((long)kC, len - t0);
                const long at = (unit * a.T + t0) * D + row_base + warp * 16 + (lane & 1) * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = i * 16 + (lane >> 1);
                    if (tok >= n) continue;
                    float o[8];
                    load8(s.v + tok * S::kVLd + warp * 16 + (lane & 1) * 8, o);
                    if (a.attn) {
                        float g[8];
                        load8(static_cast<const Tok*>(a.attn) + at + (long)tok * D, g);
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = g[j] / (1.f + expf(-o[j]));
                    }
                    store8(static_cast<Tok*>(a.y) + at + (long)tok * D, o);
                }
            }
            if (c + 2 < used) bar_arrive(3 + (c & 1), kThreads);
        }
        if constexpr (!STATES) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                *reinterpret_cast<float2*>(W + 8 * i) = make_float2(w[i][0], w[i][1]);
                *reinterpret_cast<float2*>(W + 8 * D + 8 * i) = make_float2(w[i][2], w[i][3]);
            }
        }
    }
    if constexpr (!STATES) {  // nothing is read behind the sequence's end
        const float zero[8] = {};
        for (long i = tid; i < (a.T - len) * (RW / 8); i += kThreads)
            store8(static_cast<Tok*>(a.y) + (unit * a.T + len + i / (RW / 8)) * D + row_base + i % (RW / 8) * 8, zero);
    }
}

template <int D, int RW, typename Tok, bool STATES>
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaStates& states, cudaStream_t st) {
    constexpr size_t bytes = 2 * sizeof(Stage<D, RW, sizeof(Tok) == 4 ? 2 : 1, sizeof(Tok) == 4 ? 2 : 1>);
    static_assert(bytes <= 227 * 1024, "two stages fit an SM");
    auto* kernel = delta_chunks_kernel<D, RW, Tok, STATES>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long)a.B * a.H * (D / RW)), RW * 2 + kProducers, bytes, st>>>(
        a, static_cast<const DeltaChunk*>(recs), (int)((a.T + kC - 1) / kC), states);
    return cudaGetLastError();
}

template <bool STATES>
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaStates& s, cudaStream_t st) {
    if (a.d == 64)
        return a.bf16 ? launch<64, 64, __nv_bfloat16, STATES>(a, recs, s, st) : launch<64, 64, float, STATES>(a, recs, s, st);
    return a.bf16 ? launch<128, 64, __nv_bfloat16, STATES>(a, recs, s, st) : launch<128, 32, float, STATES>(a, recs, s, st);
}

}  // namespace

cudaError_t launch_delta_chunks(const DeltaArgs& a, const void* chunks, const DeltaStates* states, cudaStream_t st) {
    return states ? launch<true>(a, chunks, *states, st) : launch<false>(a, chunks, DeltaStates{}, st);
}

}  // namespace titans
