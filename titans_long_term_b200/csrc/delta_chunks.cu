// Gated delta rule, second kernel of the chunked path: the state's way through the chunks, and y.
//
// What is serial is the state: each chunk's writes need it (X = V - gamma K W0^T), and the next chunk needs them. Rows of
// W are independent, so sixteen of them stay with one or two warps from the first chunk to the last, in registers, as the
// accumulators of tensor-core products, which is also the layout of their next A operand; nothing is exchanged with other
// rows. The chain of a chunk bounds this kernel, with few units all the more (a warp on each tensor core, its
// steps one after another), so it is kept short:
//   - at d = 128, and in fp32, a pair halves it: each warp has half of W's columns, adds up W0 K^T over them and hands the other warp its
//     tokens' part; then each has half of the tokens (the second half's eps need the first half's beta X), and gives the
//     other the fragments of l E for its columns (Exchange in delta_stage.cuh). At d = 64 in bf16 the steps are so short
//     that handing over costs more than it saves (64 chunks of 128 units: 177 us with a pair, 156 us with one warp), and one
//     warp has all;
//   - two more warps of the same rows, half of the tokens each, take what the next chunk does not wait for:
//     Y = gamma Q W0^T + P E, its gate and its stores, from the same fragments;
//   - four producer warps bring the next chunk's K, Q, V, N and P into a second stage of shared memory meanwhile, the tokens
//     split into fp16 pieces on the way.
// 128 units of 64 chunks, d = 64: 183 us, 2.9 us a chunk (155 us where the states and eps are left for the backward pass instead of y);
// 32 units of 256 chunks, d = 128: 732 us, also 2.9 us. One chain warp a tensor core: the issue slots are 36 % busy, HBM 8 %.
#include "delta_stage.cuh"

namespace titans {
namespace {

// Named barriers; all threads take part in the stages', a group's warps in its own.
constexpr int kFull = 0, kFree = 2, kPair = 4, kOutFull = 8, kOutFree = 12;

template <int D, int RW, int NP, bool STATES>
struct Warps {
    static constexpr int kPerGroup = D == 64 && NP == 1 ? 1 : 2, kGroups = RW / 16;
    static constexpr int kChain = kPerGroup * kGroups, kOut = STATES ? 0 : 2 * kGroups;
    static constexpr int kThreads = (kChain + kOut) * 32 + kProducers, kGroupThreads = (kPerGroup + 2) * 32;
    static_assert(kGroups <= 4, "sixteen barriers");
    // With one warp for all of its rows' state in a CTA of 512 threads, the chain takes over registers of the others
    static constexpr bool kShift = kPerGroup == 1 && !STATES;
    static constexpr int kChainRegs = 232, kOutRegs = 104, kProducerRegs = 72;
    static constexpr int kShares = 128 * (kChainRegs + 2 * kOutRegs + kProducerRegs);
};

// YP: pieces of W, E and P that y is taken from. A bf16 y without a gate takes one of each, 11 bits: it is rounded to 8 itself
// (128 units of 64 chunks, d = 64: 331 us for the call against 388 with two; error against 64 bits 1.69e-3 of y's norm against 1.66e-3,
// most of it that rounding). A gate's output has its own rounding, beside which sigmoid(y) has to be right to an absolute error
// that 11 bits of a large state do not give.
template <int D, int RW, typename Tok, bool STATES, int YP>
__global__ void __launch_bounds__(Warps<D, RW, sizeof(Tok) == 4 ? 2 : 1, STATES>::kThreads, 1)
    delta_chunks_kernel(DeltaArgs a, const DeltaChunk* recs, int chunks, DeltaStates st) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1;
    using T = Warps<D, RW, NP, STATES>;
    constexpr int kThreads = T::kThreads;
    using S = Stage<D, RW, NP, YP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    S* stages = reinterpret_cast<S*>(smem);
    Exchange<D, YP>* exchanges = reinterpret_cast<Exchange<D, YP>*>(smem + 2 * sizeof(S));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kSlices = D / RW;
    const long unit = blockIdx.x / kSlices;
    const int row_base = (int)(blockIdx.x % kSlices) * RW;
    const long b = unit / a.H, len = delta_length(a, b);
    const int used = (int)((len + kC - 1) / kC), col2 = 2 * (lane & 3);
    const DeltaChunk* rec = recs + unit * chunks;

    if (warp >= T::kChain + T::kOut) {  // ------------------------------ producers
        if constexpr (T::kShift) registers_down<T::kProducerRegs>();
        const int p = tid - (T::kChain + T::kOut) * 32;
        const Tok* k = static_cast<const Tok*>(a.k) + delta_key_head(a, unit) * a.T * D;
        const Tok* q = static_cast<const Tok*>(a.q) + delta_key_head(a, unit) * a.T * D;
        const Tok* v = static_cast<const Tok*>(a.v) + unit * a.T * D + row_base;
        Producer<D, RW, Tok, YP, !STATES> next;
        auto fetch = [&](int c) { next.fetch(k, q, v, (long)c * kC, (int)min((long)kC, len - (long)c * kC), p); };
        if (used > 0) fetch(0);
        for (int c = 0; c < used; ++c) {
            if (c >= 2) bar_sync(kFree + (c & 1), kThreads);
            next.store(stages[c & 1], rec[c], p);
            bar_arrive(kFull + (c & 1), kThreads);
            if (c + 1 < used) fetch(c + 1);
        }
    } else if (T::kPerGroup == 1 && warp < T::kChain) {  // ------------- the state: one warp for sixteen rows
        if constexpr (T::kShift) registers_up<T::kChainRegs>();
        Exchange<D, YP>& ex = exchanges[warp];
        const int row = row_base + warp * 16 + (lane >> 2);
        float w[D / 8][4];
        float* W = a.W + unit * D * D + (long)row * D + col2;
        auto write = [&](float* o) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                *reinterpret_cast<float2*>(o + 8 * i) = make_float2(w[i][0], w[i][1]);
                *reinterpret_cast<float2*>(o + 8 * D + 8 * i) = make_float2(w[i][2], w[i][3]);
            }
        };
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const float2 u = *reinterpret_cast<const float2*>(W + 8 * i);
            const float2 z = *reinterpret_cast<const float2*>(W + 8 * D + 8 * i);
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = z.x, w[i][3] = z.y;
        }
        for (int c = 0; c < used; ++c) {
            S& s = stages[c & 1];
            if constexpr (STATES) write(st.states + ((unit * chunks + c) * D + row) * D + col2);
            bar_sync(kFull + (c & 1), kThreads);
            const uint32_t ks = smem_u32(s.k), ns = smem_u32(s.n);
            const float k_inv = s.scal[2], n_inv = s.scal[4];
            const float* vs = s.v + warp * 16 + (lane >> 2);
            if (!STATES && c > 0) bar_sync(kOutFree + warp, T::kGroupThreads);
            // X^T = V^T - gamma W0 K^T (row: value, column: token), and beta X
            float x[8][4] = {}, r[8][4], top0, top1, i0, i1;
            {
                row_tops<D / 8>(w, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
#pragma unroll
                for (int kt = 0; kt < D / 16; ++kt) {
                    uint32_t hi[4], lo[4];
                    split_a<D / 8>(w, kt, s0, s1, hi, lo);
                    mma_row<2, NP, 0, 4>(x, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                        frag_b<D>(f, ks + e * kC * D * 2, j * 16, kt * 16, lane);
                    });
                    if constexpr (!STATES) ex.w[0][kt][lane] = as_uint4(hi);
                    if constexpr (!STATES && YP == 2) ex.w[YP - 1][kt][lane] = as_uint4(lo);
                }
                if constexpr (!STATES) ex.w_inv[0][lane] = make_float2(i0, i1);
                i0 *= k_inv, i1 *= k_inv;
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int tok = 8 * t + col2;
                const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok);
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok);
                const float* v0 = vs + tok * S::kVLd;
                x[t][0] = fmaf(-gm.x * i0, x[t][0], v0[0]), x[t][1] = fmaf(-gm.y * i0, x[t][1], v0[S::kVLd]);
                x[t][2] = fmaf(-gm.x * i1, x[t][2], v0[8]), x[t][3] = fmaf(-gm.y * i1, x[t][3], v0[S::kVLd + 8]);
                r[t][0] = bt.x * x[t][0], r[t][1] = bt.y * x[t][1], r[t][2] = bt.x * x[t][2], r[t][3] = bt.y * x[t][3];
            }
            {  // eps^T = X^T - (beta X)^T N^T
                row_tops<8>(r, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
                float acc[8][4] = {};
                unrolled<4>([&](auto kt) {
                    uint32_t hi[4], lo[4];
                    split_a<8>(r, kt, s0, s1, hi, lo);
                    mma_row<2, 2, kt, 4>(acc, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                        frag_b<kC>(f, ns + e * kC * kC * 2, j * 16, kt * 16, lane);
                    });
                });
                i0 *= n_inv, i1 *= n_inv;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    x[t][0] = fmaf(-acc[t][0], i0, x[t][0]), x[t][1] = fmaf(-acc[t][1], i0, x[t][1]);
                    x[t][2] = fmaf(-acc[t][2], i1, x[t][2]), x[t][3] = fmaf(-acc[t][3], i1, x[t][3]);
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
            for (int t = 0; t < 8; ++t) {  // E = beta eps, then l E
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + 8 * t + col2);
                const float2 l = *reinterpret_cast<const float2*>(s.rest + 8 * t + col2);
                x[t][0] *= bt.x, x[t][1] *= bt.y, x[t][2] *= bt.x, x[t][3] *= bt.y;
                r[t][0] = l.x * x[t][0], r[t][1] = l.y * x[t][1], r[t][2] = l.x * x[t][2], r[t][3] = l.y * x[t][3];
            }
            uint32_t hi[4][4], lo[4][4];
            if constexpr (!STATES) {
                row_tops<8>(x, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {
                    split_a<8>(x, kt, s0, s1, hi[kt], lo[kt]);
                    ex.e[0][kt][lane] = as_uint4(hi[kt]);
                    if constexpr (YP == 2) ex.e[YP - 1][kt][lane] = as_uint4(lo[kt]);
                }
                ex.e_inv[0][lane] = make_float2(i0, i1);
                bar_arrive(kOutFull + warp, T::kGroupThreads);
            }
            {  // W = gamma_C W + (l E)^T K
                row_tops<8>(r, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1), decay = s.gamma[kC - 1];
                i0 *= k_inv, i1 *= k_inv;
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) split_a<8>(r, kt, s0, s1, hi[kt], lo[kt]);
                float acc[D / 8][4] = {};
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
                    mma_row<2, NP, 0, D / 16>(acc, hi[kt], lo[kt], [&](uint32_t(&f)[4], int j, int e) {
                        frag_bt<D>(f, ks + e * kC * D * 2, j * 16, kt * 16, lane);
                    });
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    w[j][0] = fmaf(w[j][0], decay, acc[j][0] * i0), w[j][1] = fmaf(w[j][1], decay, acc[j][1] * i0);
                    w[j][2] = fmaf(w[j][2], decay, acc[j][2] * i1), w[j][3] = fmaf(w[j][3], decay, acc[j][3] * i1);
                }
            }
            if (c + 2 < used) bar_arrive(kFree + (c & 1), kThreads);
        }
        if constexpr (!STATES) write(W);
    } else if (warp < T::kChain) {  // ---------------------------------- the state: a pair of warps for sixteen rows
        if constexpr (T::kPerGroup == 2) {
        const int group = warp >> 1, half = warp & 1, tok0 = 32 * half;
        Exchange<D, YP>& ex = exchanges[group];
        auto pair = [&] { bar_sync(kPair + group, 64); };
        const int row = row_base + group * 16 + (lane >> 2);
        float w[D / 16][4];
        float* W = a.W + unit * D * D + (long)row * D + half * (D / 2) + col2;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const float2 u = *reinterpret_cast<const float2*>(W + 8 * i);
            const float2 z = *reinterpret_cast<const float2*>(W + 8 * D + 8 * i);
            w[i][0] = u.x, w[i][1] = u.y, w[i][2] = z.x, w[i][3] = z.y;
        }
        for (int c = 0; c < used; ++c) {
            S& s = stages[c & 1];
            if constexpr (STATES) {
                float* o = st.states + ((unit * chunks + c) * D + row) * D + half * (D / 2) + col2;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    *reinterpret_cast<float2*>(o + 8 * i) = make_float2(w[i][0], w[i][1]);
                    *reinterpret_cast<float2*>(o + 8 * D + 8 * i) = make_float2(w[i][2], w[i][3]);
                }
            }
            bar_sync(kFull + (c & 1), kThreads);
            const uint32_t ks = smem_u32(s.k), ns = smem_u32(s.n);
            const float k_inv = s.scal[2], n_inv = s.scal[4];
            const float* vs = s.v + group * 16 + (lane >> 2);
            if (!STATES && c > 0) bar_sync(kOutFree + group, T::kGroupThreads);
            float x[4][4];
            float2 inv;
            times_tokens<D, NP>(x, w, inv, ks, ex.part, half, lane, pair,
                                [&](int kt, const uint32_t(&hi)[4], const uint32_t(&lo)[4]) {
                                    if constexpr (!STATES) {
                                        ex.w[0][half * (D / 32) + kt][lane] = as_uint4(hi);
                                        if constexpr (YP == 2) ex.w[YP - 1][half * (D / 32) + kt][lane] = as_uint4(lo);
                                    }
                                });
            if constexpr (!STATES) ex.w_inv[half][lane] = inv;
            // X^T = V^T - gamma W0 K^T (row: value, column: token) of the own 32 tokens, and beta X
            float r[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int tok = tok0 + 8 * t + col2;
                const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok);
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok);
                const float* v0 = vs + tok * S::kVLd;
                x[t][0] = v0[0] - gm.x * k_inv * x[t][0];
                x[t][1] = v0[S::kVLd] - gm.y * k_inv * x[t][1];
                x[t][2] = v0[8] - gm.x * k_inv * x[t][2];
                x[t][3] = v0[S::kVLd + 8] - gm.y * k_inv * x[t][3];
                r[t][0] = bt.x * x[t][0], r[t][1] = bt.y * x[t][1];
                r[t][2] = bt.x * x[t][2], r[t][3] = bt.y * x[t][3];
            }
            // eps^T = X^T - (beta X)^T N^T: the own tokens' beta X, and for the second half the first half's
            {
                uint32_t hi[2][4], lo[2][4];
                uint4(&other)[4][32] = reinterpret_cast<uint4(&)[4][32]>(ex.part[1]);
                float2 r_inv;
                share(r, hi, lo, r_inv, other, ex.inv, lane, half == 0);
                float i0 = r_inv.x, i1 = r_inv.y;
                auto own = [&](uint32_t(&f)[4], int j, int k, int e) {
                    frag_b<kC>(f, ns + e * kC * kC * 2, tok0 + j * 16, tok0 + k * 16, lane);
                };
                float acc[4][4] = {};
                mma_row<2, 2, 0, 2>(acc, hi[0], lo[0], [&](uint32_t(&f)[4], int j, int e) { own(f, j, 0, e); });
                mma_row<2, 2, 1, 2>(acc, hi[1], lo[1], [&](uint32_t(&f)[4], int j, int e) { own(f, j, 1, e); });
                i0 *= n_inv, i1 *= n_inv;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    x[t][0] = fmaf(-acc[t][0], i0, x[t][0]), x[t][1] = fmaf(-acc[t][1], i0, x[t][1]);
                    x[t][2] = fmaf(-acc[t][2], i1, x[t][2]), x[t][3] = fmaf(-acc[t][3], i1, x[t][3]);
                }
                pair();
                if (half == 1) {
                    shared_by(hi, lo, r_inv, other, ex.inv, lane);
                    i0 = r_inv.x * n_inv, i1 = r_inv.y * n_inv;
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
                        mma_row<2, 2, 0, 2>(acc, hi[kt], lo[kt], [&](uint32_t(&f)[4], int j, int e) {
                            frag_b<kC>(f, ns + e * kC * kC * 2, 32 + j * 16, kt * 16, lane);
                        });
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        x[t][0] = fmaf(-acc[t][0], i0, x[t][0]), x[t][1] = fmaf(-acc[t][1], i0, x[t][1]);
                        x[t][2] = fmaf(-acc[t][2], i1, x[t][2]), x[t][3] = fmaf(-acc[t][3], i1, x[t][3]);
                    }
                }
            }
            if constexpr (STATES) {
                float* o = st.eps + ((unit * chunks + c) * kC + tok0) * D + row;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[(long)(8 * t + col2 + (e & 1)) * D + (e >> 1) * 8] = x[t][e];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {  // E = beta eps, then l E
                const float2 bt = *reinterpret_cast<const float2*>(s.beta + tok0 + 8 * t + col2);
                const float2 l = *reinterpret_cast<const float2*>(s.rest + tok0 + 8 * t + col2);
                x[t][0] *= bt.x, x[t][1] *= bt.y, x[t][2] *= bt.x, x[t][3] *= bt.y;
                r[t][0] = l.x * x[t][0], r[t][1] = l.y * x[t][1], r[t][2] = l.x * x[t][2], r[t][3] = l.y * x[t][3];
            }
            if constexpr (!STATES) {
                float top0, top1, i0, i1;
                row_tops<4>(x, top0, top1);
                const float s0 = pow2_scale(top0, i0), s1 = pow2_scale(top1, i1);
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    uint32_t hi[4], lo[4];
                    split_a<4>(x, kt, s0, s1, hi, lo);
                    ex.e[0][2 * half + kt][lane] = as_uint4(hi);
                    if constexpr (YP == 2) ex.e[YP - 1][2 * half + kt][lane] = as_uint4(lo);
                }
                ex.e_inv[half][lane] = make_float2(i0, i1);
                bar_arrive(kOutFull + group, T::kGroupThreads);
            }
            // W = gamma_C W + (l E)^T K
            add_outer_both<D, NP>(w, s.gamma[kC - 1], r, k_inv, ex.outer, ex.outer_inv, ks, half, lane, pair);
            if (c + 2 < used) bar_arrive(kFree + (c & 1), kThreads);
        }
        if constexpr (!STATES) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                *reinterpret_cast<float2*>(W + 8 * i) = make_float2(w[i][0], w[i][1]);
                *reinterpret_cast<float2*>(W + 8 * D + 8 * i) = make_float2(w[i][2], w[i][3]);
            }
        }
        }
    } else if constexpr (!STATES) {  // ---------------------------------- y of sixteen rows, 32 tokens a warp
        if constexpr (T::kShift) registers_down<T::kOutRegs>();
        const int group = (warp - T::kChain) >> 1, half = (warp - T::kChain) & 1, tok0 = 32 * half;
        const Exchange<D, YP>& ex = exchanges[group];
        for (int c = 0; c < used; ++c) {
            S& s = stages[c & 1];
            bar_sync(kFull + (c & 1), kThreads);
            bar_sync(kOutFull + group, T::kGroupThreads);
            const uint32_t qs = smem_u32(s.q), ps = smem_u32(s.p);
            const float q_inv = s.scal[3], p_inv = s.scal[5];
            constexpr int kParts = T::kPerGroup;  // of the columns and of the tokens, with scales of their own
            float y[4][4] = {}, acc[4][4] = {};
            auto fragments = [&](const uint4(&from)[32], const uint4(&second)[32], uint32_t(&hi)[4], uint32_t(&lo)[4]) {
                from_uint4(hi, from[lane]);
                if constexpr (YP == 2) from_uint4(lo, second[lane]);
            };
            auto take = [&](float f0, float f1) {  // y += acc, scaled back
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    y[t][0] = fmaf(acc[t][0], f0, y[t][0]), y[t][1] = fmaf(acc[t][1], f0, y[t][1]);
                    y[t][2] = fmaf(acc[t][2], f1, y[t][2]), y[t][3] = fmaf(acc[t][3], f1, y[t][3]);
                    acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
                }
            };
            // gamma W0 Q^T
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
#pragma unroll
                for (int i = 0; i < D / 16 / kParts; ++i) {
                    const int kt = part * (D / 16 / kParts) + i;
                    uint32_t hi[4], lo[4];
                    fragments(ex.w[0][kt], ex.w[YP - 1][kt], hi, lo);
                    mma_row<YP, NP, 0, 2>(acc, hi, lo, [&](uint32_t(&f)[4], int j, int e) {
                        frag_b<D>(f, qs + e * kC * D * 2, tok0 + j * 16, kt * 16, lane);
                    });
                }
                const float2 inv = ex.w_inv[part][lane];
                take(inv.x, inv.y);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 gm = *reinterpret_cast<const float2*>(s.gamma + tok0 + 8 * t + col2);
                y[t][0] *= gm.x * q_inv, y[t][1] *= gm.y * q_inv, y[t][2] *= gm.x * q_inv, y[t][3] *= gm.y * q_inv;
            }
            // + E^T P^T; token j shows in the tokens from its block of 16 on
            unrolled<4>([&](auto kt) {
                if (kt < 2 || half) {
                    uint32_t hi[4], lo[4];
                    fragments(ex.e[0][kt], ex.e[YP - 1][kt], hi, lo);
                    auto from = [&](uint32_t(&f)[4], int j, int e) {
                        frag_b<kC>(f, ps + e * kC * kC * 2, tok0 + j * 16, kt * 16, lane);
                    };
                    if (kt == (half ? 3 : 1))
                        mma_row<YP, YP, 1, 2>(acc, hi, lo, from);
                    else
                        mma_row<YP, YP, 0, 2>(acc, hi, lo, from);
                }
                if (kt == 3 || (kParts == 2 && kt == 1)) {
                    const float2 inv = ex.e_inv[kParts == 2 && kt == 3][lane];
                    take(inv.x * p_inv, inv.y * p_inv);
                }
            });
            if (c + 1 < used) bar_arrive(kOutFree + group, T::kGroupThreads);
            // Into V's place, which the chain has read, and out from there: two lanes a token, 32 or 64 bytes of its row
            float* vs = s.v + tok0 * S::kVLd + group * 16;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float* v0 = vs + (lane >> 2) + (8 * t + col2) * S::kVLd;
                v0[0] = y[t][0], v0[S::kVLd] = y[t][1], v0[8] = y[t][2], v0[S::kVLd + 8] = y[t][3];
            }
            __syncwarp();
            const long t0 = (long)c * kC + tok0;
            const int n = (int)min(32L, len - t0);
            const long at = (unit * a.T + t0) * D + row_base + group * 16 + (lane & 1) * 8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = i * 16 + (lane >> 1);
                if (tok >= n) continue;
                float o[8];
                load8(vs + tok * S::kVLd + (lane & 1) * 8, o);
                if (a.attn) {
                    float g[8];
                    load8(static_cast<const Tok*>(a.attn) + at + (long)tok * D, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = g[j] / (1.f + expf(-o[j]));
                }
                store8(static_cast<Tok*>(a.y) + at + (long)tok * D, o);
            }
            if (c + 2 < used) bar_arrive(kFree + (c & 1), kThreads);
        }
    }
    if constexpr (!STATES) {  // nothing is read behind the sequence's end
        const float zero[8] = {};
        for (long i = tid; i < (a.T - len) * (RW / 8); i += kThreads)
            store8(static_cast<Tok*>(a.y) + (unit * a.T + len + i / (RW / 8)) * D + row_base + i % (RW / 8) * 8, zero);
    }
}

template <int D, int RW, typename Tok, bool STATES, int YP>
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaStates& states, cudaStream_t st) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1;
    constexpr size_t bytes = 2 * sizeof(Stage<D, RW, NP, YP>) + RW / 16 * sizeof(Exchange<D, YP>);
    static_assert(bytes <= 227 * 1024, "two stages and the exchanges fit an SM");
    auto* kernel = delta_chunks_kernel<D, RW, Tok, STATES, YP>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    using T = Warps<D, RW, NP, STATES>;
    if constexpr (T::kShift) {  // the shares are paid for by what the launch gives
        static const bool enough = [&] {
            cudaFuncAttributes f;
            return cudaFuncGetAttributes(&f, kernel) == cudaSuccess && f.numRegs * T::kThreads >= T::kShares;
        }();
        if (!enough) return cudaErrorInvalidConfiguration;
    }
    kernel<<<(unsigned)((long)a.B * a.H * (D / RW)), T::kThreads, bytes, st>>>(
        a, static_cast<const DeltaChunk*>(recs), (int)((a.T + kC - 1) / kC), states);
    return cudaGetLastError();
}

// Rows of a CTA: as many as shared memory and the barriers have room for, but 32 at d = 128, where 64 would leave most SMs without a
// CTA at the 32 units of a wide memory's batch. That does not go by the units that a call has: from 38 on, 32 rows take a second round
// of CTAs (4096 tokens: 37 units 252 us, 38 units 422 us, 64 units 466 us; backward 0.86, 1.23 and 1.56 ms).
template <bool STATES, int YP>  // YP: in bf16; fp32 has two pieces of everything
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaStates& s, cudaStream_t st) {
    if (a.d == 64)
        return a.bf16 ? launch<64, 64, __nv_bfloat16, STATES, YP>(a, recs, s, st) : launch<64, 32, float, STATES, 2>(a, recs, s, st);
    return a.bf16 ? launch<128, 32, __nv_bfloat16, STATES, YP>(a, recs, s, st) : launch<128, 16, float, STATES, 2>(a, recs, s, st);
}

}  // namespace

cudaError_t launch_delta_chunks(const DeltaArgs& a, const void* chunks, const DeltaStates* states, cudaStream_t st) {
    if (states) return launch<true, 1>(a, chunks, *states, st);
    return delta_y_pieces(a) == 2 ? launch<false, 2>(a, chunks, DeltaStates{}, st) : launch<false, 1>(a, chunks, DeltaStates{}, st);
}

}  // namespace titans
