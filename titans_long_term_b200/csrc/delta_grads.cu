// Gated delta rule, backward: the gradients of a chunk's tokens, from its start state W0, the adjoint A of its final
// state, its residuals eps and dR (delta_common.cuh, delta_adjoint.cu):
//   E = beta eps, F = beta dR;  dV = F;  dbeta = rowdot(dR, eps)
//   dP = lower(dY E^T) o D,  dM = -strictly lower(F E^T) o D
//   dQ  = gamma dY W0 + dP K
//   dKq = -gamma F W0 + dM K          (k in its role of reading the state)
//   dKk = l E A + dP^T Q + dM^T K     (k in its role of writing it)
//   dK  = dKq + dKk
// A token enters with the factor exp(G_i) where it reads and exp(-G_i) where it writes, so
//   dG_i = q_i.dQ_i + k_i.dKq_i - k_i.dKk_i,  dG_C += sum_j k_j.(l E A)_j + gamma_C <A, W0>,
// and dg is the sum of dG from the token to the chunk's end. That needs the products above to fp32's
// precision also where dk and dq are rounded to bf16: all run on fp16 pieces of 22 bits.
//
// One CTA per (key head, chunk) goes through the value heads that share the key head and adds up their dq and dk in
// registers, in a fixed order. A warp has D/8 columns of dk and dq for all 64 tokens, so that each element of W0
// and A is loaded by one lane of one warp, straight into the B fragment it belongs to.
#include "delta_common.cuh"

namespace titans {
namespace {

constexpr int kThreads = 256;

template <int D, int NP>
struct Shared {
    __half k[NP][kC * D], q[NP][kC * D], dy[NP][kC * D];
    __half e[2][kC * D], f[2][kC * D];
    __half dp[2][kC * kC], dm[2][kC * kC];
    float gamma[kC], rest[kC], beta[kC], ghi[kC], glo[kC];
    int zeros[kC];
    float part[8][kC];  // dG of a warp's columns
    float end[8];       // its share of dG_C
    float tops[4][8];
};

// Largest of a value over the CTA; `slot` of the four in turn so that one call's reads need no barrier of their own
// before the next call's writes.
__device__ __forceinline__ float block_max(float x, float (&slot)[8], int warp, int lane) {
    x = warp_max(x);
    if (lane == 0) slot[warp] = x;
    __syncthreads();
    float t = slot[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) t = fmaxf(t, slot[i]);
    return t;
}

// t (4 x NT tiles of 16 tokens x 8 columns) = rows of A, a tile in shared memory, times B fragments in registers.
template <int D, int NA, int NT>
__device__ __forceinline__ void times_state(float (&t)[4][NT][4], uint32_t tile, const uint32_t (&b)[D / 16][NT][2][2],
                                            int lane) {
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int kt = 0; kt < D / 16; ++kt) {
            uint32_t x[NA][4];
#pragma unroll
            for (int e = 0; e < NA; ++e) frag_a<D>(x[e], tile + e * kC * D * 2, m * 16, kt * 16, lane);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_all<NA, 2>(t[m][n], x, b[kt][n]);
        }
}

// t += S B (TRANS: S^T B) for a lower triangular tile S [64][64] and the columns n0.. of a tile B [64][D].
template <int D, int NB, int NT, bool TRANS>
__device__ __forceinline__ void times_tokens(float (&t)[4][NT][4], uint32_t s, uint32_t tile, int n0, int lane) {
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        uint32_t b[NT][NB][2];
#pragma unroll
        for (int e = 0; e < NB; ++e) {
            uint32_t f[4];
            frag_bt<D>(f, tile + e * kC * D * 2, n0 & ~15, kt * 16, lane);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int at = NT == 2 ? 2 * n : (n0 & 8) >> 2;
                b[n][e][0] = at ? f[2] : f[0], b[n][e][1] = at ? f[3] : f[1];
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (TRANS ? kt < m : kt > m) continue;
            uint32_t x[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (TRANS)
                    frag_at<kC>(x[e], s + e * kC * kC * 2, m * 16, kt * 16, lane);
                else
                    frag_a<kC>(x[e], s + e * kC * kC * 2, m * 16, kt * 16, lane);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_all<2, NB>(t[m][n], x, b[n]);
        }
    }
}

template <int D, typename Tok>
__global__ void __launch_bounds__(kThreads) delta_grads_kernel(DeltaArgs a, const DeltaChunk* recs, int chunks, DeltaGrads g) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, NT = D / 64, NC = D / 8, VEC = kC * D / 8 / kThreads;
    using S = Shared<D, NP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    S& s = *reinterpret_cast<S*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n0 = warp * NC, col2 = 2 * (lane & 3);
    const long key_head = blockIdx.x / chunks, b = key_head / a.Hk;
    const int chunk = (int)(blockIdx.x % chunks), group = a.H / a.Hk;
    const long t0 = (long)chunk * kC, len = delta_length(a, b);
    const int rows = (int)min((long)kC, a.T - t0), n = (int)max(0L, min((long)kC, len - t0));  // tokens there, tokens that count
    const long tok0 = key_head * a.T + t0;
    Tok* dk = static_cast<Tok*>(g.dk) + tok0 * D;
    Tok* dq = static_cast<Tok*>(g.dq) + tok0 * D;
    const long unit0 = b * a.H + (key_head % a.Hk) * group;
    if (n == 0) {  // behind the sequence's end: zeros
        const float zero[8] = {};
        for (int i = tid; i < rows * NC; i += kThreads) store8(dk + i * 8, zero), store8(dq + i * 8, zero);
        for (int h = 0; h < group; ++h) {
            const long at = (unit0 + h) * a.T + t0;
            for (int i = tid; i < rows * NC; i += kThreads) store8(static_cast<Tok*>(g.dv) + at * D + i * 8, zero);
            for (int i = tid; i < rows; i += kThreads) g.dg[at + i] = g.dbeta[at + i] = 0.f;
        }
        return;
    }
    const uint32_t ks = smem_u32(s.k), qs = smem_u32(s.q), ys = smem_u32(s.dy), es = smem_u32(s.e), fs = smem_u32(s.f),
                   dps = smem_u32(s.dp), dms = smem_u32(s.dm);
    constexpr uint32_t kTile = kC * D * 2, kPair = kC * kC * 2;
    float k_inv, q_inv;
    {
        const DeltaChunk& r = recs[unit0 * chunks + chunk];
        const float sk = r.k_scale, sq = r.q_scale;
        k_inv = r.k_inv, q_inv = r.q_inv;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int block = i * kThreads + tid, row = block / NC;
            float x[8] = {}, z[8] = {};
            if (row < n) {
                load8(static_cast<const Tok*>(a.k) + tok0 * D + (long)block * 8, x);
                load8(static_cast<const Tok*>(a.q) + tok0 * D + (long)block * 8, z);
            }
            put8<NP>(ks + swz<D>(row, block % NC), kTile, x, sk);
            put8<NP>(qs + swz<D>(row, block % NC), kTile, z, sq);
        }
    }
    float dq_sum[4][NT][4] = {}, dk_sum[4][NT][4] = {};
    // Values of K or Q at this lane's places of row tile m and column tile j, rows +0 and +8
    auto token_at = [&](const __half* tile, float inv, int m, int j, float (&x)[4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = m * 16 + (lane >> 2) + h * 8, at = swz<D>(row, (n0 >> 3) + j) / 2 + col2;
            float2 v = __half22float2(*reinterpret_cast<const __half2*>(tile + at));
            if constexpr (NP == 2) {
                const float2 l = __half22float2(*reinterpret_cast<const __half2*>(tile + kC * D + at));
                v.x += l.x, v.y += l.y;
            }
            x[2 * h] = v.x * inv, x[2 * h + 1] = v.y * inv;
        }
    };

    for (int h = 0; h < group; ++h) {
        const long unit = unit0 + h, rec = unit * chunks + chunk, tok = unit * a.T + t0;
        const DeltaChunk& r = recs[rec];
        __syncthreads();  // the last head's tiles are no longer read
        if (tid < kC) {
            s.gamma[tid] = r.gamma[tid], s.rest[tid] = r.rest[tid], s.beta[tid] = r.beta[tid];
            s.ghi[tid] = r.ghi[tid], s.glo[tid] = r.glo[tid], s.zeros[tid] = r.zeros[tid];
        }
        float y_inv, e_inv, f_inv;
        {  // dY, E and F as pieces; dV and dbeta on the way
            float y[VEC][8], e[VEC][8], f[VEC][8], top[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid, row = block / NC;
                load8(g.fwd.eps + rec * kC * D + (long)block * 8, e[i]);
                load8(g.dr + rec * kC * D + (long)block * 8, f[i]);
                if (row < n) {
                    load8(static_cast<const Tok*>(g.dy) + tok * D + (long)block * 8, y[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[i][j] = 0.f;
                }
                float dot = 0.f;
                const float beta = r.beta[row];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dot = fmaf(e[i][j], f[i][j], dot);
                    e[i][j] *= beta, f[i][j] *= beta;
                    top[0] = fmaxf(top[0], fabsf(y[i][j]));
                    top[1] = fmaxf(top[1], fabsf(e[i][j]));
                    top[2] = fmaxf(top[2], fabsf(f[i][j]));
                }
#pragma unroll
                for (int d = NC / 2; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                if (row < rows) {
                    if (block % NC == 0) g.dbeta[tok + row] = row < n ? dot : 0.f;
                    store8(static_cast<Tok*>(g.dv) + tok * D + (long)block * 8, f[i]);
                }
            }
            const float sy = pow2_scale(block_max(top[0], s.tops[0], warp, lane), y_inv);
            const float se = pow2_scale(block_max(top[1], s.tops[1], warp, lane), e_inv);
            const float sf = pow2_scale(block_max(top[2], s.tops[2], warp, lane), f_inv);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid;
                const uint32_t at = swz<D>(block / NC, block % NC);
                put8<NP>(ys + at, kTile, y[i], sy);
                put8<2>(es + at, kTile, e[i], se);
                put8<2>(fs + at, kTile, f[i], sf);
            }
        }
        __syncthreads();
        float dp_inv, dm_inv;
        {  // warps 0..3: rows of dP; 4..7: rows of dM
            const int m0 = (warp & 3) * 16;
            const bool second = warp >= 4;
            float t[8][4] = {};
            for (int kt = 0; kt < D / 16; ++kt) {
                uint32_t x[2][4];
                if (second) {
                    frag_a<D>(x[0], fs, m0, kt * 16, lane);
                    frag_a<D>(x[1], fs + kTile, m0, kt * 16, lane);
                } else {
                    frag_a<D>(x[0], ys, m0, kt * 16, lane);
                    if constexpr (NP == 2) frag_a<D>(x[1], ys + kTile, m0, kt * 16, lane);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j * 16 > m0) continue;
                    uint32_t hi[4], lo[4];
                    frag_b<D>(hi, es, j * 16, kt * 16, lane);
                    frag_b<D>(lo, es + kTile, j * 16, kt * 16, lane);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        mma16816(t[2 * j + q], x[0], hi[2 * q], hi[2 * q + 1]);
                        mma16816(t[2 * j + q], x[0], lo[2 * q], lo[2 * q + 1]);
                        if (NP == 2 || second) mma16816(t[2 * j + q], x[1], hi[2 * q], hi[2 * q + 1]);
                    }
                }
            }
            const float inv = e_inv * (second ? -f_inv : y_inv);
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = m0 + (lane >> 2) + (e >> 1) * 8, col = 8 * j + col2 + (e & 1);
                    t[j][e] = (second ? col < row : col <= row)
                                  ? t[j][e] * inv * decay_between(s.ghi, s.glo, s.zeros, row, col)
                                  : 0.f;
                    top = fmaxf(top, fabsf(t[j][e]));
                }
            top = warp_max(top);
            if (lane == 0) s.tops[3][warp] = top;
            __syncthreads();
            const float(&w)[8] = s.tops[3];
            const float sp = pow2_scale(fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])), dp_inv);
            const float sm = pow2_scale(fmaxf(fmaxf(w[4], w[5]), fmaxf(w[6], w[7])), dm_inv);
            const float sc = second ? sm : sp;
            unsigned char* dst = reinterpret_cast<unsigned char*>(second ? s.dm : s.dp);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t hi, lo;
                    split2(t[j][2 * q] * sc, t[j][2 * q + 1] * sc, hi, lo);
                    const uint32_t at = swz<kC>(m0 + (lane >> 2) + q * 8, j) + (lane & 3) * 4;
                    *reinterpret_cast<uint32_t*>(dst + at) = hi;
                    *reinterpret_cast<uint32_t*>(dst + kPair + at) = lo;
                }
        }
        __syncthreads();
        float dG[4][2] = {};  // of rows 16 m + lane / 4, + 8
        // adds t to `sum`, and its products with the token (sign) to dG; returns their total
        auto take = [&](float(&t)[4][NT][4], float(&sum)[4][NT][4], const __half* tile, float inv, float sign) {
            float total = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float x[4];
                    token_at(tile, inv, m, j, x);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float d = t[m][j][2 * q] * x[2 * q] + t[m][j][2 * q + 1] * x[2 * q + 1];
                        dG[m][q] = fmaf(sign, d, dG[m][q]);
                        total += d;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[m][j][e] += t[m][j][e];
                }
            return total;
        };
        auto scale_rows = [&](float(&t)[4][NT][4], const float* by, float f) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float f0 = by[m * 16 + (lane >> 2)] * f, f1 = by[m * 16 + (lane >> 2) + 8] * f;
#pragma unroll
                for (int j = 0; j < NT; ++j) t[m][j][0] *= f0, t[m][j][1] *= f0, t[m][j][2] *= f1, t[m][j][3] *= f1;
            }
        };
        auto add_scaled = [&](float(&t)[4][NT][4], const float(&u)[4][NT][4], float f) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[m][j][e] = fmaf(u[m][j][e], f, t[m][j][e]);
        };
        // This lane's elements of W0 and A: rows 16 kt + 2 (lane % 4) + {0, 1, 8, 9}, columns n0 + 8 j + lane / 4
        float w0[D / 16][NT][4];
        uint32_t wb[D / 16][NT][2][2];
        float w_inv, end = 0.f;
        auto load_state = [&](const float* src, float(&x)[D / 16][NT][4]) {
            float top = 0.f;
#pragma unroll
            for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[kt][j][e] = src[(kt * 16 + col2 + (e & 1) + (e >> 1) * 8) * D + n0 + 8 * j + (lane >> 2)];
                        top = fmaxf(top, fabsf(x[kt][j][e]));
                    }
            return warp_max(top);
        };
        auto to_pieces = [&](const float(&x)[D / 16][NT][4], float sc) {
#pragma unroll
            for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        split2(x[kt][j][2 * q] * sc, x[kt][j][2 * q + 1] * sc, wb[kt][j][0][q], wb[kt][j][1][q]);
        };
        to_pieces(w0, pow2_scale(load_state(g.fwd.states + rec * D * D, w0), w_inv));
        {  // dQ = gamma dY W0 + dP K
            float t[4][NT][4] = {}, u[4][NT][4] = {};
            times_state<D, NP, NT>(t, ys, wb, lane);
            scale_rows(t, s.gamma, y_inv * w_inv);
            times_tokens<D, NP, NT, false>(u, dps, ks, n0, lane);
            add_scaled(t, u, dp_inv * k_inv);
            take(t, dq_sum, s.q[0], q_inv, 1.f);
        }
        {  // dKq = -gamma F W0 + dM K
            float t[4][NT][4] = {}, u[4][NT][4] = {};
            times_state<D, 2, NT>(t, fs, wb, lane);
            scale_rows(t, s.gamma, -f_inv * w_inv);
            times_tokens<D, NP, NT, false>(u, dms, ks, n0, lane);
            add_scaled(t, u, dm_inv * k_inv);
            take(t, dk_sum, s.k[0], k_inv, 1.f);
        }
        {  // l E A, and gamma_C <A, W0> with W0 put together again from its pieces
            float dot = 0.f;
            const float top = load_state(g.adj + rec * D * D, w0);
#pragma unroll
            for (int kt = 0; kt < D / 16; ++kt)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&wb[kt][j][0][q]));
                        const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&wb[kt][j][1][q]));
                        dot = fmaf(w0[kt][j][2 * q], (hi.x + lo.x) * w_inv, dot);
                        dot = fmaf(w0[kt][j][2 * q + 1], (hi.y + lo.y) * w_inv, dot);
                    }
            end = dot * s.gamma[kC - 1];
            to_pieces(w0, pow2_scale(top, w_inv));
            float t[4][NT][4] = {};
            times_state<D, 2, NT>(t, es, wb, lane);
            scale_rows(t, s.rest, e_inv * w_inv);
            end += take(t, dk_sum, s.k[0], k_inv, -1.f);
        }
        {  // dP^T Q + dM^T K
            float t[4][NT][4] = {}, u[4][NT][4] = {}, zero[4][NT][4] = {};
            times_tokens<D, NP, NT, true>(u, dps, qs, n0, lane);
            add_scaled(t, u, dp_inv * q_inv);
            times_tokens<D, NP, NT, true>(zero, dms, ks, n0, lane);
            add_scaled(t, zero, dm_inv * k_inv);
            take(t, dk_sum, s.k[0], k_inv, -1.f);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x = dG[m][q];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if ((lane & 3) == 0) s.part[warp][m * 16 + (lane >> 2) + q * 8] = x;
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) end += __shfl_xor_sync(0xffffffffu, end, d);
        if (lane == 0) s.end[warp] = end;
        __syncthreads();
        if (warp == 0) {  // dg_t: the sum of dG from t on, taken from the end, two tokens a lane
            double x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = kC - 1 - (2 * lane + i);
                x[i] = 0.;
#pragma unroll
                for (int w = 0; w < 8; ++w) x[i] += s.part[w][t] + (t == kC - 1 ? s.end[w] : 0.f);
            }
            const double sum = warp_prefix(x[0] + x[1], lane);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = kC - 1 - (2 * lane + i);
                if (t < rows) g.dg[tok + t] = t < n ? (float)(i ? sum : sum - x[1]) : 0.f;
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = m * 16 + (lane >> 2) + q * 8;
            if (row >= rows) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int at = row * D + n0 + 8 * j + col2;
                if constexpr (sizeof(Tok) == 4) {
                    *reinterpret_cast<float2*>(dq + at) = make_float2(dq_sum[m][j][2 * q], dq_sum[m][j][2 * q + 1]);
                    *reinterpret_cast<float2*>(dk + at) = make_float2(dk_sum[m][j][2 * q], dk_sum[m][j][2 * q + 1]);
                } else {
                    *reinterpret_cast<uint32_t*>(dq + at) = pack_bf16x2(dq_sum[m][j][2 * q], dq_sum[m][j][2 * q + 1]);
                    *reinterpret_cast<uint32_t*>(dk + at) = pack_bf16x2(dk_sum[m][j][2 * q], dk_sum[m][j][2 * q + 1]);
                }
            }
        }
}

template <int D, typename Tok>
cudaError_t launch(const DeltaArgs& a, const void* recs, const DeltaGrads& g, cudaStream_t st) {
    constexpr size_t bytes = sizeof(Shared<D, sizeof(Tok) == 4 ? 2 : 1>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    auto* kernel = delta_grads_kernel<D, Tok>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    const int chunks = (int)((a.T + kC - 1) / kC);
    kernel<<<(unsigned)((long)a.B * a.Hk * chunks), kThreads, bytes, st>>>(a, static_cast<const DeltaChunk*>(recs), chunks, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaArgs& a, const void* chunks, const DeltaGrads& g, cudaStream_t st) {
    if (a.d == 64) return a.bf16 ? launch<64, __nv_bfloat16>(a, chunks, g, st) : launch<64, float>(a, chunks, g, st);
    return a.bf16 ? launch<128, __nv_bfloat16>(a, chunks, g, st) : launch<128, float>(a, chunks, g, st);
}

}  // namespace titans
