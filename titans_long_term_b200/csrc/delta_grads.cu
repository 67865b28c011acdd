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
// and dg is the sum of dG from the token to the chunk's end (to the next decay of 0, where one comes before that). That needs the products above to fp32's
// precision also where dk and dq are rounded to bf16: all run on fp16 pieces of 22 bits.
//
// One CTA per (key head, chunk) goes through the value heads that share the key head and adds up their dq and dk in
// registers, in a fixed order. A warp has 32 tokens and 16 columns of dk and dq. Everything a product reads lies in shared memory
// as fp16 pieces, the two states one after the other and 64 rows at a time; each is read from memory twice, first for
// its largest value and <A, W0> (W0 kept in registers between the two saves 0.8 % and spills more than the 104 to 260 bytes a
// thread that the 128 registers leave no room for as it is).
// 8192 chunks of d = 64: 561 us, 1.5 TB/s of HBM; the L1 data path is 60 % busy and the issue slots 33 %, with the 16 warps that its 109 KB and 128
// registers a thread leave: phases of loads, products and barriers, of which two CTAs hide one another's.
#include "delta_common.cuh"

namespace titans {
namespace {

template <int D, int NP>
struct Shared {
    static constexpr int kGroups = D / 16, kWarps = 2 * kGroups;  // column groups; two halves of the tokens each
    __half k[NP][kC * D], q[NP][kC * D], dy[NP][kC * D];
    __half e[2][kC * D], f[2][kC * D];
    __half dp[2][kC * kC], dm[2][kC * kC];
    union {
        __half w[2][kC * D];          // 64 rows of W0 or A
        float part[kGroups][kC];      // dG of a group's columns
    };
    float gamma[kC], rest[kC], ghi[kC], glo[kC];
    int zeros[kC];
    float from[kC], to[3][48];
    float sums[kWarps];               // <A, W0>, then dG_C's other part
    float tops[6][kWarps];
};

// Row of the i-th of ten lower blocks, which go row by row.
__device__ __forceinline__ int block_row(int i) { return (i >= 1) + (i >= 3) + (i >= 6); }

template <int WARPS>
__device__ __forceinline__ float max_of(const float* x) {
    float t = x[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) t = fmaxf(t, x[i]);
    return t;
}

// Four values as floats in memory, and as pieces in a [rows][D] tile: the i-th four of its values lie at quad_at.
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}
template <int D>
__device__ __forceinline__ uint32_t quad_at(int i) {
    return swz<D>(i / (D / 4), i % (D / 4) >> 1) + (i & 1) * 8;
}
__device__ __forceinline__ void put4(uint32_t addr, uint32_t lo_offset, const float (&x)[4], float s) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) split2(x[2 * i] * s, x[2 * i + 1] * s, h[i], l[i]);
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(addr), "r"(h[0]), "r"(h[1]) : "memory");
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(addr + lo_offset), "r"(l[0]), "r"(l[1]) : "memory");
}

// a += A B for this warp's 32 tokens of the tile at `left` (NA pieces of [64][LD], 16 steps of k from column k0 on) and its 16 columns of the
// two-piece tile [64][D] at `right`, rows = k.
template <int D, int NA>
__device__ __forceinline__ void times_rows(float (&t)[2][2][4], uint32_t left, int k0, uint32_t right, int m0, int n0, int lane) {
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        uint32_t hi[4], lo[4];
        frag_bt<D>(hi, right, n0, kt * 16, lane);
        frag_bt<D>(lo, right + kC * D * 2, n0, kt * 16, lane);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t x[NA][4];
#pragma unroll
            for (int e = 0; e < NA; ++e) frag_a<D>(x[e], left + e * kC * D * 2, m0 + m * 16, k0 + kt * 16, lane);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint32_t b[2][2] = {{hi[2 * n], hi[2 * n + 1]}, {lo[2 * n], lo[2 * n + 1]}};
                mma_all<NA, 2>(t[m][n], x, b);
            }
        }
    }
}
// t += S B (TRANS: S^T B) for a lower triangular two-piece tile S [64][64] and the tile B [64][D] of NB pieces.
template <int D, int NB, bool TRANS>
__device__ __forceinline__ void times_tokens(float (&t)[2][2][4], uint32_t s, uint32_t tile, int m0, int n0, int lane) {
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        if (TRANS ? kt * 16 < m0 : kt * 16 > m0 + 16) continue;
        uint32_t f[NB][4];
#pragma unroll
        for (int e = 0; e < NB; ++e) frag_bt<D>(f[e], tile + e * kC * D * 2, n0, kt * 16, lane);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (TRANS ? kt * 16 < m0 + m * 16 : kt * 16 > m0 + m * 16) continue;
            uint32_t x[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (TRANS)
                    frag_at<kC>(x[e], s + e * kC * kC * 2, m0 + m * 16, kt * 16, lane);
                else
                    frag_a<kC>(x[e], s + e * kC * kC * 2, m0 + m * 16, kt * 16, lane);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t b[NB][2];
#pragma unroll
                for (int e = 0; e < NB; ++e) b[e][0] = f[e][2 * n], b[e][1] = f[e][2 * n + 1];
                mma_all<2, NB>(t[m][n], x, b);
            }
        }
    }
}

template <int D, typename Tok>
__global__ void __launch_bounds__(D * 4, D == 64 ? 2 : 1)
    delta_grads_kernel(DeltaArgs a, const DeltaChunk* recs, int chunks, DeltaGrads g) {
    constexpr int NP = sizeof(Tok) == 4 ? 2 : 1, kThreads = D * 4, NC = D / 8, VEC = kC * D / 8 / kThreads, QUADS = 2 * VEC;  // VEC = 2
    constexpr int VW = D * D / 8 / kThreads;  // blocks of eight values of a state a thread
    using S = Shared<D, NP>;
    constexpr int kWarps = S::kWarps;
    extern __shared__ __align__(1024) unsigned char smem[];
    S& s = *reinterpret_cast<S*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, col2 = 2 * (lane & 3);
    const int m0 = (warp & 1) * 32, group = warp >> 1, n0 = group * 16;
    const long key_head = blockIdx.x / chunks, b = key_head / a.Hk;
    const int chunk = (int)(blockIdx.x % chunks), heads = a.H / a.Hk;
    const long t0 = (long)chunk * kC, len = delta_length(a, b);
    const int rows = (int)min((long)kC, a.T - t0), n = (int)max(0L, min((long)kC, len - t0));  // tokens there, tokens that count
    const long tok0 = key_head * a.T + t0;
    Tok* dk = static_cast<Tok*>(g.dk) + tok0 * D;
    Tok* dq = static_cast<Tok*>(g.dq) + tok0 * D;
    const long unit0 = b * a.H + (key_head % a.Hk) * heads;
    if (n == 0) {  // behind the sequence's end: zeros
        const float zero[8] = {};
        for (int i = tid; i < rows * NC; i += kThreads) store8(dk + i * 8, zero), store8(dq + i * 8, zero);
        for (int h = 0; h < heads; ++h) {
            const long at = (unit0 + h) * a.T + t0;
            for (int i = tid; i < rows * NC; i += kThreads) store8(static_cast<Tok*>(g.dv) + at * D + i * 8, zero);
            for (int i = tid; i < rows; i += kThreads) g.dg[at + i] = g.dbeta[at + i] = 0.f;
        }
        return;
    }
    const uint32_t ks = smem_u32(s.k), qs = smem_u32(s.q), ys = smem_u32(s.dy), es = smem_u32(s.e), fs = smem_u32(s.f),
                   dps = smem_u32(s.dp), dms = smem_u32(s.dm), ws = smem_u32(s.w);
    constexpr uint32_t kTile = kC * D * 2;
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
    float dq_sum[2][2][4] = {}, dk_sum[2][2][4] = {};
    // Values of K or Q at this lane's places
    auto tokens = [&](const __half* tile, float inv, float(&x)[2][2][4]) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = swz<D>(m0 + m * 16 + (lane >> 2) + h * 8, (n0 >> 3) + j) / 2 + col2;
                    float2 v = __half22float2(*reinterpret_cast<const __half2*>(tile + at));
                    if constexpr (NP == 2) {
                        const float2 l = __half22float2(*reinterpret_cast<const __half2*>(tile + kC * D + at));
                        v.x += l.x, v.y += l.y;
                    }
                    x[m][j][2 * h] = v.x * inv, x[m][j][2 * h + 1] = v.y * inv;
                }
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) f(m, j, e);
    };

    for (int h = 0; h < heads; ++h) {
        const long unit = unit0 + h, rec = unit * chunks + chunk, tok = unit * a.T + t0;
        const DeltaChunk& r = recs[rec];
        const float *w0 = g.fwd.states + rec * D * D, *adj = g.adj + rec * D * D;
        __syncthreads();  // the last head's tiles are no longer read
        if (tid < kC) {
            s.gamma[tid] = r.gamma[tid], s.rest[tid] = r.rest[tid], s.from[tid] = r.from[tid];
            s.ghi[tid] = r.ghi[tid], s.glo[tid] = r.glo[tid], s.zeros[tid] = r.zeros[tid];
        }
        if (tid < 144) (&s.to[0][0])[tid] = (&r.to[0][0])[tid];
        float y_inv, e_inv, f_inv, w_inv, a_inv, sw, sa, inner;
        {  // dY, E and F as pieces; dV and dbeta on the way; the states' largest values and <A, W0>
            // Floats are read four a lane, so that a warp's load is one run; tokens in mode bf16 stay raw until they are scaled
            Block8<Tok> y[VEC];
            float e[QUADS][4], f[QUADS][4], top[5] = {}, dot_wa = 0.f;
#pragma unroll
            for (int i = 0; i < QUADS; ++i) {
                const long at = rec * kC * D + (long)(i * kThreads + tid) * 4;
                load4(g.fwd.eps + at, e[i]);
                load4(g.dr + at, f[i]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid;
                if (block / NC < n)
                    y[i].load(static_cast<const Tok*>(g.dy) + tok * D + (long)block * 8);
                else
                    y[i].clear();
            }
#pragma unroll
            for (int i = 0; i < 2 * VW; ++i) {
                float x[4], z[4];
                load4(w0 + (long)(i * kThreads + tid) * 4, x);
                load4(adj + (long)(i * kThreads + tid) * 4, z);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    top[3] = fmaxf(top[3], fabsf(x[j])), top[4] = fmaxf(top[4], fabsf(z[j]));
                    dot_wa = fmaf(x[j], z[j], dot_wa);
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float x[8];
                y[i].get(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) top[0] = fmaxf(top[0], fabsf(x[j]));
            }
#pragma unroll
            for (int i = 0; i < QUADS; ++i) {
                const int quad = i * kThreads + tid, row = quad / (D / 4);
                float dot = 0.f;
                const float beta = r.beta[row];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dot = fmaf(e[i][j], f[i][j], dot);
                    e[i][j] *= beta, f[i][j] *= beta;
                    top[1] = fmaxf(top[1], fabsf(e[i][j]));
                    top[2] = fmaxf(top[2], fabsf(f[i][j]));
                }
#pragma unroll
                for (int d = D / 8; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
                if (row < rows) {
                    if (quad % (D / 4) == 0) g.dbeta[tok + row] = row < n ? dot : 0.f;
                    store4(static_cast<Tok*>(g.dv) + tok * D + (long)quad * 4, f[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                top[i] = warp_max(top[i]);
                if (lane == 0) s.tops[i][warp] = top[i];
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) dot_wa += __shfl_xor_sync(0xffffffffu, dot_wa, d);
            if (lane == 0) s.sums[warp] = dot_wa;
            __syncthreads();
            const float sy = pow2_scale(max_of<kWarps>(s.tops[0]), y_inv);
            const float se = pow2_scale(max_of<kWarps>(s.tops[1]), e_inv);
            const float sf = pow2_scale(max_of<kWarps>(s.tops[2]), f_inv);
            sw = pow2_scale(max_of<kWarps>(s.tops[3]), w_inv), sa = pow2_scale(max_of<kWarps>(s.tops[4]), a_inv);
            inner = 0.f;
            for (int i = 0; i < kWarps; ++i) inner += s.sums[i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid;
                float x[8];
                y[i].get(x);
                put8<NP>(ys + swz<D>(block / NC, block % NC), kTile, x, sy);
            }
#pragma unroll
            for (int i = 0; i < QUADS; ++i) {
                const uint32_t at = quad_at<D>(i * kThreads + tid);
                put4(es + at, kTile, e[i], se);
                put4(fs + at, kTile, f[i], sf);
            }
        }
        // 64 rows of a state into the tile w
        auto stage_state = [&](const float* src, int row0, float sc) {
#pragma unroll
            for (int i = 0; i < QUADS; ++i) {
                float x[4];
                load4(src + (long)row0 * D + (long)(i * kThreads + tid) * 4, x);
                put4(ws + quad_at<D>(i * kThreads + tid), kTile, x, sc);
            }
        };
        stage_state(w0, 0, sw);
        __syncthreads();
        float dp_inv, dm_inv;
        {  // the ten lower 16 x 16 blocks of dP (warps w with w & 4 = 0) and of dM, shared out over their warps
            constexpr int kTeam = kWarps / 2, kMost = (10 + kTeam - 1) / kTeam;
            const bool second = warp & 4;
            const int member = (warp & 3) + (warp >> 3) * 4;
            float t[kMost][2][4] = {}, top = 0.f;
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                const int at = member + i * kTeam, br = block_row(at), bc = at - br * (br + 1) / 2;
                if (at >= 10) continue;
#pragma unroll 4
                for (int kt = 0; kt < D / 16; ++kt) {
                    uint32_t x[2][4], hi[4], lo[4];
                    frag_a<D>(x[0], second ? fs : ys, br * 16, kt * 16, lane);
                    if (NP == 2 || second) frag_a<D>(x[1], (second ? fs : ys) + kTile, br * 16, kt * 16, lane);
                    frag_b<D>(hi, es, bc * 16, kt * 16, lane);
                    frag_b<D>(lo, es + kTile, bc * 16, kt * 16, lane);
#pragma unroll
                    for (int q = 0; q < 2; ++q) mma16816(t[i][q], x[0], hi[2 * q], hi[2 * q + 1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) mma16816(t[i][q], x[0], lo[2 * q], lo[2 * q + 1]);
                    if (NP == 2 || second)
#pragma unroll
                        for (int q = 0; q < 2; ++q) mma16816(t[i][q], x[1], hi[2 * q], hi[2 * q + 1]);
                }
                const float inv = e_inv * (second ? -f_inv : y_inv);
                const int row = br * 16 + (lane >> 2);
                if (bc < br) {
                    const float f0 = s.from[row] * inv, f1 = s.from[row + 8] * inv;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float2 to = *reinterpret_cast<const float2*>(&s.to[br - 1][bc * 16 + 8 * q + col2]);
                        t[i][q][0] *= f0 * to.x, t[i][q][1] *= f0 * to.y, t[i][q][2] *= f1 * to.x, t[i][q][3] *= f1 * to.y;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int rr = row + (e >> 1) * 8, cc = bc * 16 + 8 * q + col2 + (e & 1);
                            t[i][q][e] *= (second ? cc < rr : cc <= rr) ? inv * decay_between(s.ghi, s.glo, s.zeros, rr, cc) : 0.f;
                        }
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(t[i][q][e]));
            }
            top = warp_max(top);
            if (lane == 0) s.tops[5][warp] = top;
            __syncthreads();
            float tp = 0.f, tm = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                if (i & 4)
                    tm = fmaxf(tm, s.tops[5][i]);
                else
                    tp = fmaxf(tp, s.tops[5][i]);
            }
            const float sp = pow2_scale(tp, dp_inv), sm = pow2_scale(tm, dm_inv), sc = second ? sm : sp;
            unsigned char* dst = reinterpret_cast<unsigned char*>(second ? s.dm : s.dp);
#pragma unroll
            for (int i = 0; i < kMost; ++i) {  // the upper blocks are not read
                const int at = member + i * kTeam, br = block_row(at), bc = at - br * (br + 1) / 2;
                if (at >= 10) continue;
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t hi, lo;
                        split2(t[i][q][2 * h] * sc, t[i][q][2 * h + 1] * sc, hi, lo);
                        const uint32_t to = swz<kC>(br * 16 + (lane >> 2) + h * 8, bc * 2 + q) + (lane & 3) * 4;
                        *reinterpret_cast<uint32_t*>(dst + to) = hi;
                        *reinterpret_cast<uint32_t*>(dst + kC * kC * 2 + to) = lo;
                    }
            }
        }
        __syncthreads();
        float dG[2][2] = {};  // of rows m0 + 16 m + lane / 4, + 8
        auto by_row = [&](const float* x, int m, int e) { return x[m0 + m * 16 + (lane >> 2) + (e >> 1) * 8]; };
        float u[2][2][4] = {};
        {  // dQ = gamma dY W0 + dP K, and the reading role of k: u = -gamma F W0 + dM K
            float t[2][2][4] = {}, acc[2][2][4] = {}, x[2][2][4];
#pragma unroll
            for (int part = 0; part < D / 64; ++part) {
                if (part > 0) {
                    __syncthreads();
                    stage_state(w0, part * 64, sw);
                    __syncthreads();
                }
                times_rows<D, NP>(t, ys, part * 64, ws, m0, n0, lane);
                times_rows<D, 2>(u, fs, part * 64, ws, m0, n0, lane);
            }
            times_tokens<D, NP, false>(acc, dps, ks, m0, n0, lane);
            tokens(s.q[0], q_inv, x);
            each([&](int m, int j, int e) {
                const float v = fmaf(t[m][j][e], by_row(s.gamma, m, e) * (y_inv * w_inv), acc[m][j][e] * (dp_inv * k_inv));
                dq_sum[m][j][e] += v;
                dG[m][e >> 1] = fmaf(v, x[m][j][e], dG[m][e >> 1]);
                acc[m][j][e] = 0.f;
            });
            times_tokens<D, NP, false>(acc, dms, ks, m0, n0, lane);
            each([&](int m, int j, int e) {
                u[m][j][e] = fmaf(u[m][j][e], by_row(s.gamma, m, e) * (-f_inv * w_inv), acc[m][j][e] * (dm_inv * k_inv));
            });
        }
        float end = 0.f;
        {  // the writing role of k: v = l E A + dP^T Q + dM^T K
            float v[2][2][4] = {}, acc[2][2][4] = {}, x[2][2][4];
#pragma unroll
            for (int part = 0; part < D / 64; ++part) {
                __syncthreads();
                stage_state(adj, part * 64, sa);
                __syncthreads();
                times_rows<D, 2>(v, es, part * 64, ws, m0, n0, lane);
            }
            tokens(s.k[0], k_inv, x);
            times_tokens<D, NP, true>(acc, dps, qs, m0, n0, lane);
            each([&](int m, int j, int e) {
                v[m][j][e] *= by_row(s.rest, m, e) * (e_inv * a_inv);
                end = fmaf(v[m][j][e], x[m][j][e], end);
                v[m][j][e] = fmaf(acc[m][j][e], dp_inv * q_inv, v[m][j][e]);
                acc[m][j][e] = 0.f;
            });
            times_tokens<D, NP, true>(acc, dms, ks, m0, n0, lane);
            each([&](int m, int j, int e) {
                const float z = fmaf(acc[m][j][e], dm_inv * k_inv, v[m][j][e]);
                dk_sum[m][j][e] += u[m][j][e] + z;
                dG[m][e >> 1] = fmaf(u[m][j][e] - z, x[m][j][e], dG[m][e >> 1]);
            });
        }
        __syncthreads();  // w is free: part takes its place
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x = dG[m][q];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if ((lane & 3) == 0) s.part[group][m0 + m * 16 + (lane >> 2) + q * 8] = x;
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) end += __shfl_xor_sync(0xffffffffu, end, d);
        if (lane == 0) s.sums[warp] = end;
        __syncthreads();
        if (warp == 0) {  // dg_t: the sum of dG from t on, taken from the end, two tokens a lane
            double x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = kC - 1 - (2 * lane + i);
                x[i] = 0.;
#pragma unroll
                for (int w = 0; w < S::kGroups; ++w) x[i] += s.part[w][t];
                if (t == kC - 1) {
                    x[i] += (double)inner * s.gamma[kC - 1];
                    for (int w = 0; w < kWarps; ++w) x[i] += s.sums[w];
                }
            }
            const double sum = warp_prefix(x[0] + x[1], lane), all[2] = {sum - x[1], sum};
            // Nothing flows through a decay of 0: the sum from such a token on is 0, so it gets none and the tokens before it
            // take theirs without it
            bool cut[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = kC - 1 - (2 * lane + i);
                cut[i] = s.zeros[t] != (t > 0 ? s.zeros[t - 1] : 0);
            }
            const uint32_t later = __ballot_sync(0xffffffffu, cut[0] || cut[1]) & ((1u << lane) - 1);
            const double nearest = __shfl_sync(0xffffffffu, cut[1] ? all[1] : all[0], later ? 31 - __clz(later) : 0);
            const double behind = later ? nearest : 0.;
            const double dg[2] = {cut[0] ? 0. : all[0] - behind, cut[1] ? 0. : all[1] - (cut[0] ? all[0] : behind)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = kC - 1 - (2 * lane + i);
                if (t < rows) g.dg[tok + t] = t < n ? (float)dg[i] : 0.f;
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = m0 + m * 16 + (lane >> 2) + q * 8;
            if (row >= rows) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
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
    kernel<<<(unsigned)((long)a.B * a.Hk * chunks), D * 4, bytes, st>>>(a, static_cast<const DeltaChunk*>(recs), chunks, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaArgs& a, const void* chunks, const DeltaGrads& g, cudaStream_t st) {
    if (a.d == 64) return a.bf16 ? launch<64, __nv_bfloat16>(a, chunks, g, st) : launch<64, float>(a, chunks, g, st);
    return a.bf16 ? launch<128, __nv_bfloat16>(a, chunks, g, st) : launch<128, float>(a, chunks, g, st);
}

}  // namespace titans
