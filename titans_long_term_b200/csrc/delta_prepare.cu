// Gated delta rule, first kernel of the chunked path: what a chunk's tokens need of one another (N, P and the
// decays; see delta_common.cuh), for every chunk of every unit at once, before the state is known.
//
// One CTA of 128 threads per (unit, chunk). K K^T and Q K^T are taken on the tensor cores, 16 rows a warp.
// N by blocks of 16 tokens: T_i, the inverse of I + M_ii beta, by forward substitution in fp32, a block a warp and a
// column a lane; then N_ic = T_i (M_ic - sum_{c <= j < i} M_ij beta N_jc), a column block c a warp, as tensor-core
// products of pieces, each beta N_jc turned from accumulator into the next products' B fragments in registers.
// Of N and P only the blocks on and below the diagonal are written, from registers, and read by anybody.
//
// Short dependent steps (the substitution, then products of 16 x 16 blocks) bound it: what hides their latency is other CTAs, so
// shared memory is kept to five of them an SM at d = 64 (M's pieces take the place of K and Q). 8192 chunks: 162 us at d = 64 and
// 214 us at d = 128, issue slots 48 % busy, 1.0 TB/s of HBM. With all of N by substitution the two kernels of 8192 chunks took 418 us
// instead of 339.
#include "delta_common.cuh"

namespace titans {
namespace {

constexpr int kThreads = 128;
constexpr float kForget = -104.f;  // exp of less is 0 in fp32 (half of its least value is exp(-103.97))

template <int D, typename Tok>
struct Shared {
    static constexpr int kPieces = sizeof(Tok) == 4 ? 2 : 1;
    __half k[kPieces][kC * D], q[kPieces][kC * D];
};
constexpr int kDiagLd = 18;
constexpr int kTPitch = 24;  // halves between rows of a 16 x 16 block of T: an ldmatrix hits all banks once
struct Common {
    alignas(16) float diag[4][16][kDiagLd];  // blocks on M's diagonal: diag[block][j][i] = M_ij
    alignas(16) __half t[4][2][16 * kTPitch];
    float t_inv[4];
    float beta[kC], ghi[kC], glo[kC];
    int zeros[kC];    // tokens of the chunk so far whose decay is 0
    float from[kC], to[3][48];  // as in DeltaChunk
    float tops[16];
};

// A 16 x 16 accumulator (two n-tiles) as the pieces of a B fragment with its rows as k: b[piece][n-tile][half of k].
__device__ __forceinline__ void to_fragment(const float (&x)[2][4], float s, uint32_t (&b)[2][2][2]) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t hi, lo;
            split2(x[n][2 * h] * s, x[n][2 * h + 1] * s, hi, lo);
            b[0][n][h] = transpose8(hi), b[1][n][h] = transpose8(lo);
        }
}
// acc += A B: hi hi, lo hi, hi lo.
__device__ __forceinline__ void multiply(float (&acc)[2][4], const uint32_t (&a)[2][4], const uint32_t (&b)[2][2][2]) {
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int n = 0; n < 2; ++n) mma16816(acc[n], a[e == 1], b[e == 2][n][0], b[e == 2][n][1]);
}
__device__ __forceinline__ float top16(const float (&x)[2][4]) {
    float t = 0.f;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) t = fmaxf(t, fabsf(x[n][e]));
    return warp_max(t);
}
// Two neighbouring values of row `row` (8 column block `block`, 2 (lane % 4) within) into a tile's pieces.
__device__ __forceinline__ void put2(void* tile, int row, int block, int lane, float x, float y, bool both = true) {
    uint32_t hi, lo;
    split2(x, y, hi, lo);
    uint32_t* at = static_cast<uint32_t*>(tile) + swz<kC>(row, block) / 4 + (lane & 3);
    at[0] = hi;
    if (both) at[kC * kC / 2] = lo;
}
__device__ __forceinline__ float2 get2(const void* tile, int row, int block, int lane) {
    const uint32_t* at = static_cast<const uint32_t*>(tile) + swz<kC>(row, block) / 4 + (lane & 3);
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(at));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(at + kC * kC / 2));
    return make_float2(hi.x + lo.x, hi.y + lo.y);
}

template <int D, typename Tok>
__global__ void __launch_bounds__(kThreads, sizeof(Tok) == 4 ? 3 : D == 64 ? 5 : 4) delta_prepare_kernel(DeltaArgs a, DeltaChunk* out, int chunks, int p_pieces) {
    using Tiles = Shared<D, Tok>;
    constexpr int NP = Tiles::kPieces, VEC = kC * D / 8 / kThreads;  // blocks of eight values of a thread
    extern __shared__ __align__(1024) unsigned char smem[];
    Tiles& tiles = *reinterpret_cast<Tiles*>(smem);
    Common& c = *reinterpret_cast<Common*>(smem + sizeof(Tiles));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long unit = blockIdx.x / chunks;
    const int chunk = (int)(blockIdx.x % chunks);
    const long len = delta_length(a, unit / a.H), t0 = (long)chunk * kC;
    if (t0 >= len) return;
    const int n = (int)min((long)kC, len - t0);  // the rest of the tile is zero: no decay, no write
    DeltaChunk& o = out[(long)unit * chunks + chunk];

    // K and Q, scaled by the tiles' powers of two, into shared memory
    const long row0 = delta_key_head(a, unit) * a.T + t0;
    float s[2];
    {
        Block8<Tok> raw[2][VEC];
        float x[8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const Tok* p = static_cast<const Tok*>(w ? a.q : a.k) + row0 * D;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid;
                if (block / (D / 8) < n)
                    raw[w][i].load(p + (long)block * 8);
                else
                    raw[w][i].clear();
            }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                raw[w][i].get(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
            }
            top = warp_max(top);
            if (lane == 0) c.tops[w * 4 + warp] = top;
        }
        __syncthreads();
        float inv[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            s[w] = pow2_scale(fmaxf(fmaxf(c.tops[w * 4], c.tops[w * 4 + 1]), fmaxf(c.tops[w * 4 + 2], c.tops[w * 4 + 3])),
                              inv[w]);
            const uint32_t base = smem_u32(w ? tiles.q : tiles.k);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid, row = block / (D / 8);
                raw[w][i].get(x);
                put8<NP>(base + swz<D>(row, block % (D / 8)), kC * D * 2, x, s[w]);
            }
        }
        if (tid == 0) o.k_scale = s[0], o.q_scale = s[1], o.k_inv = inv[0], o.q_inv = inv[1];
        s[0] = inv[0], s[1] = inv[1];  // from here on the inverses
    }

    // The decays, two tokens a lane. G is summed in 64 bits and kept as two floats: D needs the difference of
    // two sums to fp32's precision of exp(G_i - G_j), however far both are from 0. A decay of 0 is counted
    // apart: D_ij = 0 where one lies between. The others' sums stay above -64 * 104, where neither the sum nor its two
    // floats lose anything of a token's g, however low the marker that a decay of 0 was given as.
    if (warp == 0) {
        double g[2];
        int zero[2];
        float beta[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float x = t < n ? a.g[unit * a.T + t0 + t] : 0.f;
            beta[i] = t < n ? a.beta[unit * a.T + t0 + t] : 0.f;
            zero[i] = x < kForget;
            g[i] = zero[i] ? 0.0 : (double)x;
        }
        const double sum = warp_prefix(g[0] + g[1], lane), last = __shfl_sync(0xffffffffu, sum, 31);
        int zeros = zero[0] + zero[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, zeros, d);
            if (lane >= d) zeros += y;
        }
        const int all = __shfl_sync(0xffffffffu, zeros, 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const double G = i ? sum : sum - g[1];
            const int z = i ? zeros : zeros - zero[1];
            const float hi = (float)G;
            o.ghi[t] = c.ghi[t] = hi, o.glo[t] = c.glo[t] = (float)(G - hi), o.zeros[t] = c.zeros[t] = z;
            c.beta[t] = beta[i];
            o.gamma[t] = z ? 0.f : expf((float)G);
            o.rest[t] = z == all ? expf((float)(last - G)) : 0.f;
            o.beta[t] = beta[i];
        }
    }
    __syncthreads();

    // The decays between blocks, one or two a thread
    for (int x = tid; x < kC + 96; x += kThreads) {
        if (x < kC) {
            o.from[x] = c.from[x] = x < 16 ? 0.f : decay_between(c.ghi, c.glo, c.zeros, x, (x & ~15) - 1);
        } else {
            const int y = x - kC, block = y < 16 ? 0 : y < 48 ? 1 : 2, j = y - (block == 0 ? 0 : block == 1 ? 16 : 48);
            o.to[block][j] = c.to[block][j] = decay_between(c.ghi, c.glo, c.zeros, block * 16 + 15, j);
        }
    }
    __syncthreads();

    // Rows 16 warp .. + 15 of K K^T and Q K^T, up to the diagonal
    const uint32_t ks = smem_u32(tiles.k), qs = smem_u32(tiles.q), lo = kC * D * 2;
    const float kk_inv = s[0] * s[0], qk_inv = s[0] * s[1];
    float kk[8][4] = {}, qk[8][4] = {};
    for (int k0 = 0; k0 < D; k0 += 16) {
        uint32_t ka[NP][4], qa[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            frag_a<D>(ka[p], ks + p * lo, warp * 16, k0, lane);
            frag_a<D>(qa[p], qs + p * lo, warp * 16, k0, lane);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > warp) continue;
            uint32_t b[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) frag_b<D>(b[p], ks + p * lo, j * 16, k0, lane);
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int r = 0; r < NP - p; ++r)  // hi hi, hi lo, lo hi
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma16816(kk[2 * j + h], ka[p], b[r][2 * h], b[r][2 * h + 1]);
                        mma16816(qk[2 * j + h], qa[p], b[r][2 * h], b[r][2 * h + 1]);
                    }
        }
    }
    float p_top = 0.f, m_top = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        if (t >> 1 > warp) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = warp * 16 + (lane >> 2) + (e >> 1) * 8, j = 8 * t + 2 * (lane & 3) + (e & 1);
            // D_ij; between blocks it is a product over the end of the block before i's, two factors of at most 1
            const float d = t >> 1 < warp ? c.from[i] * c.to[warp - 1][j]
                            : j <= i      ? decay_between(c.ghi, c.glo, c.zeros, i, j)
                                          : 0.f;
            qk[t][e] *= qk_inv * d;
            kk[t][e] *= j < i ? kk_inv * d : 0.f;
            p_top = fmaxf(p_top, fabsf(qk[t][e]));
            m_top = fmaxf(m_top, fabsf(kk[t][e]));
        }
    }
    p_top = warp_max(p_top), m_top = warp_max(m_top);
    if (lane == 0) c.tops[warp] = p_top, c.tops[4 + warp] = m_top;
    __syncthreads();  // also: the tiles of K and Q are not read again

    float m_inv;
    {
        float p_inv;
        const float ps = pow2_scale(fmaxf(fmaxf(c.tops[0], c.tops[1]), fmaxf(c.tops[2], c.tops[3])), p_inv);
        const float ms = pow2_scale(fmaxf(fmaxf(c.tops[4], c.tops[5]), fmaxf(c.tops[6], c.tops[7])), m_inv);
        if (tid == 0) o.p_inv = p_inv;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t >> 1 > warp) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = warp * 16 + (lane >> 2) + h * 8;
                put2(o.P, row, t, lane, qk[t][2 * h] * ps, qk[t][2 * h + 1] * ps, p_pieces == 2);
                put2(smem, row, t, lane, kk[t][2 * h] * ms, kk[t][2 * h + 1] * ms);
                if (t >> 1 == warp) {
                    const int j = 8 * (t & 1) + 2 * (lane & 3);
                    c.diag[warp][j][row & 15] = kk[t][2 * h], c.diag[warp][j + 1][row & 15] = kk[t][2 * h + 1];
                }
            }
        }
    }
    __syncwarp();
    {  // T of block `warp`: column `lane` of the inverse (lanes 16.. go along with the first sixteen)
        const int at = warp * 16, col = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < 15; ++j) {
            const float z = x[j] * c.beta[at + j];
            float m[16];
#pragma unroll
            for (int i = (j + 1) / 2 * 2; i < 16; i += 2) {
                const float2 u = *reinterpret_cast<const float2*>(&c.diag[warp][j][i]);
                m[i] = u.x, m[i + 1] = u.y;
            }
#pragma unroll
            for (int i = j + 1; i < 16; ++i) x[i] = fmaf(-m[i], z, x[i]);
        }
        float top = 0.f, inv;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
        const float sc = pow2_scale(warp_max(top), inv);
        if (lane == 0) c.t_inv[warp] = inv;
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const __half h = __float2half_rn(x[i] * sc);
                c.t[warp][0][i * kTPitch + col] = h;
                c.t[warp][1][i * kTPitch + col] = __float2half_rn(x[i] * sc - __half2float(h));
            }
        }
    }
    __syncthreads();

    // N's column block `warp`
    float nc[4][2][4];
    uint32_t nb[3][2][2][2];  // beta N as B fragments
    float nb_inv[3];
    float n_top = 0.f;
    unrolled<4>([&](auto row_block) {
        constexpr int i = row_block;
        if (i < warp) return;
        float x[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 u = get2(smem, i * 16 + (lane >> 2) + h * 8, warp * 2 + t, lane);
                x[t][2 * h] = u.x * m_inv, x[t][2 * h + 1] = u.y * m_inv;
            }
#pragma unroll
        for (int j = 0; j < i; ++j) {
            if (j < warp) continue;
            uint32_t a[2][4];
            frag_a<kC>(a[0], smem_u32(smem), i * 16, j * 16, lane);
            frag_a<kC>(a[1], smem_u32(smem) + kC * kC * 2, i * 16, j * 16, lane);
            float acc[2][4] = {};
            multiply(acc, a, nb[j]);
            const float f = m_inv * nb_inv[j];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][e] = fmaf(-acc[t][e], f, x[t][e]);
        }
        float inv;
        uint32_t b[2][2][2], a[2][4];
        to_fragment(x, pow2_scale(top16(x), inv), b);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            ldsm4(a[e], smem_u32(c.t[i][e]) + ((lane & 7) + ((lane >> 3) & 1) * 8) * kTPitch * 2 + (lane >> 4) * 16);
        float acc[2][4] = {};
        multiply(acc, a, b);
        inv *= c.t_inv[i];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                nc[i][t][e] = acc[t][e] * inv;
                x[t][e] = nc[i][t][e] * c.beta[i * 16 + (lane >> 2) + (e >> 1) * 8];
                n_top = fmaxf(n_top, fabsf(nc[i][t][e]));
            }
        if constexpr (i < 3) to_fragment(x, pow2_scale(top16(x), nb_inv[i]), nb[i]);
    });
    n_top = warp_max(n_top);
    if (lane == 0) c.tops[8 + warp] = n_top;
    __syncthreads();
    float inv;
    const float ns = pow2_scale(fmaxf(fmaxf(c.tops[8], c.tops[9]), fmaxf(c.tops[10], c.tops[11])), inv);
    if (tid == 0) o.n_inv = inv;
    unrolled<4>([&](auto row_block) {
        constexpr int i = row_block;
        if (i < warp) return;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                put2(o.N, i * 16 + (lane >> 2) + h * 8, warp * 2 + t, lane, nc[i][t][2 * h] * ns, nc[i][t][2 * h + 1] * ns);
    });
}

template <int D, typename Tok>
cudaError_t launch(const DeltaArgs& a, DeltaChunk* out, int chunks, int p_pieces, cudaStream_t st) {
    constexpr size_t bytes = sizeof(Shared<D, Tok>) + sizeof(Common);
    auto* kernel = delta_prepare_kernel<D, Tok>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long)a.B * a.H * chunks), kThreads, bytes, st>>>(a, out, chunks, p_pieces);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prepare(const DeltaArgs& a, void* chunks_out, bool backward, cudaStream_t st) {
    const int chunks = (int)((a.T + kC - 1) / kC);
    DeltaChunk* out = static_cast<DeltaChunk*>(chunks_out);
    const int n = backward ? 2 : delta_y_pieces(a);  // pieces of P that the other kernels read
    if (a.d == 64)
        return a.bf16 ? launch<64, __nv_bfloat16>(a, out, chunks, n, st) : launch<64, float>(a, out, chunks, n, st);
    return a.bf16 ? launch<128, __nv_bfloat16>(a, out, chunks, n, st) : launch<128, float>(a, out, chunks, n, st);
}

size_t delta_chunk_bytes() { return sizeof(DeltaChunk); }

}  // namespace titans
