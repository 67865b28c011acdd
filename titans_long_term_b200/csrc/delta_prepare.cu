// Gated delta rule, first kernel of the chunked path: what a chunk's tokens need of one another (N, P and the
// decays; see delta_common.cuh), for every chunk of every unit at once, before the state is known.
//
// One CTA of 128 threads per (unit, chunk). K K^T and Q K^T are taken on the tensor cores, 16 rows a warp;
// N by forward substitution in fp32, one thread per column: x_i = M_ic - sum_{j<i} M_ij beta_j x_j, in
// blocks of 16 rows so that x stays in registers and the code small.
#include "delta_common.cuh"

namespace titans {
namespace {

constexpr int kThreads = 128;
constexpr int kLd = kC + 4;  // floats between rows of M^T

template <int D, typename Tok>
struct Shared {
    static constexpr int kPieces = sizeof(Tok) == 4 ? 2 : 1;
    __half k[kPieces][kC * D], q[kPieces][kC * D];
};
struct Common {
    alignas(16) float mt[kC * kLd];  // mt[j][i] = M_ij
    alignas(16) float z[kC * kC];    // z[j][c] = beta_j N_jc
    float beta[kC], ghi[kC], glo[kC];
    int zeros[kC];                   // tokens of the chunk so far whose decay is 0
    float tops[8];
};

template <int D, typename Tok>
__global__ void __launch_bounds__(kThreads) delta_prepare_kernel(DeltaArgs a, DeltaChunk* out, int chunks) {
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
        float x[2][VEC][8], top[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const Tok* p = static_cast<const Tok*>(w ? a.q : a.k) + row0 * D;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int block = i * kThreads + tid, row = block / (D / 8);
                if (row < n) {
                    load8(p + (long)block * 8, x[w][i]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[w][i][j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) top[w] = fmaxf(top[w], fabsf(x[w][i][j]));
            }
            top[w] = warp_max(top[w]);
            if (lane == 0) c.tops[w * 4 + warp] = top[w];
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
                put8<NP>(base + swz<D>(row, block % (D / 8)), kC * D * 2, x[w][i], s[w]);
            }
        }
        if (tid == 0) o.k_scale = s[0], o.q_scale = s[1], o.k_inv = inv[0], o.q_inv = inv[1];
        s[0] = inv[0], s[1] = inv[1];  // from here on the inverses
    }

    // The decays, two tokens a lane. G is summed in 64 bits and kept as two floats: D needs the difference of
    // two sums to fp32's precision of exp(G_i - G_j), however far both are from 0. A decay of 0 (g = -inf) is counted
    // apart: D_ij = 0 where one lies between, and the others' sums stay finite.
    if (warp == 0) {
        double g[2];
        int zero[2];
        float beta[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float x = t < n ? a.g[unit * a.T + t0 + t] : 0.f;
            beta[i] = t < n ? a.beta[unit * a.T + t0 + t] : 0.f;
            zero[i] = x == -INFINITY;
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

    // Rows 16 warp .. + 15 of K K^T and Q K^T, up to the diagonal
    const uint32_t ks = smem_u32(tiles.k), qs = smem_u32(tiles.q), lo = kC * D * 2;
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
    float p_top = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = warp * 16 + (lane >> 2) + (e >> 1) * 8, j = 8 * t + 2 * (lane & 3) + (e & 1);
            float m = 0.f, p = 0.f;
            if (j <= i) {
                const float d = decay_between(c.ghi, c.glo, c.zeros, i, j) * s[0];
                p = qk[t][e] * s[1] * d;
                m = j < i ? kk[t][e] * s[0] * d : 0.f;
            }
            qk[t][e] = p;
            p_top = fmaxf(p_top, fabsf(p));
            c.mt[j * kLd + i] = m;
        }
    p_top = warp_max(p_top);
    if (lane == 0) c.tops[warp] = p_top;
    __syncthreads();

    // P to the workspace, through the tiles of K and Q, which are not read again
    {
        float inv;
        const float ps = pow2_scale(fmaxf(fmaxf(c.tops[0], c.tops[1]), fmaxf(c.tops[2], c.tops[3])), inv);
        if (tid == 0) o.p_inv = inv;
        unsigned char* t = smem;  // at least 16 KiB
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi, l;
                split2(qk[j][2 * h] * ps, qk[j][2 * h + 1] * ps, hi, l);
                const uint32_t off = swz<kC>(warp * 16 + (lane >> 2) + h * 8, j) + (lane & 3) * 4;
                *reinterpret_cast<uint32_t*>(t + off) = hi;
                *reinterpret_cast<uint32_t*>(t + kC * kC * 2 + off) = l;
            }
        __syncthreads();
        uint4* dst = reinterpret_cast<uint4*>(o.P);
        for (int i = tid; i < (int)sizeof(o.P) / 16; i += kThreads) dst[i] = reinterpret_cast<uint4*>(t)[i];
    }

    __syncthreads();

    // N, a column a thread
    float* nb = reinterpret_cast<float*>(smem);  // nb[i][c] = N_ic
    float n_top = 0.f;
    if (tid < kC) {
        for (int bi = 0; bi < kC; bi += 16) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = c.mt[tid * kLd + bi + i];
#pragma unroll 4
            for (int j = 0; j < bi; ++j) {
                const float z = c.z[j * kC + tid];
                const float4* m = reinterpret_cast<const float4*>(c.mt + j * kLd + bi);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 r = m[i];
                    x[4 * i] = fmaf(-r.x, z, x[4 * i]), x[4 * i + 1] = fmaf(-r.y, z, x[4 * i + 1]);
                    x[4 * i + 2] = fmaf(-r.z, z, x[4 * i + 2]), x[4 * i + 3] = fmaf(-r.w, z, x[4 * i + 3]);
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float z = x[j] * c.beta[bi + j];
                c.z[(bi + j) * kC + tid] = z;
                n_top = fmaxf(n_top, fabsf(x[j]));
#pragma unroll
                for (int i = j + 1; i < 16; ++i) x[i] = fmaf(-c.mt[(bi + j) * kLd + bi + i], z, x[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) nb[(bi + i) * kC + tid] = x[i];
        }
        n_top = warp_max(n_top);
        if (lane == 0) c.tops[4 + warp] = n_top;
    }
    __syncthreads();
    {
        float inv;
        const float ns = pow2_scale(fmaxf(c.tops[4], c.tops[5]), inv);
        if (tid == 0) o.n_inv = inv;
        uint32_t* dst = reinterpret_cast<uint32_t*>(o.N);
        for (int i = tid; i < kC * kC / 2; i += kThreads) {  // a pair of neighbouring columns of one row
            const int row = i >> 5, at = (i & 31) * 4, col = (((at >> 4) ^ (row & 7)) << 3) + ((at & 15) >> 1);
            uint32_t hi, l;
            split2(nb[row * kC + col] * ns, nb[row * kC + col + 1] * ns, hi, l);
            dst[i] = hi;
            dst[kC * kC / 2 + i] = l;
        }
    }
}

template <int D, typename Tok>
cudaError_t launch(const DeltaArgs& a, DeltaChunk* out, int chunks, cudaStream_t st) {
    constexpr size_t bytes = sizeof(Shared<D, Tok>) + sizeof(Common);
    auto* kernel = delta_prepare_kernel<D, Tok>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long)a.B * a.H * chunks), kThreads, bytes, st>>>(a, out, chunks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prepare(const DeltaArgs& a, void* chunks_out, cudaStream_t st) {
    const int chunks = (int)((a.T + kC - 1) / kC);
    DeltaChunk* out = static_cast<DeltaChunk*>(chunks_out);
    if (a.d == 64)
        return a.bf16 ? launch<64, __nv_bfloat16>(a, out, chunks, st) : launch<64, float>(a, out, chunks, st);
    return a.bf16 ? launch<128, __nv_bfloat16>(a, out, chunks, st) : launch<128, float>(a, out, chunks, st);
}

size_t delta_chunk_bytes() { return sizeof(DeltaChunk); }

}  // namespace titans
