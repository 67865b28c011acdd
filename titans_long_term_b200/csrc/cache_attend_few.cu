// Attention over the paged cache for up to sixteen rows of a key/value head (rows: its new tokens times the query heads
// that share it), which reading the cache bounds: a decode step.
//
// Eight warps of a CTA take blocks of keys in turn, each with a maximum, sum and output of its own, joined in
// shared memory at the end (and over the CTAs that split a sequence by combine_kernel). Nothing is staged: a lane loads
// 16 consecutive bytes of a key or value row from the cache straight into the fragment of an m16n8k16 product.
//   S = Q K^T: the sum over d may run in any order that Q and K share, so lane % 4 takes every fourth 16-byte
//              piece of a row, in two (bf16) or four (e4m3) steps of 16 of d, and Q is loaded the same way.
//   O += P V:  column n of an output tile may stand for any d, so lane / 4 takes a piece of consecutive d and its
//              i-th value belongs to tile i; the values of two keys are paired by a byte permutation.
// While one block is multiplied the next one's keys and values are on their way: 8 KiB a warp, 64 KiB an SM.
// An e4m3 cache is converted to bf16 in registers, exactly; its scales multiply the scores and the weights.
// A page holds at least 16 tokens, so 16 keys need one look into the page table.
#include <algorithm>

#include "cache_attend.cuh"
#include "ptx.cuh"

namespace titans {
namespace {

constexpr int kWarps = 8, kM = 16;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two e4m3 values as bf16, exactly.
__device__ __forceinline__ uint32_t bf16_of(uint32_t e4m3x2) {
    const float2 f = e4m3x2_to_float2((uint16_t)e4m3x2);
    return pack_bf16x2(f.x, f.y);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, 1) attend_few_kernel(AttendArgs a) {
    constexpr int SUB = E4M3 ? 2 : 1, KEYS = 16 * SUB;  // a block: one or two times 16 keys
    constexpr int KP = D * (E4M3 ? 1 : 2) / 64;         // 16-byte pieces of a key row for each of four lanes
    constexpr int KW = E4M3 ? 8 : 4;                    // bf16 pairs of such a piece
    constexpr int VE = E4M3 && D == 128 ? 16 : 8;       // consecutive values of a value row a lane takes,
    constexpr int VG = D / 8 / VE;                      // in so many groups of 8 VE
    constexpr int VB = VE * (E4M3 ? 1 : 2);             // bytes: 16, or 8 (e4m3, d = 64)
    extern __shared__ __align__(16) float smem[];  // outputs [warps][16][D], then maxima and sums [warps][16]
    const CacheArgs& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q4 = lane & 3;
    const int units = c.B * c.Hkv, unit = blockIdx.x % units, b = unit / c.Hkv, hk = unit % c.Hkv, G = c.H / c.Hkv;
    const int rows = (int)c.T * G, count = cache_count(c, b);
    const long start = c.starts[b];
    const int seen_rows = min(rows, count * G), split = blockIdx.x / units, splits = gridDim.x / units;
    Tiles tiles{0, 0, 0};
    long see_lo = 0, see_hi = -1, sink_hi = 0;  // keys that some row sees: see_lo..see_hi, and below sink_hi
    if (seen_rows > 0) {
        see_hi = start + (seen_rows - 1) / G;
        tiles = tiles_of<KEYS>(a, start, see_hi);
        see_lo = seen_by(a, start).begin, sink_hi = seen_by(a, see_hi).sink_end;
    }
    const int first = (int)((long)tiles.count * split / splits), last = (int)((long)tiles.count * (split + 1) / splits);

    // This lane's rows r and r + 8
    long p[2];
    Seen seen[2];
    bool live[2];
    uint32_t q[KP * KW / 2][4];
    const float scale = a.scale * 1.44269504f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = r + 8 * h;
        live[h] = row < seen_rows;
        p[h] = start + row / G;
        seen[h] = seen_by(a, p[h]);
        const long at = (((long)b * c.H + hk * G + row % G) * c.T + row / G) * D;
#pragma unroll
        for (int i = 0; i < KP; ++i)
#pragma unroll
            for (int w = 0; w < KW; w += 2) {
                uint2 u = make_uint2(0, 0);
                if (live[h])
                    u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + at + (q4 + 4 * i) * 2 * KW +
                                                        2 * w);
                q[(i * KW + w) / 2][h] = u.x, q[(i * KW + w) / 2][2 + h] = u.y;
            }
    }
    // Row of the pool where 16 keys from key0 on begin, or -1
    auto find = [&](long key0) -> long {
        if (key0 > see_hi || (key0 + 15 < see_lo && key0 >= sink_hi)) return -1;
        const long at = cache_row(c, b, hk, key0);
        if (at < 0 && lane == 0) atomicOr(c.status, kStatusMissingPage);
        return at;
    };
    uint4 kb[SUB][2][KP];
    uint4 vb[SUB][4][VG];
    float ks[SUB][4], vs[SUB][4];  // e4m3: scales of the keys 2 q4 + {0, 1, 8, 9}
    auto load_k = [&](const long (&at)[SUB]) {
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < KP; ++i) {
                    kb[s][h][i] = make_uint4(0, 0, 0, 0);
                    if (at[s] >= 0)
                        kb[s][h][i] = static_cast<const uint4*>(c.pk)[(at[s] + r + 8 * h) * (4 * KP) + q4 + 4 * i];
                }
        if constexpr (E4M3) {
#pragma unroll
            for (int s = 0; s < SUB; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) ks[s][e] = at[s] >= 0 ? c.k_scale[at[s] + 2 * q4 + (e & 1) + (e >> 1) * 8] : 0.f;
        }
    };
    // Values that no row sees are zeros: their weights are 0, and 0 times an infinity or NaN would not be.
    auto load_v = [&](const long (&at)[SUB], long key0) {
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 2 * q4 + (e & 1) + (e >> 1) * 8;
                const long key = key0 + 16 * s + k;
                const bool there = at[s] >= 0 && key <= see_hi && (key >= see_lo || key < sink_hi);
#pragma unroll
                for (int g = 0; g < VG; ++g) {
                    vb[s][e][g] = make_uint4(0, 0, 0, 0);
                    const char* src = static_cast<const char*>(c.pv) + (at[s] + k) * (D * (E4M3 ? 1 : 2)) + (g * 8 + r) * VB;
                    if (there) {
                        if constexpr (VB == 16) {
                            vb[s][e][g] = *reinterpret_cast<const uint4*>(src);
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2*>(src);
                            vb[s][e][g].x = u.x, vb[s][e][g].y = u.y;
                        }
                    }
                }
                if constexpr (E4M3) vs[s][e] = there ? c.v_scale[at[s] + k] : 0.f;
            }
    };

    float o[VG][VE][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    long at[SUB], at_next[SUB];
    auto find_all = [&](int i, long (&x)[SUB]) {
#pragma unroll
        for (int s = 0; s < SUB; ++s) x[s] = i < last ? find((long)tiles[i] * KEYS + 16 * s) : -1;
    };
    int i = first + warp;
    find_all(i, at);
    load_k(at);
    load_v(at, i < last ? (long)tiles[i] * KEYS : 0);
    find_all(i + kWarps, at_next);
    for (; i < last; i += kWarps) {
        const long key0 = (long)tiles[i] * KEYS;
        float sc[2 * SUB][4] = {};
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)  // keys 8 h .. of the sixteen
#pragma unroll
                for (int j = 0; j < KP; ++j) {
                    const uint4 u = kb[s][h][j];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    if constexpr (E4M3) {
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            mma_bf16(sc[2 * s + h], q[j * 4 + t], bf16_of(w[t]), bf16_of(w[t] >> 16));
                    } else {
                        mma_bf16(sc[2 * s + h], q[j * 2], w[0], w[1]);
                        mma_bf16(sc[2 * s + h], q[j * 2 + 1], w[2], w[3]);
                    }
                }
        float kscale[SUB][4];
        bool there[SUB];
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            there[s] = at[s] >= 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) kscale[s][e] = E4M3 ? ks[s][e] * scale : scale;
        }
        load_k(at_next);
        // Scores in log2 units; -infinity where the row does not see the key
        bool whole = true;
#pragma unroll
        for (int s = 0; s < SUB; ++s) whole = whole && there[s];
#pragma unroll
        for (int h = 0; h < 2; ++h) whole = whole && (!live[h] || (key0 >= seen[h].begin && key0 + KEYS - 1 <= p[h]));
        whole = __all_sync(0xffffffffu, whole);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 2 * SUB; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int h = e >> 1;
                float x = sc[t][e] * kscale[t >> 1][(t & 1) * 2 + (e & 1)];
                if (!whole) {
                    const long key = key0 + 8 * t + 2 * q4 + (e & 1);
                    if (!there[t >> 1] || key > p[h] || (key < seen[h].begin && key >= seen[h].sink_end)) x = -INFINITY;
                }
                sc[t][e] = x;
                top[h] = fmaxf(top[h], x);
            }
        bool grown = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            grown = grown || top[h] - m[h] > 8.f || (m[h] == -INFINITY && top[h] > m[h]);
        }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float next = fmaxf(m[h], top[h]), keep = m[h] == next ? 1.f : ex2(m[h] - next);
                m[h] = next;
                l[h] *= keep;
#pragma unroll
                for (int g = 0; g < VG; ++g)
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[g][e][2 * h] *= keep, o[g][e][2 * h + 1] *= keep;
            }
        }
        const float shift[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = ex2(sc[2 * s + t][2 * h] - shift[h]), y = ex2(sc[2 * s + t][2 * h + 1] - shift[h]);
                    l[h] += x + y;
                    if constexpr (E4M3) x *= vs[s][2 * t], y *= vs[s][2 * t + 1];  // powers of two: no rounding
                    w[2 * t + h] = pack_bf16x2(x, y);
                }
#pragma unroll
            for (int g = 0; g < VG; ++g) {
                const uint32_t v[4][4] = {{vb[s][0][g].x, vb[s][0][g].y, vb[s][0][g].z, vb[s][0][g].w},
                                          {vb[s][1][g].x, vb[s][1][g].y, vb[s][1][g].z, vb[s][1][g].w},
                                          {vb[s][2][g].x, vb[s][2][g].y, vb[s][2][g].z, vb[s][2][g].w},
                                          {vb[s][3][g].x, vb[s][3][g].y, vb[s][3][g].z, vb[s][3][g].w}};
#pragma unroll
                for (int e = 0; e < VE; e += 2) {
                    uint32_t x[4];  // values e, e + 1 of the four keys
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = E4M3 ? bf16_of(v[k][e >> 2] >> (e & 2) * 8) : v[k][e >> 1];
                    mma_bf16(o[g][e], w, __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
                    mma_bf16(o[g][e + 1], w, __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
                }
            }
        }
        load_v(at_next, i + kWarps < last ? (long)tiles[i + kWarps] * KEYS : 0);
#pragma unroll
        for (int s = 0; s < SUB; ++s) at[s] = at_next[s];
        find_all(i + 2 * kWarps, at_next);
    }

    // Join the warps: row by row, in the order of the warps
    float* out = smem;
    float2* ml = reinterpret_cast<float2*>(smem + kWarps * kM * D);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int row = r + 8 * h;
        if (q4 == 0) ml[warp * kM + row] = make_float2(m[h], l[h]);
#pragma unroll
        for (int g = 0; g < VG; ++g)
#pragma unroll
            for (int n = 0; n < 2; ++n)  // column 2 q4 + n stands for d = 8 g VE + (2 q4 + n) VE + e
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    out[(warp * kM + row) * D + g * 8 * VE + (2 * q4 + n) * VE + e] = o[g][e][2 * h + n];
    }
    __syncthreads();
    for (int row = warp; row < rows && row < kM; row += kWarps) {  // one warp a row, D / 32 columns a lane
        constexpr int N = D / 32;
        const int t = row / G;
        const long orow = ((long)b * c.H + hk * G + row % G) * c.T + t;
        float top = -INFINITY, sum = 0.f, acc[N] = {};
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * kM + row].x);
        for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w * kM + row];
            if (x.x == -INFINITY && x.y == 0.f) continue;
            const float f = x.x == top ? 1.f : ex2(x.x - top);
            sum = fmaf(x.y, f, sum);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(out[(w * kM + row) * D + lane * N + i], f, acc[i]);
        }
        bool fine = fabsf(sum) < INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) fine = fine && fabsf(acc[i]) < INFINITY;
        if (row < seen_rows && !__all_sync(0xffffffffu, fine))
            attend_row<D, E4M3, KEYS>(a, b, hk, static_cast<const __nv_bfloat16*>(a.q) + orow * D, start + t, tiles, first,
                                      last, top, sum, acc);
        if (splits > 1) {
            const long prow = (long)split * c.B * c.H * c.T + orow;
#pragma unroll
            for (int i = 0; i < N; ++i) a.part[prow * D + lane * N + i] = acc[i];
            if (lane == 0) a.part_ml[prow] = make_float2(top, sum);
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int i = 0; i < N; ++i)
                static_cast<__nv_bfloat16*>(a.o)[orow * D + lane * N + i] = __float2bfloat16(acc[i] * inv);
        }
    }
}

template <int D, bool E4M3>
cudaError_t launch(const AttendArgs& a, int splits, cudaStream_t st) {
    constexpr int bytes = kWarps * kM * (D * (int)sizeof(float) + (int)sizeof(float2));
    auto* kernel = attend_few_kernel<D, E4M3>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)((long)a.c.B * a.c.Hkv * splits), kWarps * 32, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

bool attend_few_rows(int H, int Hkv, long T) { return T * (H / Hkv) <= kM; }

// CTAs for about four rounds over the SMs, so that sequences of different lengths even out, and at least 16 blocks of the
// longest possible sequence a CTA, two a warp.
int attend_few_splits(int B, int Hkv, long longest) {
    const long base = (long)B * Hkv;
    return (int)std::max(1L, std::min({longest / (16 * 16), (4 * 148L + base - 1) / base, 64L}));
}

cudaError_t launch_attend_few(const AttendArgs& a, bool e4m3, int splits, cudaStream_t st) {
    if (a.c.d == 64) return e4m3 ? launch<64, true>(a, splits, st) : launch<64, false>(a, splits, st);
    return e4m3 ? launch<128, true>(a, splits, st) : launch<128, false>(a, splits, st);
}

}  // namespace titans
