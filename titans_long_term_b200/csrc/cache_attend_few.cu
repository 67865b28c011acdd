// Attention over the paged cache for up to sixteen rows of a key/value head (rows: its new tokens times the query heads
// that share it), which reading the cache bounds: a decode step.
//
// One round of CTAs shares out all blocks of keys of all sequences evenly: CTA i of n takes blocks i total / n .. of the
// sequence of (sequence, head, block), whatever the lengths are, so it may end one head's keys, go through
// some more and begin another's. What is only a part of a head's keys goes to the workspace, two places a CTA
// (the part its range begins with, and the part it ends with), and join_kernel adds the parts up.
//
// The warps of a CTA take blocks of keys in turn, each with a maximum, sum and output of its own, joined in
// shared memory at the end of a head's keys. Nothing is staged: a lane loads 16 consecutive bytes of a key or value row
// from the cache straight into the A fragment of m16n8k16 products, whose eight columns are the rows of Q.
//   S^T = K Q^T:    the sum over d may run in any order that Q and K share, so lane % 4 takes every fourth 16-byte
//                   piece of a row, in two (bf16) or four (e4m3) steps of 16 of d, and Q is loaded the same way.
//   O^T += V^T P^T: row m of an output tile may stand for any d, so lane / 4 takes a piece of consecutive d, whose values
//                   2 i and 2 i + 1 belong to tile i; the values of two keys are paired by a byte permutation.
// With keys and values as the 16-row side, eight rows of Q (one token of up to eight heads) cost half the registers and
// instructions of the other way round. While one block is multiplied the next one's keys and values are on their way, 8 (bf16)
// or 4 KiB a warp. What bounds it: the loads in flight (three warps a scheduler, most of their stalls waiting for loads; over an
// e4m3 cache, whose conversion makes a chain of instructions besides, issue slots are 36 % busy and HBM gives 3.5 TB/s), and the latency of the
// dependent loads and the join where there is little to read. 16 heads on 4, d = 128, 8192 keys in scattered pages, calls in a
// graph over three caches in turn, this kernel | the tile kernel:
//   sequences   4 rows, bf16         4 rows, e4m3        16 rows, bf16  16 rows, e4m3
//   1           17.6 | 20.5 us       16.5 | 24.0 us      19.8 | 20.5    19.8 | 24.6
//   8           40.3 | 38.2 us       33.4 | 57.0 us      49.7 | 38.0    46.0 | 58.0
//   32          97 | 106 us          77 | 184 us         130 | 107      115 | 185
//               (5.5 TB/s)           (3.6 TB/s)
// So up to 16 rows are its own whatever the type and the batch, which costs a quarter at more than eight rows of several bf16
// sequences.
// A page holds at least 16 tokens, so 16 keys need one look into the page table, two blocks ahead of their use.
//
// An e4m3 cache is multiplied in fp16, to which one instruction converts two values exactly. Q goes to fp16
// times a power of two of its row (largest element at 2^14..2^15: exact down to 2^-28 of it). Weights go to
// fp16 as 2^(7 + z + log2 s - M), s the scale of the key's values and M the running maximum of z + log2 s over the keys whose values
// are not all zeros. Such a key's largest value is at least 2^7.8 of its scale, so what the fp16 weights lose (half a step, 2^-11
// of each, and at most 2^-25 where the largest one is 2^7 or more) is small beside the output whatever the scales are. A key without any value
// has a scale of 1 all the same and would push the others' weights out of fp16's range; it is left out of M and its weight is
// held below 2^15, as its product is 0 anyway. The sum of the weights knows nothing of the values: each lane keeps it in fp32
// beside a maximum of its own, of z alone, that the scores may pass by 32. The second exponential of a score costs nothing that
// shows (32 sequences, d = 128: 77.9 us in place of 78.6 with the sum taken back by 1 / s, which lost what s put out of range).
#include <algorithm>
#include <type_traits>

#include "cache_attend.cuh"
#include "ptx.cuh"

namespace titans {
namespace {

constexpr int kM = 16;
constexpr int kMostCtas = kSms;  // one an SM

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
constexpr int kBlock = 16;  // keys of a block: the 16 rows of an MMA's A operand, and no page is shorter
constexpr float kNothing = -3.4028234664e38f;  // below every score
constexpr float kTopBits = 7.f, kMostWeight = 32768.f;  // e4m3: the weight of the maximum, 2^7, times the 2^8 it may lag behind

// The keys of sequence b that some of its rows see.
__device__ __forceinline__ Seen keys_of(const AttendArgs& a, int b) {
    const int n = cache_count(a.c, b);
    if (n == 0) return Seen{0, 0, 0};
    const long start = a.c.starts[b];
    return seen_by_any(a, start, start + n - 1);
}
// The CTA of n whose share of `total` holds block x.
__device__ __forceinline__ int owner(long x, long n, long total) { return (int)(((x + 1) * n - 1) / total); }

// NQ: tiles of eight rows.
template <int D, bool E4M3, int NQ>
struct Few {
    // Loads in flight against registers: with 8 rows 12 warps (32 sequences: 97 us against 107 with 8; e4m3 77 against 93), with 16
    // rows 8 (130 us against 173 with 12, which spill; e4m3 115 against 124)
    static constexpr int kWarps = NQ == 2 ? 8 : 12;
    static constexpr int kRows = 8 * NQ;
    static constexpr int kBytes = kWarps * kRows * (D * (int)sizeof(float) + (int)sizeof(float2));
    static constexpr int kKP = D * (E4M3 ? 1 : 2) / 64;  // 16-byte pieces of a key row for each of four lanes
    static constexpr int kKW = E4M3 ? 8 : 4;             // pairs of values of such a piece
    static constexpr int kVE = E4M3 && D == 128 ? 16 : 8;  // consecutive values of a value row a lane takes,
    static constexpr int kVG = D / 8 / kVE;                // in so many groups of 8 kVE
};

// Keys first..last-1 (in blocks) of key/value head hk of sequence b: writes the rows' outputs, or, where that is a part of the
// keys, their place in the workspace.
template <int D, bool E4M3, int NQ>
__device__ __forceinline__ void attend_head(const AttendArgs& a, int b, int hk, Tiles tiles, int first, int last, long place,
                                            float* smem) {
    using F = Few<D, E4M3, NQ>;
    constexpr int KEYS = kBlock, KP = F::kKP, KW = F::kKW, VE = F::kVE, VG = F::kVG, W = F::kWarps;
    constexpr int VB = VE * (E4M3 ? 1 : 2);  // bytes: 16, or 8 (e4m3, d = 64)
    const CacheArgs& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q4 = lane & 3;
    const int G = c.H / c.Hkv, rows = (int)c.T * G, seen_rows = min(rows, cache_count(c, b) * G);
    const long start = c.starts[b];
    const Seen any = keys_of(a, b), every = seen_by(a, start);  // what some row sees; with `whole` below, what every row sees
    const int every_begin = seen_by(a, start + (seen_rows - 1) / G).begin;

    // Q's rows 8 n + r as B fragments
    uint32_t q[NQ][KP * KW / 2][2];
    float q_inv[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int row = 8 * n + r;
        const long at = (((long)b * c.H + hk * G + row % G) * c.T + row / G) * D;
#pragma unroll
        for (int i = 0; i < KP; ++i)
#pragma unroll
            for (int w = 0; w < KW; w += 2) {
                uint2 u = make_uint2(0, 0);
                if (row < seen_rows)
                    u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) + at + (q4 + 4 * i) * 2 * KW +
                                                        2 * w);
                q[n][(i * KW + w) / 2][0] = u.x, q[n][(i * KW + w) / 2][1] = u.y;
            }
        q_inv[n] = 1.f;
        if constexpr (E4M3) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < KP * KW; ++i) {
                const float2 f = unpack_bf16x2(q[n][i >> 1][i & 1]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = max(__float_as_int(top) >> 23, 27) - 127;
            const float up = __int_as_float((14 - e + 127) << 23);
            q_inv[n] = __int_as_float((e - 14 + 127) << 23);
#pragma unroll
            for (int i = 0; i < KP * KW; ++i) {
                const float2 f = unpack_bf16x2(q[n][i >> 1][i & 1]);
                const __half2 v = __floats2half2_rn(f.x * up, f.y * up);
                q[n][i >> 1][i & 1] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
    }
    // Rows 8 n + 2 q4 + {0, 1}, whose scores this lane has (keys r and r + 8)
    // m: the running maximum that the weights refer to, the same in all lanes of a row; sum_m (e4m3): what this lane's sum l
    // refers to, in place of m
    float scale[NQ][2], m[NQ][2], sum_m[NQ][2], l[NQ][2] = {};
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            scale[n][h] = a.scale * 1.44269504f * __shfl_sync(0xffffffffu, q_inv[n], (2 * q4 + h) * 4);
            m[n][h] = -INFINITY, sum_m[n][h] = kNothing;
        }

    // The page of 16 keys from key0 on; -2 where no row sees any of them. Only the load, so that nothing waits for it
    // until row_of.
    const int* table = c.table + (long)b * c.max_pages;
    auto page_of = [&](int key0) -> int {
        if (key0 >= any.end || (key0 + 15 < any.begin && key0 >= any.sink_end)) return -2;
        return max(table[key0 >> c.page_shift], -1);
    };
    // Row of the pool where they begin, or -1.
    auto row_of = [&](int page, int key0) -> int {
        if ((unsigned)page >= (unsigned)c.num_pages) {
            if (page != -2 && lane == 0) atomicOr(c.status, kStatusMissingPage);
            return -1;
        }
        return ((page * c.Hkv + hk) << c.page_shift) + (key0 & ((1 << c.page_shift) - 1));  // rows are fewer than 2^31
    };
    uint4 kb[2][KP];
    uint4 vb[4][VG];
    float ks[2], vs[2];  // e4m3: scales of the keys r and r + 8
    auto load_k = [&](int at) {
        if (at < 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ks[h] = 0.f;
#pragma unroll
                for (int i = 0; i < KP; ++i) kb[h][i] = make_uint4(0, 0, 0, 0);
            }
            return;
        }
        const uint4* src = static_cast<const uint4*>(c.pk) + (long)(at + r) * (4 * KP) + q4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < KP; ++i) kb[h][i] = src[32 * KP * h + 4 * i];
        if constexpr (E4M3) ks[0] = c.k_scale[at + r], ks[1] = c.k_scale[at + r + 8];
    };
    // Values that no row sees are zeros: their weights are 0, and 0 times an infinity or NaN would not be.
    auto load_v = [&](int at, int key0) {
        auto load = [&](auto all) {
            const char* src = static_cast<const char*>(c.pv) + (long)(at + 2 * q4) * (D * (E4M3 ? 1 : 2)) + r * VB;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = (e & 1) + (e >> 1) * 8;
                const bool there = all.value || any(key0 + 2 * q4 + k);
#pragma unroll
                for (int g = 0; g < VG; ++g) {
                    const char* p = src + k * (D * (E4M3 ? 1 : 2)) + g * 8 * VB;
                    uint4& v = vb[e][g];
                    if constexpr (!all.value) v = make_uint4(0, 0, 0, 0);
                    if constexpr (VB == 16) {
                        if (there) v = *reinterpret_cast<const uint4*>(p);
                    } else {
                        uint2 u = make_uint2(0, 0);
                        if (there) u = *reinterpret_cast<const uint2*>(p);
                        v.x = u.x, v.y = u.y;
                    }
                }
            }
        };
        if (at < 0) {
            vs[0] = vs[1] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int g = 0; g < VG; ++g) vb[e][g] = make_uint4(0, 0, 0, 0);
            return;
        }
        if (key0 + 16 <= any.end && (key0 >= any.begin || key0 + 16 <= any.sink_end))
            load(std::true_type{});
        else
            load(std::false_type{});
        if constexpr (E4M3) vs[0] = c.v_scale[at + r], vs[1] = c.v_scale[at + r + 8];
    };

    float o[VG][VE / 2][NQ][4] = {};
    auto page_at = [&](int i) { return i < last ? page_of(tiles[i] * KEYS) : -2; };
    int i = first + warp, at = row_of(page_at(i), tiles[i] * KEYS), page = page_at(i + W);  // page: of the block after the next one
    load_k(at);
    load_v(at, tiles[i] * KEYS);
    for (; i < last; i += W) {
        const int key0 = tiles[i] * KEYS, at_next = row_of(page, tiles[i + W] * KEYS);
        page = page_at(i + 2 * W);
        float sc[NQ][4] = {};
#pragma unroll
        for (int j = 0; j < KP; ++j) {
            const uint32_t x[4] = {kb[0][j].x, kb[0][j].y, kb[0][j].z, kb[0][j].w};
            const uint32_t y[4] = {kb[1][j].x, kb[1][j].y, kb[1][j].z, kb[1][j].w};
#pragma unroll
            for (int t = 0; t < KW / 2; ++t) {
                uint32_t f[4];
                if constexpr (E4M3) {
                    f[0] = e4m3_to_half2<false>(x[t]), f[1] = e4m3_to_half2<false>(y[t]);
                    f[2] = e4m3_to_half2<true>(x[t]), f[3] = e4m3_to_half2<true>(y[t]);
                } else {
                    f[0] = x[2 * t], f[1] = y[2 * t], f[2] = x[2 * t + 1], f[3] = y[2 * t + 1];
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const uint32_t(&u)[2] = q[n][j * KW / 2 + t];
                    if constexpr (E4M3)
                        mma_f16(sc[n], f, u[0], u[1]);
                    else
                        mma_bf16(sc[n], f, u[0], u[1]);
                }
            }
        }
        // Scores in log2 units; -infinity where the row does not see the key
        const bool whole = key0 >= every_begin && key0 + KEYS <= every.end && at >= 0;
        float v_log[2], top[NQ][2];  // e4m3: log2 of the values' scales
#pragma unroll
        for (int n = 0; n < NQ; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // keys r, r + 8
            float k_scale = 1.f;
            v_log[e] = 0.f;
            if constexpr (E4M3) {
                k_scale = ks[e];
                const float x = lg2(vs[e]);
                v_log[e] = x < 128.f ? x : 0.f;  // a slot that no row sees may hold anything, a NaN too
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float& x = sc[n][2 * e + h];
                    x *= k_scale * scale[n][h];
                    if (!whole) {
                        const Seen v = seen_by(a, start + (8 * n + 2 * q4 + h) / G);
                        if (at < 0 || !v(key0 + 8 * e + r)) x = -INFINITY;
                    }
                    top[n][h] = fmaxf(top[n][h], x + v_log[e]);
                }
        }
        load_k(at_next);
        bool grown = false;
        auto most_of = [&](int n, int h) {  // this lane's largest score of a row
            return fmaxf(sc[n][h], sc[n][2 + h]);
        };
        auto over_lanes = [&](float x) {  // the largest of a row's eight lanes
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            return x;
        };
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[n][h] = over_lanes(top[n][h]);
                grown = grown || top[n][h] - m[n][h] > 8.f || (m[n][h] == -INFINITY && top[n][h] > m[n][h]);
                if constexpr (E4M3) grown = grown || most_of(n, h) - sum_m[n][h] > 32.f;
            }
        if (__any_sync(0xffffffffu, grown)) {
            if constexpr (E4M3) {  // once more, without the keys that have no value
                uint32_t there[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t bits = 0;
#pragma unroll
                    for (int g = 0; g < VG; ++g) bits |= vb[e][g].x | vb[e][g].y | (VB == 16 ? vb[e][g].z | vb[e][g].w : 0u);
                    there[e] = __ballot_sync(0xffffffffu, (bits & 0x7f7f7f7fu) != 0);
                }
                // key r lies with the lanes q4 = r / 2, as the first or second of their four
                const uint32_t lanes = 0x11111111u << (r >> 1);
                const bool some[2] = {((r & 1 ? there[1] : there[0]) & lanes) != 0, ((r & 1 ? there[3] : there[2]) & lanes) != 0};
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (some[e]) x = fmaxf(x, sc[n][2 * e + h] + v_log[e]);
                        top[n][h] = over_lanes(x);
                        const float next = fmaxf(sum_m[n][h], most_of(n, h));
                        l[n][h] *= ex2(sum_m[n][h] - next);
                        sum_m[n][h] = next;
                    }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float next = fmaxf(m[n][h], top[n][h]), keep = m[n][h] == next ? 1.f : ex2(m[n][h] - next);
                    m[n][h] = next;
                    if constexpr (!E4M3) l[n][h] *= keep;
#pragma unroll
                    for (int g = 0; g < VG; ++g)
#pragma unroll
                        for (int e = 0; e < VE / 2; ++e) o[g][e][n][h] *= keep, o[g][e][n][2 + h] *= keep;
                }
        }
        uint32_t w[NQ][2];  // weights as B fragments
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float shift = m[n][h] == -INFINITY ? 0.f : m[n][h];
                    if constexpr (E4M3) {
                        x[h] = fminf(ex2(sc[n][2 * e + h] + (v_log[e] - shift + kTopBits)), kMostWeight);
                        l[n][h] += ex2(sc[n][2 * e + h] - sum_m[n][h]);
                    } else {
                        x[h] = ex2(sc[n][2 * e + h] - shift);
                        l[n][h] += x[h];
                    }
                }
                if constexpr (E4M3) {
                    const __half2 v = __floats2half2_rn(x[0], x[1]);
                    w[n][e] = transpose8(*reinterpret_cast<const uint32_t*>(&v));
                } else {
                    w[n][e] = transpose8(pack_bf16x2(x[0], x[1]));
                }
            }
#pragma unroll
        for (int g = 0; g < VG; ++g) {
            const uint32_t v[4][4] = {{vb[0][g].x, vb[0][g].y, vb[0][g].z, vb[0][g].w},
                                      {vb[1][g].x, vb[1][g].y, vb[1][g].z, vb[1][g].w},
                                      {vb[2][g].x, vb[2][g].y, vb[2][g].z, vb[2][g].w},
                                      {vb[3][g].x, vb[3][g].y, vb[3][g].z, vb[3][g].w}};
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) {
                uint32_t x[4], f[4];  // values 2 e, 2 e + 1 of the four keys
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (!E4M3)
                        x[k] = v[k][e];
                    else
                        x[k] = e & 1 ? e4m3_to_half2<true>(v[k][e >> 1]) : e4m3_to_half2<false>(v[k][e >> 1]);
                }
                f[0] = __byte_perm(x[0], x[1], 0x5410), f[1] = __byte_perm(x[0], x[1], 0x7632);
                f[2] = __byte_perm(x[2], x[3], 0x5410), f[3] = __byte_perm(x[2], x[3], 0x7632);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    if constexpr (E4M3)
                        mma_f16(o[g][e][n], f, w[n][0], w[n][1]);
                    else
                        mma_bf16(o[g][e][n], f, w[n][0], w[n][1]);
                }
            }
        }
        load_v(at_next, tiles[i + W] * KEYS);
        at = at_next;
    }

    // Join the warps, row by row, in their order
    float* out = smem;
    float2* ml = reinterpret_cast<float2*>(smem + W * F::kRows * D);
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float back = 1.f;  // from the weights' maximum to the sum's
            if constexpr (E4M3) {
                float most = sum_m[n][h];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                l[n][h] *= ex2(sum_m[n][h] - most);
                back = ex2(m[n][h] - kTopBits - most);  // 0 where no key had a value
                m[n][h] = most;
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], d);
            if (E4M3 && l[n][h] == 0.f) m[n][h] = -INFINITY, back = 0.f;  // no key at all
            const int row = warp * F::kRows + 8 * n + 2 * q4 + h;
            if (r == 0) ml[row] = make_float2(m[n][h], l[n][h]);
#pragma unroll
            for (int g = 0; g < VG; ++g)
#pragma unroll
                for (int e = 0; e < VE / 2; ++e)
                    *reinterpret_cast<float2*>(out + row * D + (g * 8 + r) * VE + 2 * e) =
                        make_float2(o[g][e][n][h] * back, o[g][e][n][2 + h] * back);
        }
    __syncthreads();
    const bool part = first > 0 || last < tiles.count;
    for (int row = warp; row < rows; row += W) {  // one warp a row, D / 32 columns a lane
        constexpr int N = D / 32;
        const int t = row / G;
        const long orow = ((long)b * c.H + hk * G + row % G) * c.T + t;
        float top = -INFINITY, sum = 0.f, acc[N] = {};
        for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * F::kRows + row].x);
        for (int w = 0; w < W; ++w) {
            const float2 x = ml[w * F::kRows + row];
            if (x.x == -INFINITY && x.y == 0.f) continue;
            const float f = x.x == top ? 1.f : ex2(x.x - top);
            sum = fmaf(x.y, f, sum);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = fmaf(out[(w * F::kRows + row) * D + lane * N + j], f, acc[j]);
        }
        bool fine = fabsf(sum) < INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) fine = fine && fabsf(acc[j]) < INFINITY;
        if (row < seen_rows && !__all_sync(0xffffffffu, fine))
            attend_row<D, E4M3, KEYS>(a, b, hk, static_cast<const __nv_bfloat16*>(a.q) + orow * D, start + t, tiles, first,
                                      last, top, sum, acc);
        if (row >= seen_rows) {  // a row behind the sequence's count sees nothing
            top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.f;
        }
        if (part) {
            const long prow = place * kM + row;
#pragma unroll
            for (int j = 0; j < N; ++j) a.part[prow * D + lane * N + j] = acc[j];
            if (lane == 0) a.part_ml[prow] = make_float2(top, sum);
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int j = 0; j < N; ++j)
                static_cast<__nv_bfloat16*>(a.o)[orow * D + lane * N + j] = __float2bfloat16(acc[j] * inv);
        }
    }
    __syncthreads();  // the next head's outputs come into the same places
}

template <int D, bool E4M3, int NQ>
__global__ void __launch_bounds__(Few<D, E4M3, NQ>::kWarps * 32, 1) attend_few_kernel(AttendArgs a) {
    constexpr int W = Few<D, E4M3, NQ>::kWarps, KEYS = kBlock;
    extern __shared__ __align__(16) float smem[];  // outputs [warps][rows][D], then maxima and sums [warps][rows]
    __shared__ long warp_sums[W];
    __shared__ long found[2];  // sequence where the share's first block lies, and where its blocks begin
    const CacheArgs& c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The share: prefix sums over the sequences, first for the total, then for the share's begin
    long total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        long base = 0;
        const long x0 = total * blockIdx.x / gridDim.x;
        for (int b0 = 0; b0 < c.B; b0 += W * 32) {
            const int b = b0 + threadIdx.x;
            const long n = b < c.B ? (long)tiles_of<KEYS>(keys_of(a, b)).count * c.Hkv : 0;
            long sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long y = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += y;
            }
            __syncthreads();
            if (lane == 31) warp_sums[warp] = sum;
            __syncthreads();
            long begin = base + sum - n;
            for (int w = 0; w < W; ++w) {
                if (w < warp) begin += warp_sums[w];
                base += warp_sums[w];
            }
            if (blockIdx.x == 0 && b < c.B) {
                const int tokens = cache_count(c, b);
                if (tokens > 0 && (long)c.starts[b] + tokens > capacity(c)) atomicOr(c.status, kStatusMissingPage);
            }
            if (pass && x0 >= begin && x0 < begin + n) found[0] = b, found[1] = begin;
            if (pass && blockIdx.x == 0 && b < c.B) a.begins[b] = begin;
        }
        if (pass && blockIdx.x == 0 && threadIdx.x == 0) a.begins[c.B] = total;
        total = base;
        if (total == 0) return;  // join_kernel writes the zeros
    }
    __syncthreads();
    const long x_begin = total * blockIdx.x / gridDim.x, x_end = total * (blockIdx.x + 1) / gridDim.x;
    if (x_begin == x_end) return;
    int b = (int)found[0];
    Tiles tiles = tiles_of<KEYS>(keys_of(a, b));
    int hk = (int)((x_begin - found[1]) / tiles.count), first = (int)((x_begin - found[1]) % tiles.count);
    for (long x = x_begin; x < x_end;) {
        while (tiles.count == 0 || hk == c.Hkv) hk = 0, tiles = tiles_of<KEYS>(keys_of(a, ++b));
        const int last = (int)min((long)tiles.count, first + x_end - x);
        attend_head<D, E4M3, NQ>(a, b, hk, tiles, first, last, (long)blockIdx.x * 2 + (x > x_begin), smem);
        x += last - first;
        first = 0, ++hk;
    }
}

// The rows of the heads whose keys more than one CTA had, and of sequences without any: one warp a row. A sequence that is
// alone may have all CTAs' parts, so the lanes look up their maxima and sums at once, and the outputs are read eight at a
// time (one after the other, with their divisions, cost 30 us for one sequence of 8192 keys).
template <int D, int KEYS>
__global__ void __launch_bounds__(128) join_kernel(AttendArgs a, int ctas) {
    constexpr int N = D / 32, kEach = (kMostCtas + 31) / 32, kAhead = 8;
    const CacheArgs& c = a.c;
    const int G = c.H / c.Hkv, rows = (int)c.T * G, lane = threadIdx.x & 31;
    const unsigned at = blockIdx.x * 4 + (threadIdx.x >> 5), unit = at / (unsigned)rows;  // B * H * T is below 2^31
    if (unit >= (unsigned)c.B * c.Hkv) return;
    const int row = (int)(at % (unsigned)rows), b = (int)(unit / c.Hkv), hk = (int)(unit % c.Hkv);
    const int n = tiles_of<KEYS>(keys_of(a, b)).count;
    float sum = 0.f, acc[N] = {};
    if (n > 0) {
        const long total = a.begins[c.B], x0 = a.begins[b] + (long)hk * n;
        const int c0 = owner(x0, ctas, total), c1 = owner(x0 + n - 1, ctas, total);
        if (c0 == c1) return;  // written already
        const long place0 = 2L * c0 + (x0 > total * c0 / ctas);  // the first part ends its CTA's range, the others begin theirs
        auto place = [&](int i) { return (i == 0 ? place0 : 2L * (c0 + i)) * kM + row; };
        float2 ml[kEach];
        float top = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = 32 * k + lane, cta = c0 + i;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (cta <= c1 && total * cta / ctas != total * (cta + 1) / ctas)  // with fewer blocks than CTAs some are idle
                ml[k] = a.part_ml[place(i)];
            top = fmaxf(top, ml[k].x);
            nan = nan || ml[k].x != ml[k].x;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        nan = __any_sync(0xffffffffu, nan);
        float f[kEach];
        uint32_t there[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const bool some = !(ml[k].x == -INFINITY && ml[k].y == 0.f);
            there[k] = __ballot_sync(0xffffffffu, some);
            f[k] = !some ? 0.f : nan ? NAN : ml[k].x == top ? 1.f : ex2(ml[k].x - top);
            sum = fmaf(ml[k].y, f[k], sum);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
        for (int k = 0; k < kEach; ++k)
#pragma unroll
            for (int i0 = 0; i0 < 32; i0 += kAhead) {
                if ((there[k] >> i0 & ((1u << kAhead) - 1)) == 0) continue;
                float x[kAhead][N];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float* p = a.part + place(32 * k + i0 + i) * D + lane * N;
                    const bool is = there[k] >> (i0 + i) & 1;
                    if constexpr (N == 4) {
                        const float4 u = is ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
                        x[i][0] = u.x, x[i][1] = u.y, x[i][2] = u.z, x[i][3] = u.w;
                    } else {
                        const float2 u = is ? *reinterpret_cast<const float2*>(p) : make_float2(0.f, 0.f);
                        x[i][0] = u.x, x[i][1] = u.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float w = __shfl_sync(0xffffffffu, f[k], i0 + i);
#pragma unroll
                    for (int j = 0; j < N; ++j) acc[j] = fmaf(x[i][j], w, acc[j]);
                }
            }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long orow = ((long)b * c.H + hk * G + row % G) * c.T + row / G;
#pragma unroll
    for (int j = 0; j < N; ++j)
        static_cast<__nv_bfloat16*>(a.o)[orow * D + lane * N + j] = __float2bfloat16(acc[j] * inv);
}

template <int D, bool E4M3, int NQ>
cudaError_t launch(const AttendArgs& a, int ctas, cudaStream_t st) {
    using F = Few<D, E4M3, NQ>;
    auto* kernel = attend_few_kernel<D, E4M3, NQ>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)ctas, F::kWarps * 32, F::kBytes, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long rows = (long)a.c.B * a.c.H * a.c.T;
    join_kernel<D, kBlock><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a, ctas);
    return cudaGetLastError();
}
template <int D, bool E4M3>
cudaError_t launch(const AttendArgs& a, int ctas, cudaStream_t st) {
    return a.c.T * (a.c.H / a.c.Hkv) <= 8 ? launch<D, E4M3, 1>(a, ctas, st) : launch<D, E4M3, 2>(a, ctas, st);
}

// One CTA an SM, and at least 16 blocks of the longest possible sequences each, two a warp.
int ctas_for(int B, int Hkv, long longest) {
    return (int)std::max(1L, std::min((long)kMostCtas, (longest / 16 * B * Hkv + 15) / 16));
}

}  // namespace

bool attend_few_rows(int H, int Hkv, long T) { return T * (H / Hkv) <= kM; }

size_t attend_few_bytes(int B, int Hkv, int d, long longest) {
    const size_t places = (size_t)ctas_for(B, Hkv, longest) * 2 * kM;
    return places * (d * sizeof(float) + sizeof(float2)) + ((size_t)B + 1) * sizeof(long);
}

cudaError_t launch_attend_few(const AttendArgs& args, bool e4m3, void* workspace, long longest, cudaStream_t st) {
    AttendArgs a = args;
    const int ctas = ctas_for(a.c.B, a.c.Hkv, longest);
    const size_t places = (size_t)ctas * 2 * kM;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + places * a.c.d);
    a.begins = reinterpret_cast<long*>(a.part_ml + places);
    if (a.c.d == 64) return e4m3 ? launch<64, true>(a, ctas, st) : launch<64, false>(a, ctas, st);
    return e4m3 ? launch<128, true>(a, ctas, st) : launch<128, false>(a, ctas, st);
}

}  // namespace titans
