// Attention of a chunk of new tokens over the paged cache, in one pass over the keys with a running maximum and sum.
//
// The query heads that share a key/value head read the same keys, so the rows of a tile are (token, head) pairs of
// one key/value head: row r of it is token r / G, head r % G. A CTA has NT tiles of 128 rows and walks over tiles of
// 128 keys:
//   S = Q K^T       tcgen05, both operands in shared memory, S in TMEM
//   P = exp2(c S - c m), rounded to bf16 and written over S in TMEM; one thread a row
//   O += P V        tcgen05, P from TMEM, O in TMEM
// Keys and values come from their pages in the layouts that the MMA reads: a bf16 cache by TMA, one box per page and 64
// columns, issued by one warp; an e4m3 cache through eight warps that convert and scale it (both exact in
// bf16). Values that no row of the tile sees are zeroed. One thread issues the MMAs: with two tiles, the softmax of
// one runs while the tensor core works for the other. Tiles of 64 keys with two places for S, so that the next scores are there
// before this tile's weights are, took 287 us where this form takes 280.
//
// 2 x 2048 tokens of 16 heads on 4, d = 128, over 10,000 bf16 keys: 277 us, 268 GFLOP, 0.58 of cuBLAS's bf16 rate. A tile's two
// products take 1024 cycles of the tensor core and its exponentials 1024 of the MUFU; each row's softmax waits for its scores in between.
//
// O is rescaled in TMEM only when a row's maximum has grown by more than 2^8 since the one its weights refer to: the
// weights stay below 2^8, which neither bf16 nor the fp32 sums mind, and most tiles need no pass over O.
//
// A masked weight is 0, but 0 times an infinity or NaN that another row of the tile does see is NaN. Rows that come
// out non-finite are therefore taken again key by key over just what they see (attend_row).
//
// Where there are few tiles of rows the keys are split over CTAs, each of which leaves its sum, maximum and unnormalised output in the
// workspace for combine_kernel.
#include <algorithm>
#include <type_traits>

#include "cache_attend.cuh"
#include "ptx.cuh"

namespace titans {
namespace {

constexpr int kKeys = 128;  // keys of a tile
constexpr int kRows = 128;  // rows of a tile
constexpr float kLazy = 8.f;

template <int D, int NT, int STAGES>
struct Shared {
    __nv_bfloat16 q[NT][kRows * D];  // per tile D / 64 panels of 64 columns, 128-byte swizzle
    __nv_bfloat16 k[STAGES][kKeys * D], v[STAGES][kKeys * D];
    uint32_t valid[STAGES][4];  // keys of the stage that some row sees and whose page is there
    int at[2][kKeys];           // e4m3: rows of the pool of the tile being fetched, in turn
    uint64_t q_full, full[STAGES], raw[STAGES], empty[STAGES], s_full[NT], p_full[NT][2], done;
    float share[NT][2][kRows];  // what the two threads of a row tell one another
    int bad[NT][kRows];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// umma_bf16 with A [128][16] in TMEM: lane = row, a 32-bit column holds two neighbouring K elements.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void bar_sync_producers(int threads) {
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}
// Box of the tensor map at column x, row y.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}

// Eight e4m3 values times their scale as bf16: both steps exact.
__device__ __forceinline__ uint4 to_bf16(uint32_t lo, uint32_t hi, float s) {
    const float2 a = e4m3_to_float2<false>(lo), b = e4m3_to_float2<true>(lo);
    const float2 c = e4m3_to_float2<false>(hi), d = e4m3_to_float2<true>(hi);
    return make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s), pack_bf16x2(c.x * s, c.y * s),
                      pack_bf16x2(d.x * s, d.y * s));
}

// Bits of the 32 keys from k0 on that lie in lo..end-1.
__device__ __forceinline__ uint32_t range_mask(int k0, int lo, int end) {
    const int a = max(0, min(32, lo - k0)), e = max(0, min(32, end - k0));
    const uint32_t below_a = a == 32 ? 0xffffffffu : (1u << a) - 1, below_e = e == 32 ? 0xffffffffu : (1u << e) - 1;
    return below_e & ~below_a;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Largest of 64 values in registers, in four chains.
__device__ __forceinline__ float max64(const uint32_t (&x)[32], const uint32_t (&y)[32], float top) {
    float t[4] = {top, top, top, top};
#pragma unroll
    for (int e = 0; e < 32; e += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = max3(t[i], __uint_as_float(x[e + i]), __uint_as_float(y[e + i]));
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// Warps of a CTA in groups of four: NT * kPair of softmax, one group whose first warp issues the MMAs and whose
// second one brings a bf16 cache, and for an e4m3 cache two that convert it. kPair = 2: two threads share a row, 64
// keys each, whose chain is half as long; two tiles over an e4m3 cache would have 896 threads of 72 registers then, too few for 64 scores.
// All forms but one tile over a bf16 cache spill some (84 to 128 bytes a thread stored).
// Where the launch leaves softmax too few registers it takes over some that the others do not need; what a
// thread has at launch times the threads covers the new shares (launch() checks it).
template <bool E4M3, int NT>
struct Plan {
    static constexpr int kPair = E4M3 && NT == 2 ? 1 : 2;
    static constexpr int kSoftmax = NT * kPair * 128, kProducers = E4M3 ? 256 : 32;  // threads
    static constexpr int kThreads = kSoftmax + 128 + (E4M3 ? 256 : 0);
    static constexpr int kSoftmaxRegs = NT == 1 ? 0 : E4M3 ? 136 : 104;  // 0: as launched
    static constexpr int kIssueRegs = E4M3 ? 56 : 64, kProducerRegs = 72;
    static constexpr int kShares = kSoftmax * kSoftmaxRegs + 128 * kIssueRegs + (E4M3 ? 256 * kProducerRegs : 0);
};

// The sequence with `place` longer ones, out of at most 32, a lane each.
__device__ __forceinline__ int by_length(const CacheArgs& c, int place, int lane) {
    const int end = lane < c.B ? max(c.starts[lane], -1) / 2 + cache_count(c, lane) / 2 : -1;  // halves: no overflow
    int rank = 0;
    for (int i = 0; i < c.B; ++i) {
        const int other = __shfl_sync(0xffffffffu, end, i);
        rank += other > end || (other == end && i < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < c.B && rank == place)) - 1;
}

template <int D, bool E4M3, int NT, int STAGES>
__global__ void __launch_bounds__(Plan<E4M3, NT>::kThreads, 1)
    attend_kernel(AttendArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using P = Plan<E4M3, NT>;
    constexpr int kMmaWarp = P::kSoftmax / 32, kProducer0 = E4M3 ? kMmaWarp + 4 : kMmaWarp + 1;
    using S = Shared<D, NT, STAGES>;
    constexpr int kPanel = kKeys * 128;  // bytes of a panel of 64 columns
    constexpr uint32_t kColumns = NT == 1 ? 256 : 512;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    S& s = *reinterpret_cast<S*>(smem_raw);
    const CacheArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = c.H / c.Hkv;
    const long rows = c.T * G;  // of one key/value head
    // The CTAs with the most keys start first: of up to 32 sequences the longest one, and of a sequence the last rows
    const int hk = blockIdx.x % c.Hkv, per = (int)((rows + NT * kRows - 1) / (NT * kRows)), place = blockIdx.x / c.Hkv / per;
    const int b = c.B <= 32 ? by_length(c, place, lane) : place;
    const long row0 = (long)(per - 1 - blockIdx.x / c.Hkv % per) * (NT * kRows);
    const int count = cache_count(c, b);
    const long start = c.starts[b];
    const long t_lo = row0 / G, t_hi = min(min(row0 + NT * kRows, rows) - 1, (long)count * G - 1) / G;
    Tiles tiles{0, 0, 0};
    Seen seen_any{0, 0, 0};  // keys that some row of the CTA sees
    if (row0 < (long)count * G) {
        seen_any = seen_by_any(a, start + t_lo, start + t_hi);
        tiles = tiles_of<kKeys>(seen_any);
        if (tid == 0 && start + t_hi >= capacity(c)) atomicOr(c.status, kStatusMissingPage);
    }
    const int first = (int)((long)tiles.count * blockIdx.z / gridDim.z);
    const int last = (int)((long)tiles.count * (blockIdx.z + 1) / gridDim.z), n = last - first;

    if (warp == kMmaWarp) {
        tmem_alloc(&s.tmem, kColumns);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(&s.q_full, P::kSoftmax);
        for (int i = 0; i < STAGES; ++i)
            mbar_init(&s.full[i], E4M3 ? P::kProducers : 1), mbar_init(&s.raw[i], 1), mbar_init(&s.empty[i], 1);
        for (int i = 0; i < NT; ++i) mbar_init(&s.s_full[i], 1), mbar_init(&s.p_full[i][0], P::kPair * 128), mbar_init(&s.p_full[i][1], P::kPair * 128);
        mbar_init(&s.done, 1);
        s.abort = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int* abort_flag = &s.abort;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!*abort_flag && mbar_wait(bar, parity)) return true;
        *abort_flag = 1;
        atomicOr(c.status, kStatusTimeoutMma);
        return false;
    };
    // The same for a whole warp, whose lanes agree on the outcome.
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };

    if (warp < kMmaWarp) {  // --------------------------------------------------- softmax: one or two threads a row
        if constexpr (P::kSoftmaxRegs > 0) registers_up<P::kSoftmaxRegs>();
        constexpr bool kTwo = P::kPair == 2;
        constexpr int kChunks = kTwo ? 2 : 4;          // 32 keys each
        constexpr int kOut = D / 32 / P::kPair;        // 32 columns of the output each
        const int tile = warp / (4 * P::kPair), half = kTwo ? (warp >> 2) & 1 : 0, r = (warp & 3) * 32 + lane;
        const long row = row0 + tile * kRows + r;
        const int t = (int)(row / G), h = hk * G + (int)(row % G);
        const bool live = row < rows && t < count;
        const bool any = __any_sync(0xffffffffu, live);
        const long p = start + t, out = (((long)b * c.H + h) * c.T + t) * D;
        const float sign = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
        const float scale = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * 1.44269504f;
        if (n > 0) {
            // the row of Q; a scale that is not positive goes into its sign, so that the largest score is the largest weight's
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + out;
            const uint32_t base = smem_u32(s.q[tile]);
#pragma unroll 4
            for (int i = half * kOut * 4; i < (half + 1) * kOut * 4; ++i) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live) u = *reinterpret_cast<const uint4*>(q + 8 * i);
                uint32_t w[4] = {u.x, u.y, u.z, u.w};
                if (sign < 0.f)
                    for (int e = 0; e < 4; ++e) w[e] ^= 0x80008000u;
                if (sign == 0.f) w[0] = w[1] = w[2] = w[3] = 0;
                st_shared_v4(base + (i >> 3) * kPanel + sw128_off(r, (i & 7) * 8), w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            arrive(&s.q_full);
        }
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32 lanes of TMEM a warp
        const uint32_t ts = tmem + lane_base + tile * 128 + half * 64, tp = tmem + lane_base + tile * 128 + half * 32;
        const uint32_t to = tmem + lane_base + NT * 128 + tile * D + half * kOut * 32;
        auto pair_sync = [&] {  // the two warps that share 32 rows
            if constexpr (kTwo) asm volatile("bar.sync %0, 64;" ::"r"(2 + tile * 4 + (warp & 3)) : "memory");
        };
        const Seen seen = seen_by(a, p);
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int stage = j % STAGES;
            ok = ok && wait_warp(&s.s_full[tile], j & 1);
            if (!ok) {  // given up, but the other warp of the rows may wait for this one
                if (any) pair_sync();
                continue;
            }
            tc_fence_after();
            if (!any) {
                tc_fence_before();
                arrive(&s.p_full[tile][0]);
                arrive(&s.p_full[tile][1]);
                continue;
            }
            // all of a thread's scores in registers where it has 64, else 64 at a time, read twice
            uint32_t x[2][32];
            tmem_ld32(ts, x[0]);
            tmem_ld32(ts + 32, x[1]);
            const int k0 = tiles[first + j] * kKeys;
            const bool whole = k0 >= seen.begin && k0 + kKeys <= seen.end &&
                               (s.valid[stage][0] & s.valid[stage][1] & s.valid[stage][2] & s.valid[stage][3]) == ~0u;
            const bool all_whole = __all_sync(0xffffffffu, whole || !live);
            uint32_t mask[kChunks];
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                mask[i] = ~0u;
                if (!all_whole) {
                    const int kc = k0 + 32 * (i + 2 * half);
                    mask[i] = (range_mask(kc, seen.begin, seen.end) | range_mask(kc, 0, min(seen.sink_end, seen.end))) & s.valid[stage][i + 2 * half];
                }
            }
            auto masked = [&](uint32_t(&v)[32], uint32_t bits) {  // -infinity where the row does not see the key
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = bits >> e & 1 ? v[e] : 0xff800000u;
            };
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kChunks; i += 2) {
                if (i > 0) tmem_ld32(ts + 32 * i, x[0]), tmem_ld32(ts + 32 * i + 32, x[1]);
                tmem_wait_ld();
                if (!all_whole) masked(x[0], mask[i]), masked(x[1], mask[i + 1]);
                top = max64(x[0], x[1], top);
            }
            if constexpr (kTwo) {  // the other half's; and the scores that P will overwrite have been read
                s.share[tile][half][r] = top;
                pair_sync();
                top = fmaxf(top, s.share[tile][half ^ 1][r]);
            }
            const bool grown = j == 0 || (top - m) * scale > kLazy || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, grown)) {
                const float next = fmaxf(m, top);
                const float keep = m == next ? 1.f : ex2((m - next) * scale);
                m = next;
                l *= keep;
                if (j > 0) {
#pragma unroll
                    for (int i = 0; i < 2 * kOut; ++i) {
                        uint32_t o[16];
                        tmem_ld16(to + 16 * i, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                        tmem_st16(to + 16 * i, o);
                    }
                }
            }
            const float shift = m == -INFINITY ? 0.f : m * scale;
            float sum[4] = {};
            auto weights = [&](auto whole_tile) {
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    if (!kTwo && i % 2 == 0) {
                        tmem_ld32(ts + 32 * i, x[0]), tmem_ld32(ts + 32 * i + 32, x[1]);
                        tmem_wait_ld();
                        if constexpr (!whole_tile.value) masked(x[0], mask[i]), masked(x[1], mask[i + 1]);
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float y[2];
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const float u = fmaf(__uint_as_float(x[i & 1][e + f]), scale, -shift);
                            y[f] = ex2(u);
                            sum[(e & 2) + f] += y[f];
                        }
                        w[e / 2] = pack_bf16x2(y[0], y[1]);
                    }
                    tmem_st16(tp + 16 * i, w);
                    if (i == kChunks / 2 - 1 || i == kChunks - 1) {  // half of the weights: the MMA may begin
                        tmem_wait_st();
                        tc_fence_before();
                        arrive(&s.p_full[tile][i == kChunks - 1]);
                    }
                }
            };
            if (all_whole)
                weights(std::true_type{});
            else
                weights(std::false_type{});
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (n > 0 && ok) ok = wait_warp(&s.done, 0);
        tc_fence_after();
        // The row's output, or its part of it
        const bool partial = gridDim.z > 1;
        const long prow = (((long)blockIdx.z * c.B + b) * c.H + h) * c.T + t;
        float m2 = m * scale;
        if constexpr (kTwo) {
            pair_sync();  // the last maxima have been read
            s.share[tile][half][r] = l;
            pair_sync();
            l = s.share[tile][0][r] + s.share[tile][1][r];
        }
        if (any) {
            const float inv = partial || l == 0.f ? 1.f : 1.f / l;
            bool fine = l == l && l < INFINITY;
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                uint32_t o[32];
                if (n > 0 && ok) {
                    tmem_ld32(to + 32 * i, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float v = n > 0 && ok ? __uint_as_float(o[e]) * inv : 0.f;
                    fine = fine && fabsf(v) < INFINITY;
                    o[e] = __float_as_uint(v);
                }
                if (!live || !ok) continue;
                const int col = (half * kOut + i) * 32;
                if (partial) {
                    uint4* dst = reinterpret_cast<uint4*>(a.part + prow * D + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + out + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            w[f] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * f]), __uint_as_float(o[8 * e + 2 * f + 1]));
                        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            fine = fine || !live || n == 0 || !ok;
            if constexpr (kTwo) {
                if (half) s.bad[tile][r] = !fine;
                pair_sync();  // also: what the other half stored comes before what is stored below
                fine = half || (fine && !s.bad[tile][r]);
            }
            uint32_t again = __ballot_sync(0xffffffffu, !fine);
            __syncwarp();
            while (again) {  // rows that infinities or NaN reached, maybe through keys that they do not see
                const int who = __ffs(again) - 1;
                again &= again - 1;
                const long wq = __shfl_sync(0xffffffffu, out, who), wp = __shfl_sync(0xffffffffu, p, who);
                const long wprow = __shfl_sync(0xffffffffu, prow, who);
                float rm, rl, acc[D / 32];
                attend_row<D, E4M3, kKeys>(a, b, hk, static_cast<const __nv_bfloat16*>(a.q) + wq, wp, tiles, first, last, rm, rl, acc);
                const float rinv = partial || rl == 0.f ? 1.f : 1.f / rl;
                if (lane == who) m2 = rm, l = rl;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    if (partial)
                        a.part[wprow * D + lane * (D / 32) + i] = acc[i];
                    else
                        static_cast<__nv_bfloat16*>(a.o)[wq + lane * (D / 32) + i] = __float2bfloat16(acc[i] * rinv);
                }
            }
        }
        if (half == 0) {
            if (partial) {
                if (row < rows) a.part_ml[prow] = live ? make_float2(m2, l) : make_float2(-INFINITY, 0.f);
            } else if (row < rows && !live) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + out);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
            }
        }
    } else if (E4M3 ? warp >= kProducer0 : warp == kProducer0) {  // ------------- producers
        if constexpr (P::kSoftmaxRegs > 0) registers_down<E4M3 ? P::kProducerRegs : P::kIssueRegs>();
        // keys that no row of the CTA sees are neither looked up nor read
        bool ok = true;
        if constexpr (!E4M3) {  // one warp
            int raw_uses[STAGES] = {}, last_parity[STAGES];
            uint64_t* last_bar[STAGES] = {};
            const int page = 1 << c.page_shift, per_tile = kKeys >> c.page_shift;
            for (int j = 0; j < n && ok; ++j) {
                const int stage = j % STAGES;
                const int k0 = tiles[first + j] * kKeys;
                // one lane a page: is any of its keys needed, and where does it lie
                int y = -1;
                if (lane < per_tile) {
                    const int key = k0 + (lane << c.page_shift);
                    // the page's keys that are needed are its first ones (sinks, up to the end) or its last ones (window)
                    if (key < seen_any.end && (seen_any(key) || seen_any(min(key + page, seen_any.end) - 1))) {
                        const long r = cache_row(c, b, hk, key);
                        if (r >= 0)
                            y = (int)r;
                        else
                            atomicOr(c.status, kStatusMissingPage);
                    }
                }
                const uint32_t pages = __ballot_sync(0xffffffffu, y >= 0);
                uint32_t valid[4], all = ~0u;  // lane's key 32 i + lane
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = 32 * i + lane;
                    valid[i] = __ballot_sync(0xffffffffu, seen_any(k0 + key) && (pages >> (key >> c.page_shift) & 1));
                    all &= valid[i];
                }
                if (j >= STAGES && !(ok = wait_warp(&s.empty[stage], (j / STAGES - 1) & 1))) break;
                uint64_t* bar = all == ~0u ? &s.full[stage] : &s.raw[stage];
                last_bar[stage] = bar, last_parity[stage] = (all == ~0u ? j / STAGES : raw_uses[stage]) & 1;
                if (lane < 4) s.valid[stage][lane] = lane == 0 ? valid[0] : lane == 1 ? valid[1] : lane == 2 ? valid[2] : valid[3];
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(pages) * page * D * 4);
                __syncwarp();
                if (y >= 0) {
                    const uint32_t at = (uint32_t)(lane << c.page_shift) * 128;
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        tma_load_2d(smem_u32(s.k[stage]) + x * kPanel + at, &k_map, bar, x * 64, y);
                        tma_load_2d(smem_u32(s.v[stage]) + x * kPanel + at, &v_map, bar, x * 64, y);
                    }
                }
                if (all == ~0u) continue;
                // values that no row sees become zeros before the MMA reads the stage; their scores are masked
                if (!(ok = wait_warp(&s.raw[stage], raw_uses[stage]++ & 1))) break;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    for (uint32_t dead = ~valid[i]; dead; dead &= dead - 1) {
                        const int key = 32 * i + __ffs(dead) - 1;
                        if (lane < D / 8)
                            st_shared_v4(smem_u32(s.v[stage]) + (lane >> 3) * kPanel + key * 128 + (lane & 7) * 16, 0, 0, 0, 0);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&s.full[stage]);
            }
            if (!ok)  // given up: the copies in flight still land here
                for (int i = 0; i < STAGES; ++i)
                    if (last_bar[i]) mbar_wait(last_bar[i], last_parity[i]);
        } else {
            constexpr int LANES = D / 16, PASSES = kKeys * LANES / P::kProducers;  // 16 bytes a lane
            const int i0 = tid - kProducer0 * 32, sub = i0 % LANES, group = i0 / LANES;
            for (int j = 0; j < n; ++j) {  // to the end in any case: the barrier below takes all threads
                const int stage = j % STAGES;
                int* rows_at = s.at[j & 1];
                uint32_t there = 0;
                if (i0 < kKeys) {
                    const int key = tiles[first + j] * kKeys + i0;
                    long at = -1;
                    if (seen_any(key)) {
                        at = cache_row(c, b, hk, key);
                        if (at < 0) atomicOr(c.status, kStatusMissingPage);
                    }
                    rows_at[i0] = (int)at;
                    there = __ballot_sync(0xffffffffu, at >= 0);
                }
                bar_sync_producers(P::kProducers);
                uint4 kx[PASSES], vx[PASSES];
                float ks[PASSES], vs[PASSES];
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {  // in flight while the stage is still read
                    const long r = rows_at[i * (P::kProducers / LANES) + group];
                    kx[i] = vx[i] = make_uint4(0, 0, 0, 0), ks[i] = vs[i] = 0.f;
                    if (r >= 0) {
                        kx[i] = static_cast<const uint4*>(c.pk)[r * LANES + sub], ks[i] = c.k_scale[r];
                        vx[i] = static_cast<const uint4*>(c.pv)[r * LANES + sub], vs[i] = c.v_scale[r];
                    }
                }
                if (j >= STAGES && ok) ok = wait(&s.empty[stage], (j / STAGES - 1) & 1);
                if (!ok) continue;
                if (i0 < kKeys && lane == 0) s.valid[stage][i0 >> 5] = there;
                const uint32_t off = (sub >> 2) * kPanel, col = (sub & 3) * 16;
                const uint32_t kb = smem_u32(s.k[stage]) + off, vb = smem_u32(s.v[stage]) + off;
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int r = i * (P::kProducers / LANES) + group;
                    uint4 w = to_bf16(kx[i].x, kx[i].y, ks[i]);
                    st_shared_v4(kb + sw128_off(r, col), w.x, w.y, w.z, w.w);
                    w = to_bf16(kx[i].z, kx[i].w, ks[i]);
                    st_shared_v4(kb + sw128_off(r, col + 8), w.x, w.y, w.z, w.w);
                    w = to_bf16(vx[i].x, vx[i].y, vs[i]);
                    st_shared_v4(vb + sw128_off(r, col), w.x, w.y, w.z, w.w);
                    w = to_bf16(vx[i].z, vx[i].w, vs[i]);
                    st_shared_v4(vb + sw128_off(r, col + 8), w.x, w.y, w.z, w.w);
                }
                fence_proxy_async_smem();
                arrive(&s.full[stage]);
            }
        }
    } else if (warp != kMmaWarp) {
        if constexpr (P::kSoftmaxRegs > 0) registers_down<P::kIssueRegs>();
    } else {  // ---------------------------------------------------------------- one thread issues the MMAs
        if constexpr (P::kSoftmaxRegs > 0) registers_down<P::kIssueRegs>();
        // The whole warp walks the loop and one elected lane issues: what the MMAs take then stays in uniform registers,
        // without which issuing them takes longer than they do.
        const int steps = __shfl_sync(0xffffffffu, n, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const bool lead = elect_one();
        const uint32_t id_s = idesc_bf16_f32(128, kKeys, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
        // descriptors of the first tile and stage; an offset in bytes is added as its sixteenth
        const uint64_t q0 = sdesc_sw128(smem_u32(s.q[0]), 16, 1024), kd0 = sdesc_sw128(smem_u32(s.k[0]), 16, 1024);
        const uint64_t v0 = sdesc_sw128(smem_u32(s.v[0]), kPanel, 1024);
        constexpr uint32_t kTile = kKeys * D * 2 / 16;
        auto scores = [&](int i, int stage) {
            const uint64_t k = kd0 + stage * kTile;
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * kPanel + (ks & 3) * 32) / 16;
                    umma_bf16(tm + i * 128, q0 + i * kTile + off, k + off, id_s, ks > 0);
                }
                umma_commit(&s.s_full[i]);
            }
            __syncwarp();
        };
        bool ok = true;
        if (steps > 0) {
            ok = wait_warp(&s.q_full, 0) && wait_warp(&s.full[0], 0);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < NT; ++i) scores(i, 0);
            }
        }
        int stage = 0, next = 1, next_phase = 0;  // of the tile after this one
        for (int j = 0; j < steps && ok; ++j) {
            const uint64_t v = v0 + stage * kTile;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // the halves of P in the order in which they are written
                    ok = ok && wait_warp(&s.p_full[i][part], j & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (lead) {
#pragma unroll
                        for (int u = 0; u < kKeys / 32; ++u) {
                            const int ks = P::kPair == 2 ? (u & 1) + 2 * part + (u >> 1) * 4 : u + 4 * part;
                            umma_bf16_ts(tm + NT * 128 + i * D, tm + i * 128 + ks * 8, v + ks * 128, id_o,
                                         part > 0 || u > 0 ? 1u : j > 0);
                        }
                        if (part == 1 && i == NT - 1) umma_commit(j + 1 < steps ? &s.empty[stage] : &s.done);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (j + 1 < steps) {
                    if (i == 0) {
                        if (!(ok = wait_warp(&s.full[next], next_phase))) break;
                        tc_fence_after();
                    }
                    scores(i, next);
                }
            }
            stage = next;
            if (++next == STAGES) next = 0, next_phase ^= 1;
        }
        // Nothing of this CTA may still be at work when its TMEM is freed, an aborted pass's MMAs neither.
        if (!ok) {
            if (lead) umma_commit(&s.done);
            __syncwarp();
            mbar_wait(&s.done, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kColumns);
    }
}

// Joins the parts of a row: one warp a row.
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(AttendArgs a, int splits) {
    constexpr int N = D / 32;
    const CacheArgs& c = a.c;
    const long rows = (long)c.B * c.H * c.T, row = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    float m = -INFINITY;
    bool nan = false;
    for (int s = 0; s < splits; ++s) {
        const float x = a.part_ml[s * rows + row].x;
        m = fmaxf(m, x);
        nan = nan || x != x;
    }
    float l = 0.f, acc[N] = {};
    for (int s = 0; s < splits; ++s) {
        const float2 ml = a.part_ml[s * rows + row];
        if (ml.x == -INFINITY && ml.y == 0.f) continue;
        const float w = ml.x == m ? 1.f : exp2f(ml.x - m);
        l = fmaf(ml.y, w, l);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(a.part[(s * rows + row) * D + lane * N + i], w, acc[i]);
    }
    const float inv = nan ? NAN : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < N; ++i)
        static_cast<__nv_bfloat16*>(a.o)[row * D + lane * N + i] = __float2bfloat16(acc[i] * inv);
}

// The bf16 pool as [num_pages * Hkv * page][d], boxes of one page and 64 columns.
bool encode_pool(CUtensorMap* m, const CacheArgs& c, const void* pool) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess && q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)c.d, ((cuuint64_t)c.num_pages * c.Hkv) << c.page_shift};
    const cuuint64_t strides[1] = {(cuuint64_t)c.d * 2};
    const cuuint32_t box[2] = {64, 1u << c.page_shift}, ones[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3, int NT>
cudaError_t launch(const AttendArgs& a, int splits, cudaStream_t st) {
    constexpr int STAGES = D == 64 ? 4 : NT == 1 ? 3 : 2;
    using S = Shared<D, NT, STAGES>;
    static_assert(sizeof(S) <= 227 * 1024, "fits an SM");
    auto* kernel = attend_kernel<D, E4M3, NT, STAGES>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S));
    if (e != cudaSuccess) return e;
    const long rows = a.c.T * (a.c.H / a.c.Hkv);
    const dim3 grid((unsigned)((rows + NT * kRows - 1) / (NT * kRows) * a.c.B * a.c.Hkv), 1, (unsigned)splits);
    if constexpr (Plan<E4M3, NT>::kSoftmaxRegs > 0) {
        static const bool enough = [&] {
            cudaFuncAttributes f;
            return cudaFuncGetAttributes(&f, kernel) == cudaSuccess &&
                   f.numRegs * Plan<E4M3, NT>::kThreads >= Plan<E4M3, NT>::kShares;
        }();
        if (!enough) return cudaErrorInvalidConfiguration;
    }
    CUtensorMap k_map{}, v_map{};
    if (!E4M3 && (!encode_pool(&k_map, a.c, a.c.pk) || !encode_pool(&v_map, a.c, a.c.pv))) return cudaErrorInvalidValue;
    kernel<<<grid, Plan<E4M3, NT>::kThreads, sizeof(S), st>>>(a, k_map, v_map);
    return cudaGetLastError();
}

// How the rows and keys are shared out: tiles of rows a CTA, and splits of the keys. One CTA fits an SM, and more splits than
// fill one round of them only add parts to join (128 rows of 16 heads, 8192 keys: 35 us with 148 CTAs at most, 48 us with
// 296); a split has no less than four tiles of the longest possible sequence, the lengths themselves are on the device.
// A CTA with two tiles of rows takes about 1.45 times as long as one with one, so it is the choice where it does not leave too many SMs
// idle. 2048 tokens of 16 heads on 4, 8000 keys, two tiles in one round against one tile in two: bf16 139 against 192 us at d = 128 and
// 127 against 164 at d = 64, e4m3 187 against 264 and 156 against 197: factors of 1.42 to 1.59, which choose alike but for
// batches of two against three rounds.
struct Shares {
    int tiles, splits;
};
Shares shares(int B, int H, int Hkv, long T, long longest) {
    const long rows = T * (H / Hkv), most = std::min(64L, (longest + 4 * kKeys - 1) / (4 * kKeys));
    auto splits = [&](long ctas) { return std::max(1L, std::min(most, kSms / ctas)); };
    auto rounds = [&](long ctas) { return (double)((ctas * splits(ctas) + kSms - 1) / kSms) / splits(ctas); };
    const long one = (rows + kRows - 1) / kRows * B * Hkv, two = (rows + 2 * kRows - 1) / (2 * kRows) * B * Hkv;
    return 1.45 * rounds(two) < rounds(one) ? Shares{2, (int)splits(two)} : Shares{1, (int)splits(one)};
}

}  // namespace

size_t attend_workspace_bytes(int B, int H, int Hkv, long T, int d, long longest) {
    if (attend_few_rows(H, Hkv, T)) return attend_few_bytes(B, Hkv, d, longest);
    const int splits = shares(B, H, Hkv, T, longest).splits;
    return splits == 1 ? 0 : (size_t)splits * B * H * T * (d * sizeof(float) + sizeof(float2));
}

cudaError_t launch_cache_attend(const AttendArgs& args, bool e4m3, void* workspace, long longest, cudaStream_t st) {
    if (attend_few_rows(args.c.H, args.c.Hkv, args.c.T)) return launch_attend_few(args, e4m3, workspace, longest, st);
    AttendArgs a = args;
    const auto [tiles, splits] = shares(a.c.B, a.c.H, a.c.Hkv, a.c.T, longest);
    const size_t n = (size_t)splits * a.c.B * a.c.H * a.c.T;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + (splits > 1 ? n * a.c.d : 0));
    const bool two = tiles == 2;
    cudaError_t e;
    if (a.c.d == 64) {
        e = e4m3 ? (two ? launch<64, true, 2>(a, splits, st) : launch<64, true, 1>(a, splits, st))
                 : (two ? launch<64, false, 2>(a, splits, st) : launch<64, false, 1>(a, splits, st));
    } else {
        e = e4m3 ? (two ? launch<128, true, 2>(a, splits, st) : launch<128, true, 1>(a, splits, st))
                 : (two ? launch<128, false, 2>(a, splits, st) : launch<128, false, 1>(a, splits, st));
    }
    if (e != cudaSuccess || splits == 1) return e;
    auto* kernel = a.c.d == 64 ? combine_kernel<64> : combine_kernel<128>;
    kernel<<<(unsigned)(((long)a.c.B * a.c.H * a.c.T + 3) / 4), 128, 0, st>>>(a, splits);
    return cudaGetLastError();
}

}  // namespace titans
