// Attention of a chunk of new tokens over the paged cache, in one pass over the keys with a running maximum and sum.
//
// The query heads that share a key/value head read the same keys, so the rows of a tile are (token, head) pairs of
// one key/value head: row r of it is token r / G, head r % G. A CTA has NT tiles of 128 rows and walks over tiles of
// 128 keys:
//   S = Q K^T       tcgen05, both operands in shared memory, S in TMEM
//   P = exp2(c S - c m), rounded to bf16 and written over S in TMEM; one thread a row
//   O += P V        tcgen05, P from TMEM, O in TMEM
// Four producer warps gather keys and values from their pages into the layouts that the MMA reads, an e4m3 cache
// converted and scaled on the way (both exact in bf16), what no row sees as zeros. One thread issues the MMAs: with
// two tiles, the softmax of one runs while the tensor core works for the other.
//
// O is rescaled in TMEM only when a row's maximum has grown by more than 2^8 since the one its weights refer to: the
// weights stay below 2^8, which neither bf16 nor the fp32 sums mind, and most tiles need no pass over O.
//
// A masked weight is 0, but 0 times an infinity or NaN that another row of the tile does see is NaN. Rows that come
// out non-finite are therefore taken again key by key over just what they see (attend_row).
//
// With few rows the keys are split over CTAs, each of which leaves its sum, maximum and unnormalised output in the
// workspace for combine_kernel.
#include <algorithm>

#include "cache.h"
#include "ptx.cuh"

namespace titans {
namespace {

constexpr int kKeys = 128;  // keys of a tile
constexpr int kRows = 128;  // rows of a tile
constexpr float kLazy = 8.f;

// The keys that the row at position p sees: j < sink_end, or begin <= j <= p.
struct Seen {
    long begin, sink_end;
};
__device__ __forceinline__ Seen seen_by(const AttendArgs& a, long p) {
    const long begin = a.window ? max(0L, p - a.window + 1) : 0L;
    return {begin, min((long)a.sinks, begin)};
}

// The tiles of keys that rows at positions p0..p1 see: 0..head-1 and tail..end-1.
struct Tiles {
    int head, tail, count;
    __device__ int operator[](int i) const { return i < head ? i : tail + i - head; }
};
__device__ __forceinline__ Tiles tiles_of(const AttendArgs& a, long p0, long p1) {
    Tiles t{0, 0, 0};
    if (p1 < 0) return t;
    const long end = p1 / kKeys + 1;
    t.tail = (int)(seen_by(a, max(p0, 0L)).begin / kKeys);
    // the last row has the widest view of the sinks: those before its own window
    t.head = (int)min((long)t.tail, (seen_by(a, p1).sink_end + kKeys - 1) / kKeys);
    t.count = t.head + (int)end - t.tail;
    return t;
}

// N consecutive values of a row of the pool.
template <int N, bool E4M3>
__device__ __forceinline__ void load_row(const void* pool, const float* scales, long row, int col, int D, float (&x)[N]) {
    if constexpr (E4M3) {
        const float s = scales[row];
        const uint16_t* p = reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(pool) + row * D + col);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = e4m3x2_to_float2(p[i]);
            x[2 * i] = f.x * s;
            x[2 * i + 1] = f.y * s;
        }
    } else {
        const __nv_bfloat162* p =
            reinterpret_cast<const __nv_bfloat162*>(static_cast<const __nv_bfloat16*>(pool) + row * D + col);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 f = __bfloat1622float2(p[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// One row by one warp, key by key, over tiles first..last-1: m (log2 units), l and D / 32 columns a lane.
template <int D, bool E4M3>
__device__ __noinline__ void attend_row(const AttendArgs& a, int b, int hk, const __nv_bfloat16* q, long p, Tiles tiles,
                                        int first, int last, float& m, float& l, float (&acc)[D / 32]) {
    constexpr int N = D / 32;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 31;
    const Seen s = seen_by(a, p);
    float qr[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        qr[i] = __bfloat162float(q[lane * N + i]) * (a.scale * 1.44269504f);
        acc[i] = 0.f;
    }
    m = -INFINITY, l = 0.f;
    for (int i = first; i < last; ++i) {
        const long j0 = (long)tiles[i] * kKeys;
        for (long j = j0; j < j0 + kKeys && j <= p; ++j) {
            if (j >= s.sink_end && j < s.begin) continue;
            const long at = cache_row(c, b, hk, j);
            if (at < 0) continue;
            float x[N], z = 0.f;
            load_row<N, E4M3>(c.pk, c.k_scale, at, lane * N, D, x);
#pragma unroll
            for (int i = 0; i < N; ++i) z = fmaf(qr[i], x[i], z);
#pragma unroll
            for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
            const float top = fmaxf(m, z);
            if (top == -INFINITY && z == z) continue;
            const float keep = m == top ? 1.f : exp2f(m - top), w = exp2f(z - top);
            m = top;
            l = l * keep + w;
            load_row<N, E4M3>(c.pv, c.v_scale, at, lane * N, D, x);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(w, x[i], acc[i] * keep);
        }
    }
}

template <int D, int NT, int STAGES>
struct Shared {
    __nv_bfloat16 q[NT][kRows * D];  // per tile D / 64 panels of 64 columns, 128-byte swizzle
    __nv_bfloat16 k[STAGES][kKeys * D], v[STAGES][kKeys * D];
    uint32_t valid[STAGES][4];  // keys of the stage that exist
    long at[2][kKeys];          // rows of the pool of the tile being fetched, in turn
    uint64_t q_full, full[STAGES], empty[STAGES], s_full[NT], p_full[NT], done;
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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Eight e4m3 values times their scale as bf16: both steps exact.
__device__ __forceinline__ uint4 to_bf16(uint32_t lo, uint32_t hi, float s) {
    const float2 a = e4m3x2_to_float2((uint16_t)lo), b = e4m3x2_to_float2((uint16_t)(lo >> 16));
    const float2 c = e4m3x2_to_float2((uint16_t)hi), d = e4m3x2_to_float2((uint16_t)(hi >> 16));
    return make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s), pack_bf16x2(c.x * s, c.y * s),
                      pack_bf16x2(d.x * s, d.y * s));
}

// Bits of the 32 keys from k0 on that lie in lo..hi.
__device__ __forceinline__ uint32_t range_mask(long k0, long lo, long hi) {
    const int a = (int)max(0L, min(32L, lo - k0)), e = (int)max(0L, min(32L, hi + 1 - k0));
    const uint32_t below_a = a == 32 ? 0xffffffffu : (1u << a) - 1, below_e = e == 32 ? 0xffffffffu : (1u << e) - 1;
    return below_e & ~below_a;
}

template <int D, bool E4M3, int NT, int STAGES>
__global__ void __launch_bounds__(NT * 128 + 160, 1) attend_kernel(AttendArgs a) {
    using S = Shared<D, NT, STAGES>;
    constexpr int kPanel = kKeys * 128;  // bytes of a panel of 64 columns
    constexpr uint32_t kColumns = NT == 1 ? 256 : 512;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    S& s = *reinterpret_cast<S*>(smem_raw);
    const CacheArgs& c = a.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = c.H / c.Hkv;
    const long rows = c.T * G;  // of one key/value head
    const int units = c.B * c.Hkv, unit = blockIdx.x % units, b = unit / c.Hkv, hk = unit % c.Hkv;
    // the last rows see the most keys and start first
    const long row0 = (long)(gridDim.x / units - 1 - blockIdx.x / units) * (NT * kRows);
    const int count = cache_count(c, b);
    const long start = c.starts[b];
    const long t_lo = row0 / G, t_hi = min(min(row0 + NT * kRows, rows) - 1, (long)count * G - 1) / G;
    Tiles tiles{0, 0, 0};
    if (row0 < (long)count * G) tiles = tiles_of(a, start + t_lo, start + t_hi);
    const int first = (int)((long)tiles.count * blockIdx.z / gridDim.z);
    const int last = (int)((long)tiles.count * (blockIdx.z + 1) / gridDim.z), n = last - first;

    if (warp == NT * 4 + 4) {
        tmem_alloc(&s.tmem, kColumns);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(&s.q_full, NT * 128);
        for (int i = 0; i < STAGES; ++i) mbar_init(&s.full[i], 128), mbar_init(&s.empty[i], 1);
        for (int i = 0; i < NT; ++i) mbar_init(&s.s_full[i], 1), mbar_init(&s.p_full[i], 128);
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

    if (warp < NT * 4) {  // -------------------------------------------------- softmax: one thread a row
        const int tile = warp >> 2;
        const long row = row0 + tid;
        const int t = (int)(row / G), h = hk * G + (int)(row % G);
        const bool live = row < rows && t < count;
        const bool any = __any_sync(0xffffffffu, live);
        const long p = start + t, out = (((long)b * c.H + h) * c.T + t) * D;
        const float sign = a.scale < 0.f ? -1.f : a.scale == 0.f ? 0.f : 1.f;
        const float scale = (a.scale == 0.f ? 1.f : fabsf(a.scale)) * 1.44269504f;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + out;
        if (n > 0) {
            // the row of Q; a scale that is not positive goes into its sign, so that the largest score is the largest weight's
            const uint32_t base = smem_u32(s.q[tile]), r = tid & 127;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
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
        const uint32_t ts = tmem + lane_base + tile * 128, to = tmem + lane_base + NT * 128 + tile * D;
        const Seen seen = seen_by(a, p);
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int stage = j % STAGES;
            const long k0 = (long)tiles[first + j] * kKeys;
            if (!(ok = wait(&s.s_full[tile], j & 1))) break;
            tc_fence_after();
            if (any) {
                const bool whole = k0 >= seen.begin && k0 + kKeys - 1 <= p &&
                                   (s.valid[stage][0] & s.valid[stage][1] & s.valid[stage][2] & s.valid[stage][3]) == ~0u;
                const bool all_whole = __all_sync(0xffffffffu, whole || !live);
                float top = -INFINITY;
                uint32_t mask[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mask[i] = ~0u;
                    if (!all_whole) {
                        const long kc = k0 + 32 * i;
                        mask[i] = (range_mask(kc, seen.begin, p) | range_mask(kc, 0, seen.sink_end - 1)) & s.valid[stage][i];
                    }
                    uint32_t r[32];
                    tmem_ld32(ts + 32 * i, r);
                    tmem_wait_ld();
                    if (all_whole) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(r[e]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            top = fmaxf(top, mask[i] >> e & 1 ? __uint_as_float(r[e]) : -INFINITY);
                    }
                }
                const bool grown = j == 0 || (top - m) * scale > kLazy || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grown)) {
                    const float next = fmaxf(m, top);
                    const float keep = m == next ? 1.f : ex2((m - next) * scale);
                    m = next;
                    l *= keep;
                    if (j > 0) {
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            uint32_t r[32];
                            tmem_ld32(to + 32 * i, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * keep);
                            tmem_st32(to + 32 * i, r);
                        }
                    }
                }
                const float shift = m == -INFINITY ? 0.f : m * scale;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t r[32], w[16];
                    tmem_ld32(ts + 32 * i, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float x = ex2(fmaf(__uint_as_float(r[e]), scale, -shift));
                        float y = ex2(fmaf(__uint_as_float(r[e + 1]), scale, -shift));
                        if (!all_whole) {
                            x = mask[i] >> e & 1 ? x : 0.f;
                            y = mask[i] >> (e + 1) & 1 ? y : 0.f;
                        }
                        l += x + y;
                        w[e / 2] = pack_bf16x2(x, y);
                    }
                    tmem_st16(ts + 16 * i, w);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            arrive(&s.p_full[tile]);
        }
        if (n > 0 && ok) ok = wait(&s.done, 0);
        tc_fence_after();
        // The row's output, or its part of it
        const bool partial = gridDim.z > 1;
        const long prow = (((long)blockIdx.z * c.B + b) * c.H + h) * c.T + t;
        float m2 = m * scale;
        if (any && ok) {
            const float inv = partial || l == 0.f ? 1.f : 1.f / l;
            bool fine = l == l && l < INFINITY;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t r[32];
                if (n > 0) {
                    tmem_ld32(to + 32 * i, r);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float x = n > 0 ? __uint_as_float(r[e]) * inv : 0.f;
                    fine = fine && fabsf(x) < INFINITY;
                    r[e] = __float_as_uint(x);
                }
                if (!live) continue;
                if (partial) {
                    uint4* dst = reinterpret_cast<uint4*>(a.part + prow * D + 32 * i);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + out + 32 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            w[f] = pack_bf16x2(__uint_as_float(r[8 * e + 2 * f]), __uint_as_float(r[8 * e + 2 * f + 1]));
                        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            uint32_t again = __ballot_sync(0xffffffffu, live && n > 0 && !fine);
            __syncwarp();  // what a lane stored above comes before what the others store below
            while (again) {  // rows that infinities or NaN reached, maybe through keys that they do not see
                const int who = __ffs(again) - 1;
                again &= again - 1;
                const long wq = __shfl_sync(0xffffffffu, out, who), wp = __shfl_sync(0xffffffffu, p, who);
                const long wprow = __shfl_sync(0xffffffffu, prow, who);
                float rm, rl, acc[D / 32];
                attend_row<D, E4M3>(a, b, hk, static_cast<const __nv_bfloat16*>(a.q) + wq, wp, tiles, first, last, rm, rl, acc);
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
        if (partial) {
            if (row < rows) a.part_ml[prow] = live ? make_float2(m2, l) : make_float2(-INFINITY, 0.f);
        } else if (row < rows && !live) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + out);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
        }
    } else if (warp < NT * 4 + 4) {  // ----------------------------------------- producers
        const int i0 = tid - NT * 128;
        constexpr int LANES = E4M3 ? D / 16 : D / 8, PASSES = kKeys * LANES / 128;  // 16 bytes a lane
        const int sub = i0 % LANES, group = i0 / LANES;
        // keys that no row of the CTA sees are neither looked up nor read
        const long see_hi = start + t_hi;
        const Seen lo = seen_by(a, start + t_lo), hi = seen_by(a, see_hi);
        bool ok = true, pending = false;  // copies begun whose stage has not been announced
        int stage_of_last = 0;
        auto landed = [&] {  // the copies of the last stage that was begun
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            arrive(&s.full[stage_of_last]);
        };
        for (int j = 0; j < n; ++j) {  // to the end in any case: the barrier below takes all 128 threads
            const int stage = j % STAGES;
            const long key = (long)tiles[first + j] * kKeys + i0;
            long at = -1;
            if (key <= see_hi && (key >= lo.begin || key < hi.sink_end)) {
                at = cache_row(c, b, hk, key);
                if (at < 0) atomicOr(c.status, kStatusMissingPage);
            }
            long* rows_at = s.at[j & 1];
            rows_at[i0] = at;
            const uint32_t there = __ballot_sync(0xffffffffu, at >= 0);
            asm volatile("bar.sync 1, 128;" ::: "memory");
            uint4 kx[E4M3 ? PASSES : 1], vx[E4M3 ? PASSES : 1];
            float ks[E4M3 ? PASSES : 1], vs[E4M3 ? PASSES : 1];
            if constexpr (E4M3) {  // in flight while the stage is still read
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const long r = rows_at[i * (128 / LANES) + group];
                    kx[i] = vx[i] = make_uint4(0, 0, 0, 0), ks[i] = vs[i] = 0.f;
                    if (r >= 0) {
                        kx[i] = static_cast<const uint4*>(c.pk)[r * LANES + sub], ks[i] = c.k_scale[r];
                        vx[i] = static_cast<const uint4*>(c.pv)[r * LANES + sub], vs[i] = c.v_scale[r];
                    }
                }
            }
            if (j >= STAGES && ok) {
                // the last stage's copies are awaited first where the wait for a free stage may depend on them
                if (pending && !mbar_try_wait(&s.empty[stage], (j / STAGES - 1) & 1)) landed(), pending = false;
                ok = wait(&s.empty[stage], (j / STAGES - 1) & 1);
            }
            if (!ok) continue;
            if (lane == 0) s.valid[stage][i0 >> 5] = there;
            const uint32_t kb = smem_u32(s.k[stage]), vb = smem_u32(s.v[stage]);
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = i * (128 / LANES) + group;
                if constexpr (E4M3) {
                    const uint32_t off = (sub >> 2) * kPanel, col = (sub & 3) * 16;
                    uint4 w = to_bf16(kx[i].x, kx[i].y, ks[i]);
                    st_shared_v4(kb + off + sw128_off(r, col), w.x, w.y, w.z, w.w);
                    w = to_bf16(kx[i].z, kx[i].w, ks[i]);
                    st_shared_v4(kb + off + sw128_off(r, col + 8), w.x, w.y, w.z, w.w);
                    w = to_bf16(vx[i].x, vx[i].y, vs[i]);
                    st_shared_v4(vb + off + sw128_off(r, col), w.x, w.y, w.z, w.w);
                    w = to_bf16(vx[i].z, vx[i].w, vs[i]);
                    st_shared_v4(vb + off + sw128_off(r, col + 8), w.x, w.y, w.z, w.w);
                } else {
                    const long src = rows_at[r];
                    const uint32_t off = (sub >> 3) * kPanel + sw128_off(r, (sub & 7) * 8);
                    const long at = src < 0 ? 0 : src * LANES + sub;
                    cp_async16_zfill(kb + off, static_cast<const uint4*>(c.pk) + at, src >= 0);
                    cp_async16_zfill(vb + off, static_cast<const uint4*>(c.pv) + at, src >= 0);
                }
            }
            if constexpr (E4M3) {
                fence_proxy_async_smem();
                arrive(&s.full[stage]);
            } else {
                asm volatile("cp.async.commit_group;" ::: "memory");
                if (pending) {
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    fence_proxy_async_smem();
                    arrive(&s.full[stage_of_last]);
                }
                pending = true;
                stage_of_last = stage;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (pending) landed();
    } else if (lane == 0 && n > 0) {  // ---------------------------------------- the thread that issues the MMAs
        const uint32_t id_s = idesc_bf16_f32(128, kKeys, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
        auto scores = [&](int i, int stage) {
            const uint32_t q = smem_u32(s.q[i]), k = smem_u32(s.k[stage]);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks >> 2) * kPanel + (ks & 3) * 32;
                umma_bf16(tmem + i * 128, sdesc_sw128(q + off, 16, 1024), sdesc_sw128(k + off, 16, 1024), id_s, ks > 0);
            }
            umma_commit(&s.s_full[i]);
        };
        bool ok = wait(&s.q_full, 0) && wait(&s.full[0], 0);
        if (ok) {
            tc_fence_after();
            for (int i = 0; i < NT; ++i) scores(i, 0);
        }
        for (int j = 0; j < n && ok; ++j) {
            const int stage = j % STAGES;
            for (int i = 0; i < NT && ok; ++i) {
                if (!(ok = wait(&s.p_full[i], j & 1))) break;
                tc_fence_after();
                const uint32_t v = smem_u32(s.v[stage]);
#pragma unroll
                for (int ks = 0; ks < kKeys / 16; ++ks)
                    umma_bf16_ts(tmem + NT * 128 + i * D, tmem + i * 128 + ks * 8, sdesc_sw128(v + ks * 2048, kPanel, 1024),
                                 id_o, j > 0 || ks > 0);
                if (i == NT - 1) umma_commit(j + 1 < n ? &s.empty[stage] : &s.done);
                if (j + 1 < n) {
                    if (i == 0) {
                        if (!(ok = wait(&s.full[(j + 1) % STAGES], ((j + 1) / STAGES) & 1))) break;
                        tc_fence_after();
                    }
                    scores(i, (j + 1) % STAGES);
                }
            }
        }
        // Nothing of this CTA may still be at work when its TMEM is freed, an aborted pass's MMAs neither.
        if (!ok) {
            umma_commit(&s.done);
            mbar_wait(&s.done, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == NT * 4 + 4) {
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
    kernel<<<grid, NT * 128 + 160, sizeof(S), st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || splits == 1) return e;
    combine_kernel<D><<<(unsigned)(((long)a.c.B * a.c.H * a.c.T + 3) / 4), 128, 0, st>>>(a, splits);
    return cudaGetLastError();
}

}  // namespace

// Splits of the keys: enough CTAs for two rounds over the SMs, and no less than four tiles of the longest
// possible sequence each. The lengths themselves are on the device.
int attend_splits(int B, int H, int Hkv, long T, long longest) {
    const long rows = T * (H / Hkv), base = ((rows + kRows - 1) / kRows) * B * Hkv;
    const long most = std::max(1L, longest / kKeys / 4);
    return (int)std::max(1L, std::min({most, 2 * 148L / base, 64L}));
}

size_t attend_workspace_bytes(int B, int H, long T, int d, int splits) {
    return splits == 1 ? 0 : (size_t)splits * B * H * T * (d * sizeof(float) + sizeof(float2));
}

cudaError_t launch_cache_attend(const AttendArgs& args, bool e4m3, int splits, void* workspace, cudaStream_t st) {
    AttendArgs a = args;
    const size_t n = (size_t)splits * a.c.B * a.c.H * a.c.T;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + (splits > 1 ? n * a.c.d : 0));
    // Two tiles of rows a CTA where that still leaves a CTA for most SMs
    const long rows = a.c.T * (a.c.H / a.c.Hkv);
    const bool two = rows > kRows && (rows + 2 * kRows - 1) / (2 * kRows) * a.c.B * a.c.Hkv * splits >= 100;
    if (a.c.d == 64) {
        if (e4m3) return two ? launch<64, true, 2>(a, splits, st) : launch<64, true, 1>(a, splits, st);
        return two ? launch<64, false, 2>(a, splits, st) : launch<64, false, 1>(a, splits, st);
    }
    if (e4m3) return two ? launch<128, true, 2>(a, splits, st) : launch<128, true, 1>(a, splits, st);
    return two ? launch<128, false, 2>(a, splits, st) : launch<128, false, 1>(a, splits, st);
}

}  // namespace titans
