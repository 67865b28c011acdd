// Paged key/value cache: writing new tokens (as bf16, or as 8-bit floats with a scale of their own) and
// reading them back, and the C ABI.
//
// An e4m3 token keeps one scale per head, the smallest power of two with max |x| <= 448 * scale. A power of
// two makes the division and the multiplication exact: the one rounding of the round trip is the
// conversion to 4 significant bits, and what read returns is exact in bf16.
//
// Both kernels move bytes: d/8 lanes hold one row, 16 bytes of bf16 each, k and v of the same token together, so that the
// table is looked up once and two loads are in flight. Writing 25,600 rows of keys and of values (d = 128) to e4m3 and reading them back takes
// 14.7 us for 40 MB (2.7 TB/s: each call is a launch and three dependent loads long), one token of 32 sequences 6.4 us.
#include <cmath>
#include <new>
#include <string>

#include "../../include/titans_mem.h"
#include "cache.h"

namespace titans {
namespace {

constexpr int kThreads = 256;

// 8 bf16 of a lane <-> 8 e4m3; scale is the row's power of two, found over the row's `LANES` lanes.
template <int LANES>
__device__ __forceinline__ uint2 quantise(uint4 u, float& scale) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float x[8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[i]);
        top = m < INFINITY ? fmaxf(top, m) : top;  // NaN and infinities have no say in the scale
    }
#pragma unroll
    for (int s = LANES / 2; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    // top = 1.f * 2^x and 448 = 1.75 * 2^8: 2^(x-8) is enough up to 1.75, 2^(x-7) above
    const int bits = __float_as_int(top);
    int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
    e = top == 0.f ? 0 : max(e, -117);  // -117: the smallest value, 2^-9 of the scale, is a normal bf16 still
    scale = __int_as_float((e + 127) << 23);
    const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    if (e == 120) {  // 256 * 2^120 would be read back as an infinity; NaN stays NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fabsf(x[i]) > 240.f ? copysignf(240.f, x[i]) : x[i];
    }
    uint2 r;
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    r.x = h[0] | (uint32_t)h[1] << 16;
    r.y = h[2] | (uint32_t)h[3] << 16;
    return r;
}

__device__ __forceinline__ uint32_t bf16x2_scaled(float2 f, float scale) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 dequantise(uint2 u, float scale) {
    return make_uint4(bf16x2_scaled(e4m3_to_float2<false>(u.x), scale), bf16x2_scaled(e4m3_to_float2<true>(u.x), scale),
                      bf16x2_scaled(e4m3_to_float2<false>(u.y), scale), bf16x2_scaled(e4m3_to_float2<true>(u.y), scale));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) append_kernel(CacheArgs a, const uint4* k, const uint4* v) {
    constexpr int LANES = D / 8;
    const long rows = (long)a.B * a.Hkv * a.T;
    const long row = ((long)blockIdx.x * kThreads + threadIdx.x) / LANES;
    const int lane = threadIdx.x % LANES;
    const bool in = row < rows;
    const long unit = in ? row / a.T : 0;
    const int t = in ? (int)(row - unit * a.T) : 0, b = (int)(unit / a.Hkv), h = (int)(unit % a.Hkv);
    long at = -1;
    if (in && t < cache_count(a, b)) {
        at = cache_row(a, b, h, (long)a.starts[b] + t);
        if (at < 0 && lane == 0) atomicOr(a.status, kStatusMissingPage);
    }
    uint4 x = make_uint4(0, 0, 0, 0), z = x;
    if (at >= 0) {
        x = k[row * LANES + lane];
        z = v[row * LANES + lane];
    }
    if constexpr (E4M3) {  // every lane takes part in the shuffles
        float ks, vs;
        const uint2 kq = quantise<LANES>(x, ks), vq = quantise<LANES>(z, vs);
        if (at >= 0) {
            static_cast<uint2*>(a.pk)[at * LANES + lane] = kq;
            static_cast<uint2*>(a.pv)[at * LANES + lane] = vq;
            if (lane == 0) a.k_scale[at] = ks, a.v_scale[at] = vs;
        }
    } else if (at >= 0) {
        static_cast<uint4*>(a.pk)[at * LANES + lane] = x;
        static_cast<uint4*>(a.pv)[at * LANES + lane] = z;
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) read_kernel(CacheArgs a, uint4* k, uint4* v) {
    constexpr int LANES = D / 8;
    const long row = ((long)blockIdx.x * kThreads + threadIdx.x) / LANES;
    const int lane = threadIdx.x % LANES;
    if (row >= (long)a.B * a.Hkv * a.T) return;
    const long unit = row / a.T;
    const int t = (int)(row - unit * a.T), b = (int)(unit / a.Hkv), h = (int)(unit % a.Hkv);
    uint4 x = make_uint4(0, 0, 0, 0), z = x;
    if (t < cache_count(a, b)) {
        const long at = cache_row(a, b, h, (long)a.starts[b] + t);
        if (at < 0) {
            if (lane == 0) atomicOr(a.status, kStatusMissingPage);
        } else if constexpr (E4M3) {
            x = dequantise(static_cast<const uint2*>(a.pk)[at * LANES + lane], a.k_scale[at]);
            z = dequantise(static_cast<const uint2*>(a.pv)[at * LANES + lane], a.v_scale[at]);
        } else {
            x = static_cast<const uint4*>(a.pk)[at * LANES + lane];
            z = static_cast<const uint4*>(a.pv)[at * LANES + lane];
        }
    }
    k[row * LANES + lane] = x;
    v[row * LANES + lane] = z;
}

__global__ void clear_status_kernel(unsigned* status, unsigned bits) { atomicAnd(status, ~bits); }

unsigned blocks(const CacheArgs& a) {
    const long per = kThreads / (a.d / 8);
    return (unsigned)(((long)a.B * a.Hkv * a.T + per - 1) / per);
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& a, bool e4m3, const void* k, const void* v, cudaStream_t st) {
    auto* kernel = a.d == 64 ? (e4m3 ? append_kernel<64, true> : append_kernel<64, false>)
                             : (e4m3 ? append_kernel<128, true> : append_kernel<128, false>);
    kernel<<<blocks(a), kThreads, 0, st>>>(a, static_cast<const uint4*>(k), static_cast<const uint4*>(v));
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheArgs& a, bool e4m3, void* k, void* v, cudaStream_t st) {
    auto* kernel = a.d == 64 ? (e4m3 ? read_kernel<64, true> : read_kernel<64, false>)
                             : (e4m3 ? read_kernel<128, true> : read_kernel<128, false>);
    kernel<<<blocks(a), kThreads, 0, st>>>(a, static_cast<uint4*>(k), static_cast<uint4*>(v));
    return cudaGetLastError();
}

// Takes `bits` out of the status word, in the stream's order; bits that another stream sets meanwhile stay.
cudaError_t launch_clear_status(unsigned* status, unsigned bits, cudaStream_t st) {
    clear_status_kernel<<<1, 1, 0, st>>>(status, bits);
    return cudaGetLastError();
}

void set_last_error(const std::string& msg);

}  // namespace titans

struct titans_cache {
    titans_cache_config cfg;
    int device;
    unsigned* status;
};

namespace {

titans_status_t fail(titans_status_t s, const std::string& msg) {
    titans::set_last_error(msg);
    return s;
}
titans_status_t cuda_fail(cudaError_t e, const char* what) {
    return fail(TITANS_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

titans_status_t check_cfg(const titans_cache_config* c) {
    if (!c) return fail(TITANS_EINVAL, "config is NULL");
    if (c->B <= 0 || c->H <= 0 || c->Hkv <= 0 || c->num_pages <= 0 || c->max_pages <= 0)
        return fail(TITANS_EINVAL, "B, H, Hkv, num_pages and max_pages must be positive");
    if (c->H % c->Hkv) return fail(TITANS_EINVAL, "Hkv must divide H");
    if ((long)c->B * c->H > (1L << 24)) return fail(TITANS_EINVAL, "B * H must be at most 2^24");
    if (c->type != TITANS_CACHE_BF16 && c->type != TITANS_CACHE_E4M3) return fail(TITANS_EINVAL, "unknown type");
    if (c->d != 64 && c->d != 128) return fail(TITANS_EUNSUPPORTED, "d must be 64 or 128");
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return fail(TITANS_EUNSUPPORTED, "page must be 16, 32, 64 or 128");
    if ((long)c->max_pages * c->page > (1L << 31) - 1024)  // positions, rounded up to a tile or two, are 32-bit
        return fail(TITANS_EUNSUPPORTED, "max_pages * page must be at most 2^31 - 1024");
    if ((long)c->num_pages * c->Hkv * c->page >= (1L << 31))
        return fail(TITANS_EUNSUPPORTED, "num_pages * Hkv * page must be below 2^31");
    return TITANS_OK;
}

titans_status_t check_ptr(const void* p, const char* name, unsigned align, bool optional = false) {
    if (!p && !optional) return fail(TITANS_EINVAL, std::string(name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) & (align - 1))
        return fail(TITANS_EINVAL, std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
    return TITANS_OK;
}

// What every call checks; fills `a`.
titans_status_t make_args(titans_cache* c, long T, const titans_cache_pages* pages, const int* table, const int* starts,
                          const int* counts, titans::CacheArgs* a) {
    if (!c) return fail(TITANS_EINVAL, "handle is NULL");
    if (!pages) return fail(TITANS_EINVAL, "pages is NULL");
    if (T < 1) return fail(TITANS_EINVAL, "T must be >= 1");
    if (T >= (1L << 31) / c->cfg.d || (long)c->cfg.B * c->cfg.H * T >= (1L << 31))
        return fail(TITANS_EUNSUPPORTED, "T * d and B * H * T must be below 2^31");
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != c->device) return fail(TITANS_EINVAL, "the handle belongs to another device than the current one");
    const bool scaled = c->cfg.type == TITANS_CACHE_E4M3;
    titans_status_t s = check_ptr(pages->k, "pages k", 16);
    if (s == TITANS_OK) s = check_ptr(pages->v, "pages v", 16);
    if (s == TITANS_OK && scaled) s = check_ptr(pages->k_scale, "pages k_scale", 4);
    if (s == TITANS_OK && scaled) s = check_ptr(pages->v_scale, "pages v_scale", 4);
    if (s == TITANS_OK) s = check_ptr(table, "table", 4);
    if (s == TITANS_OK) s = check_ptr(starts, "starts", 4);
    if (s == TITANS_OK) s = check_ptr(counts, "counts", 4, true);
    if (s != TITANS_OK) return s;
    a->d = c->cfg.d;
    a->B = c->cfg.B;
    a->H = c->cfg.H;
    a->Hkv = c->cfg.Hkv;
    a->page_shift = c->cfg.page == 16 ? 4 : c->cfg.page == 32 ? 5 : c->cfg.page == 64 ? 6 : 7;
    a->num_pages = c->cfg.num_pages;
    a->max_pages = c->cfg.max_pages;
    a->T = T;
    a->pk = pages->k;
    a->pv = pages->v;
    a->k_scale = pages->k_scale;
    a->v_scale = pages->v_scale;
    a->table = table;
    a->starts = starts;
    a->counts = counts;
    a->status = c->status;
    return TITANS_OK;
}

titans_status_t launched(cudaError_t e) { return e == cudaSuccess ? TITANS_OK : cuda_fail(e, "kernel launch"); }

}  // namespace

extern "C" {

titans_status_t titans_cache_init(const titans_cache_config* cfg, titans_cache_t* out) {
    if (!out) return fail(TITANS_EINVAL, "out is NULL");
    *out = nullptr;
    const titans_status_t s = check_cfg(cfg);
    if (s != TITANS_OK) return s;
    titans_cache* c = new (std::nothrow) titans_cache();
    if (!c) return fail(TITANS_EINVAL, "out of host memory");
    c->cfg = *cfg;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaMalloc(&c->status, sizeof(unsigned));
    if (e == cudaSuccess) {
        e = cudaMemset(c->status, 0, sizeof(unsigned));
        // a first call may come on a stream that does not wait for the default one
        if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
        if (e != cudaSuccess) cudaFree(c->status);
    }
    if (e != cudaSuccess) {
        delete c;
        return cuda_fail(e, "allocating the status word");
    }
    *out = c;
    return TITANS_OK;
}

titans_status_t titans_cache_destroy(titans_cache_t c) {
    if (!c) return fail(TITANS_EINVAL, "handle is NULL");
    // A binding may let go of a handle at any time, also while this thread captures a graph, which a plain cudaFree
    // would end.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    const bool swapped = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
    cudaFree(c->status);
    if (swapped) cudaThreadExchangeStreamCaptureMode(&mode);
    delete c;
    return TITANS_OK;
}

titans_status_t titans_cache_sync_status(titans_cache_t c, void* stream) {
    if (!c) return fail(TITANS_EINVAL, "handle is NULL");
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev != c->device) e = cudaSetDevice(c->device);
    if (e != cudaSuccess) return cuda_fail(e, "choosing the handle's device");
    // All in the caller's stream: the default stream's order would not hold for calls on other streams.
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned h = 0;
    e = cudaMemcpyAsync(&h, c->status, sizeof(unsigned), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && h) e = titans::launch_clear_status(c->status, h, st);
    if (e == cudaSuccess && h) e = cudaStreamSynchronize(st);
    if (dev != c->device) cudaSetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e, "reading the status word");
    if (h) return fail(TITANS_EDEVICE, "device status " + std::to_string(h) +
                                           " (2: a wait timed out, 16: a token's page is missing)");
    return TITANS_OK;
}

titans_status_t titans_cache_append(titans_cache_t c, const void* k, const void* v, long T,
                                    const titans_cache_pages* pages, const int* table, const int* starts,
                                    const int* counts, void* stream) {
    titans::CacheArgs a{};
    titans_status_t s = make_args(c, T, pages, table, starts, counts, &a);
    if (s == TITANS_OK) s = check_ptr(k, "k", 16);
    if (s == TITANS_OK) s = check_ptr(v, "v", 16);
    if (s != TITANS_OK) return s;
    return launched(titans::launch_cache_append(a, c->cfg.type == TITANS_CACHE_E4M3, k, v,
                                                static_cast<cudaStream_t>(stream)));
}

titans_status_t titans_cache_read(titans_cache_t c, const titans_cache_pages* pages, const int* table,
                                  const int* starts, const int* counts, long T, void* k, void* v, void* stream) {
    titans::CacheArgs a{};
    titans_status_t s = make_args(c, T, pages, table, starts, counts, &a);
    if (s == TITANS_OK) s = check_ptr(k, "k", 16);
    if (s == TITANS_OK) s = check_ptr(v, "v", 16);
    if (s != TITANS_OK) return s;
    return launched(titans::launch_cache_read(a, c->cfg.type == TITANS_CACHE_E4M3, k, v,
                                              static_cast<cudaStream_t>(stream)));
}

size_t titans_cache_attend_workspace_bytes(titans_cache_t c, long T) {
    if (!c || T < 1 || T >= (1L << 31) / c->cfg.d) return 0;  // refused by the call itself
    return titans::attend_workspace_bytes(c->cfg.B, c->cfg.H, c->cfg.Hkv, T, c->cfg.d,
                                           (long)c->cfg.max_pages * c->cfg.page);
}

titans_status_t titans_cache_attend(titans_cache_t c, const void* q, long T, const titans_cache_pages* pages,
                                    const int* table, const int* starts, const int* counts, int window, int sinks,
                                    float scale, void* o, void* workspace, size_t workspace_bytes, void* stream) {
    titans::AttendArgs a{};
    titans_status_t s = make_args(c, T, pages, table, starts, counts, &a.c);
    if (s == TITANS_OK) s = check_ptr(q, "q", 16);
    if (s == TITANS_OK) s = check_ptr(o, "o", 16);
    if (s != TITANS_OK) return s;
    if (window < 0 || sinks < 0) return fail(TITANS_EINVAL, "window and sinks must be >= 0");
    if (!(std::fabs(scale) <= 0x1p100f)) return fail(TITANS_EINVAL, "|scale| must be at most 2^100");
    const size_t need = titans_cache_attend_workspace_bytes(c, T);
    if ((s = check_ptr(workspace, "workspace", 16, need == 0)) != TITANS_OK) return s;
    if (workspace_bytes < need) return fail(TITANS_EINVAL, "workspace is too small");
    a.q = q;
    a.o = o;
    a.window = window;
    a.sinks = sinks;
    a.scale = scale;
    return launched(titans::launch_cache_attend(a, c->cfg.type == TITANS_CACHE_E4M3, workspace,
                                                (long)c->cfg.max_pages * c->cfg.page, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
