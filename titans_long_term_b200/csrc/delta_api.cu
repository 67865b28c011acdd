// C ABI of the gated delta rule: argument checks and dispatch.
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "../../include/titans_mem.h"
#include "delta.h"

namespace titans {
void set_last_error(const std::string& msg);
}

namespace {

titans_status_t fail(titans_status_t s, const std::string& msg) {
    titans::set_last_error(msg);
    return s;
}

titans_status_t check_cfg(const titans_delta_config* c) {
    if (!c) return fail(TITANS_EINVAL, "config is NULL");
    if (c->B <= 0 || c->H <= 0 || c->Hk <= 0) return fail(TITANS_EINVAL, "B, H and Hk must be positive");
    if (c->H % c->Hk) return fail(TITANS_EINVAL, "Hk must divide H");
    if ((long)c->B * c->H > (1L << 24)) return fail(TITANS_EINVAL, "too many units (at most 2^24)");
    if (c->mode != TITANS_BF16 && c->mode != TITANS_FP32) return fail(TITANS_EINVAL, "unknown mode");
    if (c->d != 64 && c->d != 128) return fail(TITANS_EUNSUPPORTED, "d must be 64 or 128");
    return TITANS_OK;
}

titans_status_t check_tokens(const titans_delta_config* c, long T) {
    if (T < 1) return fail(TITANS_EINVAL, "T must be >= 1");
    if (T >= (1L << 31) / c->d) return fail(TITANS_EUNSUPPORTED, "T * d must be below 2^31");
    if ((long)c->B * c->H * ((T + 63) / 64) >= (1L << 31) / 2)
        return fail(TITANS_EUNSUPPORTED, "B * H * ceil(T / 64) must be below 2^30");
    return TITANS_OK;
}

struct Arg {
    const char* name;
    const void* p;
    unsigned align;
    bool optional;
};

template <int N>
titans_status_t check_ptrs(const Arg (&args)[N]) {
    for (const Arg& a : args) {
        if (!a.p && !a.optional) return fail(TITANS_EINVAL, std::string(a.name) + " is NULL");
        if (reinterpret_cast<uintptr_t>(a.p) & (a.align - 1))
            return fail(TITANS_EINVAL, std::string(a.name) + " is not " + std::to_string(a.align) + "-byte aligned");
    }
    return TITANS_OK;
}

titans_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return TITANS_OK;
    return fail(TITANS_ECUDA, std::string("kernel launch: ") + cudaGetErrorString(e));
}

titans::DeltaArgs make_args(const titans_delta_config* c, const void* k, const void* q, const void* v, const float* g,
                            const float* beta, const int* lengths, long T, float* W, const void* attn, void* y) {
    titans::DeltaArgs a{};
    a.d = c->d;
    a.B = c->B;
    a.H = c->H;
    a.Hk = c->Hk;
    a.bf16 = c->mode == TITANS_BF16;
    a.T = T;
    a.k = k;
    a.q = q;
    a.v = v;
    a.attn = attn;
    a.g = g;
    a.beta = beta;
    a.lengths = lengths;
    a.W = W;
    a.y = y;
    return a;
}

// Up to this many tokens go one by one, with the state in registers: 0.5 us a token, against 16.5 us for the chunked path's two
// launches and its work on 64 tokens (16 to 128 units, d = 64 and 128: 10.3 us for 16 tokens, 12.4 to 14.5 for 24, 16.5 to
// 18.5 for 32).
constexpr long kTokens = 24;

long records(const titans_delta_config* c, long T) { return (long)c->B * c->H * ((T + 63) / 64); }
struct Backward {  // offsets in the workspace of the backward pass, 1 KiB aligned
    size_t states, eps, adj, dr, bytes;
};
Backward backward_layout(const titans_delta_config* c, long T) {
    const size_t n = (size_t)records(c, T), matrix = n * c->d * c->d * sizeof(float), tokens = n * 64 * c->d * sizeof(float);
    Backward b;
    b.states = n * titans::delta_chunk_bytes();
    b.eps = b.states + matrix;
    b.adj = b.eps + tokens;
    b.dr = b.adj + matrix;
    b.bytes = b.dr + tokens;
    return b;
}
size_t forward_bytes(const titans_delta_config* c, long T) {
    return T <= kTokens ? 0 : (size_t)records(c, T) * titans::delta_chunk_bytes();
}

}  // namespace

extern "C" {

size_t titans_delta_workspace_bytes(const titans_delta_config* cfg, long T, int call) {
    if (check_cfg(cfg) != TITANS_OK || check_tokens(cfg, T) != TITANS_OK) return (size_t)-1;
    if (call != 0 && call != 1) {
        fail(TITANS_EINVAL, "call must be 0 (forward) or 1 (backward)");
        return (size_t)-1;
    }
    return call ? backward_layout(cfg, T).bytes : forward_bytes(cfg, T);
}

titans_status_t titans_delta_forward(const titans_delta_config* cfg, const void* k, const void* q, const void* v,
                                     const float* g, const float* beta, const int* lengths, long T, float* W,
                                     const void* attn, void* y, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    titans_status_t s = check_cfg(cfg);
    if (s == TITANS_OK) s = check_tokens(cfg, T);
    if (s != TITANS_OK) return s;
    const size_t need = titans_delta_workspace_bytes(cfg, T, 0);
    const Arg args[] = {{"k", k, 16, false},       {"q", q, 16, false},           {"v", v, 16, false},
                        {"g", g, 4, false},        {"beta", beta, 4, false},      {"lengths", lengths, 4, true},
                        {"W", W, 16, false},       {"attn", attn, 16, true},      {"y", y, 16, false},
                        {"workspace", workspace, 16, need == 0}};
    if ((s = check_ptrs(args)) != TITANS_OK) return s;
    if (workspace_bytes < need) return fail(TITANS_EINVAL, "workspace is too small");
    const titans::DeltaArgs a = make_args(cfg, k, q, v, g, beta, lengths, T, W, attn, y);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T <= kTokens) return launched(titans::launch_delta_tokens(a, st));
    const cudaError_t e = titans::launch_delta_prepare(a, workspace, false, st);
    return launched(e != cudaSuccess ? e : titans::launch_delta_chunks(a, workspace, nullptr, st));
}

titans_status_t titans_delta_step(const titans_delta_config* cfg, const void* k, const void* q, const void* v,
                                  const float* g, const float* beta, float* W, const void* attn, void* y,
                                  void* stream) {
    titans_status_t s = check_cfg(cfg);
    if (s != TITANS_OK) return s;
    const Arg args[] = {{"k", k, 16, false},      {"q", q, 16, false}, {"v", v, 16, false},     {"g", g, 4, false},
                        {"beta", beta, 4, false}, {"W", W, 16, false}, {"attn", attn, 16, true}, {"y", y, 16, false}};
    if ((s = check_ptrs(args)) != TITANS_OK) return s;
    return launched(titans::launch_delta_tokens(make_args(cfg, k, q, v, g, beta, nullptr, 1, W, attn, y),
                                                static_cast<cudaStream_t>(stream)));
}

titans_status_t titans_delta_backward(const titans_delta_config* cfg, const void* k, const void* q, const void* v,
                                      const float* g, const float* beta, const int* lengths, long T, const float* W,
                                      const void* dy, const float* dW, void* dk, void* dq, void* dv, float* dg,
                                      float* dbeta, float* dW0, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    titans_status_t s = check_cfg(cfg);
    if (s == TITANS_OK) s = check_tokens(cfg, T);
    if (s != TITANS_OK) return s;
    const Arg args[] = {{"k", k, 16, false},   {"q", q, 16, false},     {"v", v, 16, false},
                        {"g", g, 4, false},    {"beta", beta, 4, false}, {"lengths", lengths, 4, true},
                        {"W", W, 16, false},   {"dy", dy, 16, false},   {"dW", dW, 16, true},
                        {"dk", dk, 16, false}, {"dq", dq, 16, false},   {"dv", dv, 16, false},
                        {"dg", dg, 4, false},  {"dbeta", dbeta, 4, false}, {"dW0", dW0, 16, false},
                        {"workspace", workspace, 16, false}};
    if ((s = check_ptrs(args)) != TITANS_OK) return s;
    const Backward at = backward_layout(cfg, T);
    if (workspace_bytes < at.bytes) return fail(TITANS_EINVAL, "workspace is too small");
    char* ws = static_cast<char*>(workspace);
    const titans::DeltaArgs a =
        make_args(cfg, k, q, v, g, beta, lengths, T, const_cast<float*>(W), nullptr, nullptr);  // W is only read
    titans::DeltaGrads o{};
    o.dy = dy;
    o.dW = dW;
    o.dk = dk;
    o.dq = dq;
    o.dv = dv;
    o.dg = dg;
    o.dbeta = dbeta;
    o.dW0 = dW0;
    o.fwd = {reinterpret_cast<float*>(ws + at.states), reinterpret_cast<float*>(ws + at.eps)};
    o.adj = reinterpret_cast<float*>(ws + at.adj);
    o.dr = reinterpret_cast<float*>(ws + at.dr);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = titans::launch_delta_prepare(a, ws, true, st);
    if (e == cudaSuccess) e = titans::launch_delta_chunks(a, ws, &o.fwd, st);
    if (e == cudaSuccess) e = titans::launch_delta_adjoint(a, ws, o, st);
    if (e == cudaSuccess) e = titans::launch_delta_grads(a, ws, o, st);
    return launched(e);
}

}  // extern "C"
