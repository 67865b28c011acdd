// Host-side launch interface of the gated delta rule's kernels (not part of the C ABI).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

namespace titans {

struct DeltaArgs {
    int d, B, H, Hk;
    bool bf16;  // dtype of k, q, v, attn, y
    long T;
    const void *k, *q, *v, *attn;  // attn: NULL for y = W q
    const float *g, *beta;
    const int* lengths;  // NULL: all T
    float* W;
    void* y;
};

// Pieces of the state, the writes and P that y is taken from (delta_chunks.cu).
inline int delta_y_pieces(const DeltaArgs& a) { return a.bf16 && !a.attn ? 1 : 2; }

// Token by token, one warp for eight rows of a unit's state (delta_step.cu): any T >= 1.
cudaError_t launch_delta_tokens(const DeltaArgs& a, cudaStream_t st);

// The chunked path. Per (unit, chunk) record of delta_chunk_bytes(), written by the first kernel and read by the
// others (delta_prepare.cu); units * ceil(T / 64) records.
size_t delta_chunk_bytes();
cudaError_t launch_delta_prepare(const DeltaArgs& a, void* chunks, bool backward, cudaStream_t st);
// The state's way through the chunks, and y (delta_chunks.cu). With `states` it writes, in place of y and
// the final state, every chunk's start state [units][chunks][d][d] and residuals eps [units][chunks][64][d], fp32.
struct DeltaStates {
    float *states, *eps;
};
cudaError_t launch_delta_chunks(const DeltaArgs& a, const void* chunks, const DeltaStates* states, cudaStream_t st);

struct DeltaGrads {
    const void* dy;
    const float* dW;  // adjoint of the final state, NULL: zero
    void *dk, *dq, *dv;
    float *dg, *dbeta, *dW0;
    DeltaStates fwd;    // what launch_delta_chunks left
    float *adj, *dr;    // every chunk's adjoint of its final state [units][chunks][d][d], and dR [units][chunks][64][d]
};
// The adjoint's way back through the chunks: adj, dr, dW0 (delta_adjoint.cu).
cudaError_t launch_delta_adjoint(const DeltaArgs& a, const void* chunks, const DeltaGrads& g, cudaStream_t st);
// The tokens' gradients, from the states and adjoints of their chunk (delta_grads.cu).
cudaError_t launch_delta_grads(const DeltaArgs& a, const void* chunks, const DeltaGrads& g, cudaStream_t st);

}  // namespace titans
