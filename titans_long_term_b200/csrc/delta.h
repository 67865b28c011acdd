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

// Token by token, one warp for eight rows of a unit's state (delta_step.cu): any T >= 1.
cudaError_t launch_delta_tokens(const DeltaArgs& a, cudaStream_t st);

}  // namespace titans
