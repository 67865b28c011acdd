// Host-side launch interface of the paged cache's kernels (not part of the C ABI).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

#include "cache.cuh"

namespace titans {

cudaError_t launch_cache_append(const CacheArgs& a, bool e4m3, const void* k, const void* v, cudaStream_t st);
cudaError_t launch_cache_read(const CacheArgs& a, bool e4m3, void* k, void* v, cudaStream_t st);

struct AttendArgs {
    CacheArgs c;
    const void* q;  // [B, H, T, d] bf16
    void* o;
    int window, sinks;
    float scale;
    float* part;      // unnormalised outputs of the splits [splits][B, H, T][d]
    float2* part_ml;  // their maxima (log2) and sums [splits][B, H, T]
};
// Few rows a key/value head (one token of a decode step, say): cache_attend_few.cu.
bool attend_few_rows(int H, int Hkv, long T);
int attend_few_splits(int B, int Hkv, long longest);
cudaError_t launch_attend_few(const AttendArgs& a, bool e4m3, int splits, cudaStream_t st);
int attend_splits(int B, int H, int Hkv, long T, long longest);
size_t attend_workspace_bytes(int B, int H, long T, int d, int splits);
cudaError_t launch_cache_attend(const AttendArgs& a, bool e4m3, int splits, void* workspace, cudaStream_t st);

}  // namespace titans
