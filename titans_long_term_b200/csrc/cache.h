// Host-side launch interface of the paged cache's kernels (not part of the C ABI).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>

#include "cache.cuh"

namespace titans {

constexpr long kSms = 148;  // of a B200

cudaError_t launch_cache_append(const CacheArgs& a, bool e4m3, const void* k, const void* v, cudaStream_t st);
cudaError_t launch_cache_read(const CacheArgs& a, bool e4m3, void* k, void* v, cudaStream_t st);

struct AttendArgs {
    CacheArgs c;
    const void* q;  // [B, H, T, d] bf16
    void* o;
    int window, sinks;
    float scale;
    float* part;      // workspace: unnormalised outputs of parts of the keys, d each,
    float2* part_ml;  // their maxima (log2) and sums,
    long* begins;     // and, for few rows, the first block of each sequence, then the number of blocks
};
// Few rows a key/value head (one token of a decode step, say): cache_attend_few.cu.
bool attend_few_rows(int H, int Hkv, long T);
size_t attend_few_bytes(int B, int Hkv, int d, long longest);
cudaError_t launch_attend_few(const AttendArgs& a, bool e4m3, void* workspace, long longest, cudaStream_t st);
// longest: tokens that a sequence's row of the page table has room for.
size_t attend_workspace_bytes(int B, int H, int Hkv, long T, int d, long longest);
cudaError_t launch_cache_attend(const AttendArgs& a, bool e4m3, void* workspace, long longest, cudaStream_t st);

}  // namespace titans
