// attn.cuh -- what the two attention kernels over the 4-bit cache share
// (cache.cu: up to 16 queries a head of the cache; attn_wide.cu: more).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace ufp4 {

struct AttnArgs {
    const void *q;
    int64_t q_token, q_head;
    int32_t q_fp32, planes, two_p;
    CacheHalf k, v;
    const int32_t *table;
    int64_t ld_table;
    int32_t width, pages, page_shift;
    const int32_t *lens;
    const uint64_t *mask;
    int32_t batch, m, heads, kv, group, dim, rht, qtiles, splits;
    uint32_t signs;              // of the rotation
    float scale;
    void *out;
    int64_t o_token, o_head;
    int32_t out_fp32;
    float *lse;
    int32_t clustered;                   // the splits of a sequence are a cluster, which joins them
    float *part_o, *part_m, *part_l;     // else, splits > 1: of each split and query
};

constexpr int kSplitKeys = 128;      // a split's keys are a multiple of this

// 2^x, within 2 units in the last place; 0 below 2^-126.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Keys [first, last) of a sequence of `len` (at most UFP4_MAX_KEYS, so that a
// tile past its end fits 32 bits) that split s of n takes.
__device__ __forceinline__ int split_keys(int len, int n) {
    return max((len + n - 1) / n + kSplitKeys - 1, kSplitKeys) / kSplitKeys * kSplitKeys;
}
__device__ __forceinline__ void split_range(int len, int s, int n, int &first, int &last) {
    const int per = split_keys(len, n);
    first = (int)min((int64_t)s * per, (int64_t)len);
    last = min(first + per, len);
}

// More than 16 queries a head (rows of 64 or 128 elements): the same results
// by the tensor cores' 128-row tiles.  Splits are joined by the caller.
cudaError_t launch_attn_wide(const AttnArgs &a, int grid, int padded, cudaStream_t s);
constexpr int kWideQueries = 128;

}  // namespace ufp4
