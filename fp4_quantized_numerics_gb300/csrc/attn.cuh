// attn.cuh -- what the two attention kernels over the 4-bit cache share
// (cache.cu: up to 16 queries a head of the cache; attn_wide.cu: more).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "dequant.cuh"
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
// In a branch seldom taken: keeps its arithmetic, which has no effects, from
// being done for every tile and chosen from.
__device__ __forceinline__ void seldom() { asm volatile(""); }

// The weights of the values are probabilities times row scales.  A query's are
// brought into FP16's range by a power of two of its own, 2^-we, as its
// probabilities are by 2^-mx: both follow what the query has seen, by steps.
constexpr int kLeastExponent = -110;     // (of what is held: 2^(14 - e) and 2^(e - 14) are normal)
// What stands for row scales within 2^kEvenScales of one another: the largest.
// (2^10 of the 2^25 to 2^28 that FP16 has below 2^11 to 2^14.  Tokens whose sizes
// differ by 4 and channels by 6 often have more than 2^4 in a tile.)
constexpr int kEvenScales = 10;
// (b >> 23) - 127 as fp32: floor(log2) of the positive number with the bits b.
__device__ __forceinline__ float bits_exponent(uint32_t b) {
    return __uint_as_float(0x4B000000u | b >> 23) - (8388608.0f + 127.0f);
}
// floor(log2) of a row scale (-127: zero, subnormal or not finite).
__device__ __forceinline__ float scale_exponent(float v) { return bits_exponent(finite_bits(v)); }
// The exponent of a power of two.
__device__ __forceinline__ int power_of(float p) { return (int)(__float_as_uint(p) >> 23) - 127; }
struct Rise {
    float mx;
    int we;
    float l_back, o_back;                // what the sums so far are multiplied by
};
// Whether keys whose largest score is `top`, and largest weight 2^(top + w) (its
// exponent, without the scale's fraction), pass what counts by more than
// `slack`; limit: we + slack.  (Differences of scores first, beside which the
// exponents would vanish where scores are large.)
__device__ __forceinline__ bool passes(float mx, float limit, float top, float w, float slack) {
    const float d = top - mx;            // (NaN where neither has seen anything)
    return d > slack || d + w > limit;
}
// mx and we after such keys; or keys that do not pass, but raise the maximum and
// have the largest weight (else a weight of old would be rounded up by each).
__device__ __forceinline__ Rise rise_to(float mx, int we, float top, float w, float slack) {
    const float v = fmaxf(top, mx), back = mx - v;
    const float of_new = floorf(w + (top - v)), of_old = ceilf((float)we + back);
    if (!passes(mx, (float)we + slack, top, w, slack) && !(top > mx && of_new >= of_old))
        return Rise{mx, we, 1.0f, 1.0f};
    // New weights end below 2^(to + 2); what the old ones are given is not less
    // than before, so that sums only shrink.  (Held so that 2^(14 - we) is a
    // normal number; where v is not finite, at a limit.)
    const int to = (int)fminf(fmaxf(fmaxf(of_new, of_old), (float)kLeastExponent), 127.0f);
    return Rise{v, to, exp2_fast(back), exp2_fast(back + (float)(we - to))};
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
