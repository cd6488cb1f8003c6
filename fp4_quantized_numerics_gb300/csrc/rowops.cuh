// rowops.cuh -- pieces shared by the row-wise operators around the grouped
// GEMMs (moe.cu, activation.cu): vectors of row elements as fp32, and the
// division that turns a flat work index into (row, place in the row).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <type_traits>

namespace ufp4 {

// n / d by a multiplication: q = floor(n m / 2^64) with m = ceil(2^64 / d).
// m d exceeds 2^64 by less than d, so q is exact while n d < 2^64; the entry
// points' limits (rows x width < 2^38, width <= 2^24) keep it there.
struct RowDiv {
    uint64_t m;    // 0 stands for d = 1
    uint32_t d;
};
inline RowDiv make_rowdiv(uint32_t d) { return RowDiv{d == 1 ? 0 : ~0ull / d + 1, d}; }
__device__ __forceinline__ uint64_t row_of(uint64_t n, RowDiv f) { return f.m ? __umul64hi(n, f.m) : n; }

// V consecutive elements to and from fp32 registers: V = 8 in 16-byte
// accesses (the pointer 16-byte aligned), V = 1 by element.
template <int V>
__device__ __forceinline__ void load_f32(const __nv_bfloat16 *p, float (&f)[V]) {
    static_assert(V == 8 || V == 1, "vector of 8 or single element");
    if constexpr (V == 8) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
        f[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void load_f32(const float *p, float (&f)[V]) {
    if constexpr (V == 8) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        f[0] = __ldg(p);
    }
}

// Rounds to nearest even, once, on the way out.
template <int V>
__device__ __forceinline__ void store_f32(__nv_bfloat16 *p, const float (&f)[V]) {
    if constexpr (V == 8) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        *p = __float2bfloat16_rn(f[0]);
    }
}
template <int V>
__device__ __forceinline__ void store_f32(float *p, const float (&f)[V]) {
    if constexpr (V == 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *p = f[0];
    }
}

// Whether a tensor of `cols` elements of esz bytes a row (stride ld elements)
// can be taken in vectors of 8.
inline bool vec8(const void *p, int64_t ld, int64_t cols, size_t esz) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * (int64_t)esz) % 16 == 0 && cols % 8 == 0;
}

// Calls f with a null pointer of the element type of `dtype` (0 BF16, 1 FP32).
template <class F>
void by_type(int dtype, F f) {
    if (dtype == 0) f(static_cast<__nv_bfloat16 *>(nullptr));
    else f(static_cast<float *>(nullptr));
}

}  // namespace ufp4
