// rowops.cuh -- pieces shared by the row-wise operators around the grouped
// GEMMs (moe.cu, activation.cu): how a thread finds and reads its part of a
// row, and the division that turns a flat work index into (row, part).
//
// Two layouts, chosen by alignment (`whole`):
//  * whole: a thread owns N consecutive elements, in accesses of 16 or 32
//    bytes on such boundaries; rows are multiples of N long.
//  * strided (anything else): a warp owns 32 N consecutive elements of a row,
//    lane l the elements l, l + 32, ...: every access of the warp is one run
//    of neighbouring elements, whatever the row's alignment, and the work of
//    finding the place is shared by N elements.
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

// ------------------------------------------------------- 16 and 32 bytes
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[4]) {
    const uint4 v = __ldg(static_cast<const uint4 *>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[8]) {
    asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
}
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[4]) {
    *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
}

// ------------------------------------------- N consecutive elements as fp32
template <int N>
__device__ __forceinline__ void load_whole(const __nv_bfloat16 *p, float (&f)[N]) {
    uint32_t w[N / 2];
    load_words(p, w);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <int N>
__device__ __forceinline__ void load_whole(const float *p, float (&f)[N]) {
#pragma unroll
    for (int h = 0; h < N / 8; ++h) {
        uint32_t w[8];
        load_words(p + 8 * h, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 * h + i] = __uint_as_float(w[i]);
    }
}
// Rounds to nearest even, once, on the way out.
template <int N>
__device__ __forceinline__ void store_whole(__nv_bfloat16 *p, const float (&f)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    store_words(p, w);
}
template <int N>
__device__ __forceinline__ void store_whole(float *p, const float (&f)[N]) {
#pragma unroll
    for (int h = 0; h < N / 8; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[8 * h + i]);
        store_words(p + 8 * h, w);
    }
}

__device__ __forceinline__ float load_one(const __nv_bfloat16 *p) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short *>(p)) << 16);
}
__device__ __forceinline__ float load_one(const float *p) { return __ldg(p); }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }

// ---------------------------------------------------------- a thread's part
// Elements col, col + kStep, ... of a row of `cols` (those below cols; in the
// whole layout all N or none).
template <bool WHOLE, int N>
struct Part {
    static constexpr uint32_t kStep = WHOLE ? 1 : 32;
    uint32_t col, cols;

    __device__ __forceinline__ bool has(int i) const { return col + i * kStep < cols; }
    template <class T>
    __device__ __forceinline__ void load(const T *row, float (&f)[N]) const {
        if constexpr (WHOLE) {
            load_whole<N>(row + col, f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = has(i) ? load_one(row + col + i * kStep) : 0.0f;
        }
    }
    template <class T>
    __device__ __forceinline__ void store(T *row, const float (&f)[N]) const {
        if constexpr (WHOLE) {
            store_whole<N>(row + col, f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (has(i)) store_one(row + col + i * kStep, f[i]);
        }
    }
};

// Units of work in a row: threads' parts (whole) or warps' segments.
inline uint32_t units_of(bool whole, int n, int64_t cols) {
    const int64_t per = whole ? n : 32 * n;
    return (uint32_t)((cols + per - 1) / per);
}

// Whether a tensor (row stride ld elements of esz bytes) allows whole parts of
// n elements: its accesses are n * esz bytes, at most 32.
inline bool whole_rows(const void *p, int64_t ld, size_t esz, int n) {
    const size_t a = n * esz < 32 ? n * esz : 32;
    return reinterpret_cast<uintptr_t>(p) % a == 0 && (size_t)ld * esz % a == 0;
}

// Calls f with a null pointer of the element type of `dtype` (0 BF16, 1 FP32).
template <class F>
auto by_type(int dtype, F f) {
    return dtype == 0 ? f(static_cast<__nv_bfloat16 *>(nullptr)) : f(static_cast<float *>(nullptr));
}
inline size_t type_size(int dtype) { return dtype == 0 ? 2 : 4; }
template <class P>
using Elem = std::remove_pointer_t<P>;
template <class F>
auto by_bool(bool b, F f) {
    return b ? f(std::true_type()) : f(std::false_type());
}

}  // namespace ufp4
