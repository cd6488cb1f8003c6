// rowops.cuh -- pieces shared by the row-wise operators around the grouped
// GEMMs (moe.cu, activation.cu): how a thread finds and reads its part of a
// row, and the division that turns a flat work index into (row, part).
//
// Three layouts, chosen by alignment:
//  * kWhole: a thread owns N consecutive elements, in accesses of 16 or 32
//    bytes on such boundaries; rows are multiples of N long.
//  * kPairs (rows on two-element boundaries, of even length) and kSingles
//    (anything): a warp owns 32 N consecutive elements of a row, a lane two
//    neighbours (or one) of every 64 (32): every access of the warp is one run
//    of neighbouring elements, and finding the place is shared by N elements.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include <type_traits>

namespace ufp4 {

// The row kernels are launched with programmatic stream serialization: the
// grid is set up while the last CTAs of the kernel before it in the stream
// end.  Each begins by waiting until its predecessor has completed and its
// writes are visible; nothing but parameters is read before, and every CTA
// waits, so a kernel's end implies the end of all before it.  Against plain
// launches, back to back: 3 to 5 us less between a pass's kernels of 80 to
// 430 us; 493 x 1408 gated forward 2.6 -> 2.2 us, 128 tokens' combine gradient
// 4.2 -> 4.0 us.  Allowing the successor explicitly from the start makes the
// short kernels slower (2.9, 4.6 us): its waiting CTAs take the SMs early.
//
// Returns 0 out of the asm statement: added to the index that every address is
// made from, it keeps the front end, to which the value is unknown, from
// moving loads above the wait, whatever it may assume of the data.  Behind the
// front end the order is the instruction's own: no access to memory passes
// griddepcontrol.wait.  (Outputs are __restrict__, so that loads move past
// stores; inputs are not, which would make their loads non-coherent ones.)
__device__ __forceinline__ uint32_t begin_in_order() {
    uint32_t zero;
    asm volatile("griddepcontrol.wait;\n\tmov.u32 %0, 0;" : "=r"(zero)::"memory");
    return zero;
}
// (grid: a multiple of `cluster` CTAs in y; 1: none)
template <class... Params, class... Args>
cudaError_t launch_in_order_smem(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, unsigned cluster,
                                 cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = cluster;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
template <class... Params, class... Args>
cudaError_t launch_in_order(void (*kernel)(Params...), uint64_t grid, unsigned block, cudaStream_t s, Args... args) {
    return launch_in_order_smem(kernel, dim3((unsigned)grid), block, 0, 1, s, args...);
}

// n / d by a multiplication: q = floor(n m / 2^64) with m = ceil(2^64 / d).
// m d exceeds 2^64 by less than d, so q is exact while n d < 2^64; the entry
// points' limits (rows x width < 2^38, width <= 2^24) keep it there.
struct RowDiv {
    uint64_t m;    // 0 stands for d = 1
    uint32_t d;
};
inline RowDiv make_rowdiv(uint32_t d) { return RowDiv{d == 1 ? 0 : ~0ull / d + 1, d}; }
__device__ __forceinline__ uint64_t row_of(uint64_t n, RowDiv f) { return f.m ? __umul64hi(n, f.m) : n; }

// ------------------------------------------------------ 8, 16 and 32 bytes
// Plain loads, not the non-coherent kind (__ldg), whose data has to stay as it
// is from the launch on: these kernels are launched before their inputs are
// complete.
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[2]) {
    const uint2 v = *static_cast<const uint2 *>(p);
    w[0] = v.x; w[1] = v.y;
}
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[4]) {
    const uint4 v = *static_cast<const uint4 *>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}
__device__ __forceinline__ void load_words(const void *p, uint32_t (&w)[8]) {
    asm("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
}
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[2]) {
    *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
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
// As they lie in memory (N of 16 bits, or 8 of 32 bits a half): what a thread
// holds while a load is under way.
template <class T, int N>
struct Raw {
    uint32_t w[N * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T *p) {
        constexpr int kWords = N * sizeof(T) / 4;
        if constexpr (kWords <= 8) {
            load_words(p, w);
        } else {
            uint32_t a[8], b[8];
            load_words(p, a);
            load_words(p + 8, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = a[i];
                w[8 + i] = b[i];
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};
template <int N, class T>
__device__ __forceinline__ void load_whole(const T *p, float (&f)[N]) {
    Raw<T, N> r;
    r.load(p);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = r[i];
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
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}
__device__ __forceinline__ float load_one(const float *p) { return *p; }
__device__ __forceinline__ float2 load_two(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 load_two(const float *p) {
    return *reinterpret_cast<const float2 *>(p);
}
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_two(__nv_bfloat16 *p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store_two(float *p, float a, float b) {
    *reinterpret_cast<float2 *>(p) = make_float2(a, b);
}

// ---------------------------------------------------------- a thread's part
constexpr int kWhole = 0, kPairs = 1, kSingles = 2;

// N elements of a row of `cols`, from `col`: those for which has(i).
template <int L, int N>
struct Part {
    uint32_t col, cols;

    // Part u of a row (kWhole: this thread's; else this warp's).
    __device__ __forceinline__ Part(uint32_t u, uint32_t cols_) : cols(cols_) {
        const uint32_t lane = threadIdx.x & 31u;
        col = L == kWhole ? u * N : u * (32 * N) + (L == kPairs ? 2 * lane : lane);
    }
    // Offset of element i from col.
    static __device__ __forceinline__ constexpr uint32_t at(int i) {
        return L == kWhole ? i : L == kPairs ? i / 2 * 64 + i % 2 : i * 32;
    }
    __device__ __forceinline__ bool has(int i) const { return col + at(i) < cols; }
    template <class T>
    __device__ __forceinline__ void load(const T *row, float (&f)[N]) const {
        const T *p = row + col;
        if constexpr (L == kWhole) {
            load_whole<N>(p, f);
        } else if constexpr (L == kPairs) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 v = has(i) ? load_two(p + at(i)) : make_float2(0.0f, 0.0f);
                f[i] = v.x;
                f[i + 1] = v.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = has(i) ? load_one(p + at(i)) : 0.0f;
        }
    }
    template <class T>
    __device__ __forceinline__ void store(T *row, const float (&f)[N]) const {
        T *p = row + col;
        if constexpr (L == kWhole) {
            store_whole<N>(p, f);
        } else if constexpr (L == kPairs) {
#pragma unroll
            for (int i = 0; i < N; i += 2)
                if (has(i)) store_two(p + at(i), f[i], f[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (has(i)) store_one(p + at(i), f[i]);
        }
    }
};

// Parts of a row.
inline uint32_t parts_of(int layout, int n, int64_t cols) {
    const int64_t per = layout == kWhole ? n : 32 * n;
    return (uint32_t)((cols + per - 1) / per);
}
// Threads of `parts` parts.
inline uint64_t threads_of(int layout, uint64_t parts) { return layout == kWhole ? parts : parts * 32; }

// Whether a tensor (row stride ld elements of esz bytes) can be accessed n
// elements at a time, in at most 32 bytes.
inline bool rows_by(const void *p, int64_t ld, size_t esz, int n) {
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
template <int N>
using Int = std::integral_constant<int, N>;

}  // namespace ufp4
