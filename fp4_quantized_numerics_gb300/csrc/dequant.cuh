// dequant.cuh -- 4-bit codes as FP16 matrix operands in registers (gemv.cu,
// cache.cu): the few-token products and the attention multiply quantized
// tensors by unquantized ones with mma.sync, FP16 in and fp32 out.
//
// A grid value times its block's E4M3 scale has at most 7 significant bits and
// lies between 2^-10 and 2688, so FP16 holds it exactly; the tensor or row
// scale, an fp32, is applied to the accumulators.  The other operand is brought
// to FP16 by a power of two (and, where it has more than 11 significant bits,
// as the sum of two FP16 values), so that the products are exact too and the
// sums are fp32's.
//
// Rates measured per SM and clock: 64 lanes of cvt.f16x2.e2m1x2, 123 weights of
// mma.m16n8k16 with 8 columns, 124 (E2M1) and 118 (E1M2) weights of both with
// the scaling between them; a stream at the measured copy bandwidth brings 42.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace ufp4 {

// What a decoded value has to be multiplied by: E1M2's come out as m 2^-9.
template <int GRID>
constexpr float kDecoded = GRID == kE1M2 ? 256.0f : 1.0f;

// 8 codes (a word of a packed row) as 4 FP16 pairs.  E2M1: elements (0,1),
// (2,3), (4,5), (6,7), converted byte by byte.  E1M2: (0,2), (4,6), (1,3),
// (5,7): a code's magnitude and sign moved into a byte are the E4M3 subnormal
// m 2^-9, and two bytes are converted at once.  code_order() is that order.
template <int GRID>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
    if constexpr (GRID == kE1M2) {
        const uint32_t even = (w & 0x07070707u) | ((w << 4) & 0x80808080u);
        const uint32_t odd = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);
        asm("{\n\t.reg .b16 a, b, c, d;\n\t"
            "mov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
            "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(even), "r"(odd));
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
    }
}
// Element (of 8) at place i of decode8's result.
template <int GRID>
__host__ __device__ constexpr int code_order(int i) {
    return GRID == kE1M2 ? (i < 4 ? 2 * i : 2 * i - 7) : i;
}

// The E4M3 byte that `sel` (a byte number in both low nibbles) picks, as an
// FP16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t bytes, uint32_t sel) {
    const uint16_t two = (uint16_t)__byte_perm(bytes, 0, sel);
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    return h;
}
__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two fp32 values as an FP16 pair (a low).
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float2 f16_unpair(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// What rounding two values to the FP16 pair h left, as an FP16 pair (0 beside
// an infinity, which is all there).
__device__ __forceinline__ uint32_t f16_rest(float a, float b, uint32_t h) {
    const float2 f = f16_unpair(h);
    return f16_pair(isinf(f.x) ? 0.0f : a - f.x, isinf(f.y) ? 0.0f : b - f.y);
}

// 16 bytes to shared memory without a register (zeros where `real` is false,
// and nothing is read).
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}

// D += A B: A 16 x 16 (a lane's rows lane/4 and lane/4 + 8), B 16 x 8 (its
// column lane/4), D 16 x 8 fp32 (columns 2 (lane%4) and the next).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^e as fp32 for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The exponent that brings magnitudes up to `bits` (an fp32's, finite) below
// 2^15: floor(log2) held where both 2^(14 - e) and 2^(e - 14) are normal.
__device__ __forceinline__ int top_exponent(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127;
    return e < -110 ? -110 : e;
}
// The bits of a magnitude, 0 for what is not finite.
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// The bits of the largest finite magnitude of 16.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[16]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max3_nan(top, fabsf(v[i]), fabsf(v[i + 1]));
    if (top < __uint_as_float(0x7F800000u)) return __float_as_uint(top);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) bits = max(bits, finite_bits(v[i]));
    return bits;
}

// y = (1/4) H16 diag(d) x, in the order of ufp4_quantize's butterflies; and
// its inverse.  Bit j of `signs` set: d_j = -1.
__device__ __forceinline__ void rotate16(float (&v)[16], uint32_t signs) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) ^ ((signs << (31 - i)) & 0x80000000u));
    fwht16(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= 0.25f;
}
__device__ __forceinline__ void rotate16_back(float (&v)[16], uint32_t signs) {
    fwht16(v);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(__float_as_uint(v[i] * 0.25f) ^ ((signs << (31 - i)) & 0x80000000u));
}

}  // namespace ufp4
