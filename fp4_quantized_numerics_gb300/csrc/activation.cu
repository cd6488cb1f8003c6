// activation.cu -- the gated activation of an expert's feed-forward layer and
// the 8-bit checkpoints its backward pass reads.  The contract (formats,
// layouts, formulas) is in include/ufp4.h; the pages give no kernels for it.
//
// The dual quantizer already leaves the GEMM operands of the backward pass in
// 4 bits; what the gated activation's own gradient needs is gate and up,
// 8 bytes an element pair in fp32.  At 8 bits and a scale byte per 32 they
// cost 2.06 bytes, written by the pass that reads them anyway.  Scales are
// powers of two, so that dividing by them and multiplying back are exact and
// the restored values are exact in bf16 as well.
//
// Bound by memory: at most 3 instructions a byte moved.  One GB300, "of
// measured" is of the 6676 GB/s of a plain copy:
//   98304 x 1408, fp32 in, BF16 out, INT8 kept:
//     k_swiglu 233 us, 7.2 TB/s (107 %; reads run faster than a copy), without
//     checkpoints 190 us; k_swiglu_bwd 197 us (106 %);
//   65536 x 8192 BF16: k_ckpt_save 243 us (INT8; E4M3 228; 100 and 107 %),
//     k_ckpt_load 229 us (106 %).
// With 8 elements a thread k_ckpt_save takes 321 us (E4M3 301) and k_ckpt_load
// 277: too few bytes in flight, and the scale's arithmetic shared by half as
// many elements.  The activation's kernels, which hold more, take the same.
//
// In the whole layout (rowops.cuh) a thread owns 16 consecutive elements (8
// where rows allow no more) and two (four) neighbouring lanes one 32-element
// block; in pairs a half warp owns each
// block, in singles the warp.  Those two are bound by instructions (72 % of
// the issue slots in k_ckpt_save): 65536 x 1002 and 1001 BF16 58 and 64 us
// saved (52 and 47 % of measured; with a warp reduction per block 72 and 64),
// 49 and 52 us restored; x 1000 (whole, by eights) 43 and 38 us, in fp32 49
// and 49 us (100 %).  The activation on 49152 rows of 1002, 1001 and 1000
// BF16: forward 90, 109 and 69 us (66, 55 and 86 %), without checkpoints 45,
// 57 and 43, backward 94, 119 and 68 us (63, 50 and 88 %).
#include "common.cuh"
#include "internal.h"
#include "rowops.cuh"

#include <cuda_fp16.h>

#include <initializer_list>
#include <type_traits>

namespace ufp4 {

namespace {

// 256 threads a CTA are up to 10 % slower where the launch counts and 3-6 % on
// BF16 tensors, 64 up to 80 % (too few resident warps for the lighter kernels).
constexpr int kThreads = 128;
constexpr int kInt8 = 0, kE4M3 = 1, kNone = -1;

// ------------------------------------------------------------ block scales
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Scale byte of a block from the bits of its largest magnitude (as integers
// magnitudes compare like the floats, and a NaN is above all).
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    const int e = (int)(top >> 23) + (FMT == kE4M3 && (top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)min(max(e - (FMT == kE4M3 ? 8 : 6), 0), FMT == kE4M3 ? 246 : 248);
}
// 2^(127 - b); 0 for the non-finite block, whose codes are 0.
__device__ __forceinline__ float scale_inv(uint32_t b) { return __uint_as_float(b == 255u ? 0u : (254u - b) << 23); }
// 2^(b - 127); NaN for the non-finite block.
__device__ __forceinline__ float scale_of(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FC00000u) : e8m0_to_f32(b);
}

// The 8-bit code of x (already in units of the scale), in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t code_of(float x) {
    if constexpr (FMT == kInt8) {
        // sign(x) min(|x|, 127); then adding 1.5 * 2^23 rounds to an integer,
        // ties to even, whose two's complement is in the low mantissa bits
        float c;
        asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(c) : "f"(x), "f"(127.0f));
        return __float_as_uint(__fadd_rn(c, 12582912.0f));
    } else {
        return e4m3_from_f32(x);
    }
}
// The code of x under the factor scale_inv gave its block.
template <int FMT>
__device__ __forceinline__ uint32_t block_code(float x, float inv) {
    return inv == 0.0f ? 0u : code_of<FMT>(x * inv) & 0xFFu;
}
// Codes of 4 elements, the first in the lowest byte.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float *x, float inv) {
    if constexpr (FMT == kInt8) {
        const uint32_t lo = __byte_perm(code_of<FMT>(x[0] * inv), code_of<FMT>(x[1] * inv), 0x0040);
        const uint32_t hi = __byte_perm(code_of<FMT>(x[2] * inv), code_of<FMT>(x[3] * inv), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * inv), "f"(x[0] * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * inv), "f"(x[2] * inv));
        return (uint32_t)hi << 16 | lo;
    }
}

template <int FMT>
__device__ __forceinline__ float value_of(uint32_t code, float scale) {
    if constexpr (FMT == kInt8) return (float)(int8_t)code * scale;
    else return e4m3_to_f32(code) * scale;
}
// Values of 4 codes.
template <int FMT>
__device__ __forceinline__ void values4(uint32_t w, float scale, float *x) {
    if constexpr (FMT == kInt8) {
        // code + 128 in the low mantissa bits of 2^23, then 2^23 + 128 taken off
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.0f) * scale;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
    }
}

// ------------------------------------------------------------- activation
// silu(g) u and the gradients, by e = exp(-g) and 1 / (1 + e).  Below g = -80,
// before exp(-g) leaves fp32's range (at 88.7), e is exp(g / 2) instead: there
// 1 / (1 + exp(-g)) is exp(g) = e e to fp32's precision (and 1 + e is 1), and
// as the results, products with it, need not be small, each of two factors
// takes one e, its `tail`, which is 1 above.
//
// EXACT (fp32 results): the library's exp and division; otherwise 2^x and the
// reciprocal as the hardware gives them, whose relative error (in all within
// (6 + |g|) 2^-23) disappears in the rounding to bf16.
__device__ __forceinline__ bool far(float g) { return g < -80.0f; }
template <bool EXACT>
__device__ __forceinline__ float exp_of(float g) {
    if constexpr (EXACT) {
        return expf(g * (far(g) ? 0.5f : -1.0f));
    } else {
        constexpr float kLog2e = 1.4426950408889634f;
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * (far(g) ? 0.5f * kLog2e : -kLog2e)));
        return e;
    }
}
template <bool EXACT>
__device__ __forceinline__ float quotient(float a, float b) {
    if constexpr (EXACT) {
        return a / b;
    } else {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b));
        return a * r;
    }
}
template <bool EXACT>
__device__ __forceinline__ float gated(float g, float u) {
    const float e = exp_of<EXACT>(g), tail = far(g) ? e : 1.0f;
    return quotient<EXACT>(g * tail, 1.0f + e) * (u * tail);
}
// In place: u becomes the gradient of d silu(g) u by g, and g that by u.
template <bool EXACT>
__device__ __forceinline__ void gated_bwd(float d, float &g, float &u) {
    const float e = exp_of<EXACT>(g), tail = far(g) ? e : 1.0f;
    const float s = quotient<EXACT>(1.0f, 1.0f + e) * tail, gs = g * s;   // (where tail is not 1, 1 - s is)
    d *= tail;
    u = d * u * fmaf(gs, 1.0f - s, s);
    g = d * gs;
}

// ------------------------------------------------------------------- work
// The row and part a thread owns.  All lanes of a block are in or out together.
template <int L, int N>
struct Place {
    int64_t row;
    Part<L, N> part;

    __device__ __forceinline__ Place(RowDiv parts, uint32_t cols, uint64_t i)
        : row((int64_t)row_of(i, parts)), part((uint32_t)(i - (uint64_t)row * parts.d), cols) {}
};
template <int L>
__device__ __forceinline__ uint64_t part_index() {
    const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    return L == kWhole ? i : i / 32;
}

// max(|a|, |b|, |c|), NaN if any is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Bits of the block's largest magnitude, over the 32 / N lanes that hold it;
// NaN above all.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(const float (&x)[N]) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i + 1 < N; i += 2) m = max3_abs(m, x[i], x[i + 1]);
    m = max3_abs(m, x[N - 1], 0.0f);
    uint32_t a = __float_as_uint(m) & 0x7FFFFFFFu;
    constexpr uint32_t kLanes = 32 / N, kOne = (1u << kLanes) - 1u;
    const uint32_t lanes = kOne << (threadIdx.x & (32u - kLanes));
#pragma unroll
    for (uint32_t d = 1; d < kLanes; d <<= 1) a = max(a, __shfl_xor_sync(lanes, a, d));
    return a;
}

// Writes the checkpoint of this thread's elements (0 where it has none).
template <int FMT, int L, int N>
__device__ __forceinline__ void keep(const float (&x)[N], const Place<L, N> &p, const Ckpt &c, int64_t ld,
                                     uint32_t nb) {
    const uint32_t col = p.part.col;
    uint8_t *codes = c.codes + p.row * ld + col, *scales = c.scales + p.row * nb + col / 32;
    if constexpr (L == kWhole) {
        const uint32_t b = scale_byte<FMT>(lanes_max(x));
        const float inv = scale_inv(b);
        if (col % 32 == 0) *scales = (uint8_t)b;
        if (!p.part.has(0)) return;
        uint32_t w[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i) w[i] = b == 255u ? 0u : codes4<FMT>(x + 4 * i, inv);
        store_words(codes, w);
    } else {
        // 8 / kStep maxima over 32 / kStep lanes: three (two) exchanges that
        // halve their number and two that join; lanes 4 k .. 4 k + 3 of a
        // block's lanes end up with the k-th, turn it into a scale, and the
        // others take the factor from there
        constexpr int kStep = L == kPairs ? 2 : 1, kLanes = 32 / kStep;
        const uint32_t lane = threadIdx.x & 31u, first = lane & ~(kLanes - 1u), k = lane % kLanes / 4;
        uint32_t m[8 / kStep];
#pragma unroll
        for (int i = 0; i < 8; i += kStep)
            m[i / kStep] = kStep == 2 ? max(abs_bits(x[i]), abs_bits(x[i + kStep - 1])) : abs_bits(x[i]);
#pragma unroll
        for (int n = 4 / kStep, d = kLanes / 2; n; n /= 2, d /= 2) {
            const bool upper = lane & d;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const uint32_t mine = upper ? m[i + n] : m[i], theirs = upper ? m[i] : m[i + n];
                m[i] = max(mine, __shfl_xor_sync(0xFFFFFFFFu, theirs, d));
            }
        }
        m[0] = max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 2));
        m[0] = max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
        const uint32_t b = scale_byte<FMT>(m[0]);
        const uint32_t start = col - kStep * (lane - first) + p.part.at((int)k * kStep);   // of the k-th block
        if (lane % 4 == 0 && start < p.part.cols) scales[k * kStep] = (uint8_t)b;
        const float inv = scale_inv(b);
#pragma unroll
        for (int i = 0; i < 8; i += kStep) {
            const float f = __shfl_sync(0xFFFFFFFFu, inv, first + 4 * (i / kStep));
            if (!p.part.has(i)) continue;
            const uint32_t c0 = block_code<FMT>(x[i], f);
            if constexpr (kStep == 2)
                *reinterpret_cast<uint16_t *>(codes + p.part.at(i)) =
                    (uint16_t)(block_code<FMT>(x[i + 1], f) << 8 | c0);
            else
                codes[p.part.at(i)] = (uint8_t)c0;
        }
    }
}
template <int FMT, int L, int N>
__device__ __forceinline__ void restore(const Ckpt &c, const Place<L, N> &p, int64_t ld, uint32_t nb,
                                        float (&x)[N]) {
    const uint32_t col = p.part.col;
    const uint8_t *codes = c.codes + p.row * ld + col, *scales = c.scales + p.row * nb + col / 32;
    if constexpr (L == kWhole) {
        uint32_t w[N / 4];
        load_words(codes, w);
        const float s = scale_of(*scales);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) values4<FMT>(w[i], s, x + 4 * i);
    } else {
        constexpr int kStep = L == kPairs ? 2 : 1, kLanes = 32 / kStep;
        const uint32_t lane = threadIdx.x & 31u, k = lane % kLanes, first = lane - k;
        const uint32_t lanes = kLanes == 32 ? 0xFFFFFFFFu : 0xFFFFu << first;
        float mine = 0.0f;   // lane k: the scale of the k-th block
        if (k < 8 / kStep && (col - kStep * k) + p.part.at((int)k * kStep) < p.part.cols)
            mine = scale_of(scales[k * kStep]);
        uint32_t w[8 / kStep];
#pragma unroll
        for (int i = 0; i < 8; i += kStep) {
            if constexpr (kStep == 2)
                w[i / 2] = p.part.has(i) ? *reinterpret_cast<const uint16_t *>(codes + p.part.at(i)) : 0u;
            else
                w[i] = p.part.has(i) ? codes[p.part.at(i)] : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; i += kStep) {
            const float s = __shfl_sync(lanes, mine, first + i / kStep);
            x[i] = value_of<FMT>(w[i / kStep] & 0xFFu, s);
            if constexpr (kStep == 2) x[i + 1] = value_of<FMT>(w[i / 2] >> 8, s);
        }
    }
}

// ---------------------------------------------------------------- kernels
template <class T, int FMT, int L, int N>
__global__ void __launch_bounds__(kThreads) k_ckpt_save(const T *x, int64_t ld, Ckpt c, int64_t ldc,
                                                        uint32_t cols, uint32_t nb, RowDiv parts, uint64_t work) {
    const uint32_t zero = begin_in_order();
    // (with an early return for the threads past the end, the eights of a
    // 65536 x 1000 BF16 tensor take 57 us instead of 44)
    const uint64_t i = part_index<L>() + zero;
    const Place<L, N> p(parts, cols, i);
    float v[N] = {};
    if (i < work && (L != kWhole || p.part.has(0))) p.part.load(x + p.row * ld, v);
    if (i < work) keep<FMT>(v, p, c, ldc, nb);
}

template <class T, int FMT, int L, int N>
__global__ void __launch_bounds__(kThreads) k_ckpt_load(Ckpt c, int64_t ldc, T *__restrict__ x, int64_t ld,
                                                        uint32_t cols, uint32_t nb, RowDiv parts, uint64_t work) {
    const uint32_t zero = begin_in_order();
    const uint64_t i = part_index<L>() + zero;
    if (i >= work) return;
    const Place<L, N> p(parts, cols, i);
    if (L == kWhole && !p.part.has(0)) return;
    float v[N];
    restore<FMT>(c, p, ldc, nb, v);
    p.part.store(x + p.row * ld, v);
}

template <class Ti, class To, int FMT, int L, int N>
__global__ void __launch_bounds__(kThreads) k_swiglu(const Ti *gate, int64_t ld_gate,
                                                     const Ti *up, int64_t ld_up, To *__restrict__ h,
                                                     int64_t ld_h, Ckpt cg, Ckpt cu, int64_t ldc, uint32_t cols,
                                                     uint32_t nb, RowDiv parts, uint64_t work) {
    constexpr bool kExact = std::is_same<To, float>::value;
    const uint32_t zero = begin_in_order();
    const uint64_t i = part_index<L>() + zero;
    if (i >= work) return;
    const Place<L, N> p(parts, cols, i);
    float g[N] = {}, u[N] = {};
    const bool in = L != kWhole || p.part.has(0);
    if (in) {
        p.part.load(gate + p.row * ld_gate, g);
        p.part.load(up + p.row * ld_up, u);
    }
    const auto keep_both = [&] {
        if constexpr (FMT != kNone) {
            keep<FMT>(g, p, cg, ldc, nb);
            keep<FMT>(u, p, cu, ldc, nb);
        }
    };
    // (49152 x 1001 BF16 in the other order 117 us instead of 109; in the whole
    // layout, checkpoints first, 98304 x 1408 233 us both ways, x 1000 72, not 69)
    if constexpr (L != kWhole) keep_both();
    if (in) {
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = gated<kExact>(g[e], u[e]);
        p.part.store(h + p.row * ld_h, o);
    }
    if constexpr (L == kWhole) keep_both();
}

template <class Td, class To, int FMT, int L, int N>
__global__ void __launch_bounds__(kThreads) k_swiglu_bwd(const Td *dh, int64_t ld_dh, Ckpt cg, Ckpt cu,
                                                         int64_t ldc, To *__restrict__ dgate, int64_t ld_dgate,
                                                         To *__restrict__ dup, int64_t ld_dup, uint32_t cols,
                                                         uint32_t nb, RowDiv parts, uint64_t work) {
    constexpr bool kExact = std::is_same<To, float>::value;
    const uint32_t zero = begin_in_order();
    const uint64_t i = part_index<L>() + zero;
    if (i >= work) return;
    const Place<L, N> p(parts, cols, i);
    if (L == kWhole && !p.part.has(0)) return;
    float d[N], g[N], u[N];
    p.part.load(dh + p.row * ld_dh, d);
    restore<FMT>(cg, p, ldc, nb, g);
    restore<FMT>(cu, p, ldc, nb, u);
#pragma unroll
    for (int e = 0; e < N; ++e) gated_bwd<kExact>(d[e], g[e], u[e]);
    p.part.store(dgate + p.row * ld_dgate, u);
    p.part.store(dup + p.row * ld_dup, g);
}

// -------------------------------------------------------------- launching
// The work over rows x cols in one of the layouts: the widest that all of
// `tensors` allow.
struct Tensor {
    const void *p;
    int64_t ld;
    int dtype;
};
struct Grid {
    int layout, elems;
    uint32_t nb;       // blocks of a row
    RowDiv parts;
    uint64_t work;
    unsigned ctas;
};
Grid grid_of(int64_t rows, int64_t cols, std::initializer_list<Tensor> tensors) {
    const auto by = [&](int n) {
        for (const Tensor &t : tensors)
            if (!rows_by(t.p, t.ld, type_size(t.dtype), n)) return false;
        return cols % n == 0;
    };
    Grid g;
    g.layout = by(16) || by(8) ? kWhole : by(2) ? kPairs : kSingles;
    g.elems = by(16) ? 16 : 8;
    g.nb = (uint32_t)((cols + 31) / 32);
    // whole: parts for all of the last block, so that its lanes are all there
    const uint32_t parts = g.layout == kWhole ? 32 / g.elems * g.nb : parts_of(g.layout, g.elems, cols);
    g.parts = make_rowdiv(parts);
    g.work = (uint64_t)rows * parts;
    g.ctas = (unsigned)((threads_of(g.layout, g.work) + kThreads - 1) / kThreads);
    return g;
}
// Calls f with the layout and the elements of a thread.
template <class F>
void by_layout(const Grid &g, F f) {
    if (g.layout == kWhole && g.elems == 16) f(Int<kWhole>(), Int<16>());
    else if (g.layout == kWhole) f(Int<kWhole>(), Int<8>());
    else if (g.layout == kPairs) f(Int<kPairs>(), Int<8>());
    else f(Int<kSingles>(), Int<8>());
}
template <class F>
void by_format(int fmt, F f) {
    if (fmt == kInt8) f(Int<kInt8>());
    else f(Int<kE4M3>());
}

}  // namespace

cudaError_t launch_ckpt_save(const void *x, int dtype, int64_t ld, const Ckpt &c, int fmt, int64_t rows, int64_t cols,
                             cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const Grid g = grid_of(rows, cols, {{x, ld, dtype}});
    by_type(dtype, [&](auto *t) {
        using T = Elem<decltype(t)>;
        by_format(fmt, [&](auto f) {
            by_layout(g, [&](auto w, auto n) {
                e = launch_in_order(k_ckpt_save<T, decltype(f)::value, decltype(w)::value, decltype(n)::value>, g.ctas,
                                    kThreads, s, static_cast<const T *>(x), ld, c, ckpt_ld(cols), cols, g.nb, g.parts,
                                    g.work);
            });
        });
    });
    return e;
}

cudaError_t launch_ckpt_load(const Ckpt &c, int fmt, int64_t rows, int64_t cols, void *x, int dtype, int64_t ld,
                             cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const Grid g = grid_of(rows, cols, {{x, ld, dtype}});
    by_type(dtype, [&](auto *t) {
        using T = Elem<decltype(t)>;
        by_format(fmt, [&](auto f) {
            by_layout(g, [&](auto w, auto n) {
                e = launch_in_order(k_ckpt_load<T, decltype(f)::value, decltype(w)::value, decltype(n)::value>, g.ctas,
                                    kThreads, s, c, ckpt_ld(cols), static_cast<T *>(x), ld, cols, g.nb, g.parts,
                                    g.work);
            });
        });
    });
    return e;
}

cudaError_t launch_swiglu(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int in_dtype,
                          int64_t rows, int64_t cols, void *h, int h_dtype, int64_t ld_h, const Ckpt &cg,
                          const Ckpt &cu, int fmt, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const Grid gr = grid_of(rows, cols, {{gate, ld_gate, in_dtype}, {up, ld_up, in_dtype}, {h, ld_h, h_dtype}});
    by_type(in_dtype, [&](auto *ti) {
        using Ti = Elem<decltype(ti)>;
        by_type(h_dtype, [&](auto *to) {
            using To = Elem<decltype(to)>;
            by_layout(gr, [&](auto w, auto n) {
                auto go = [&](auto f) {
                    e = launch_in_order(k_swiglu<Ti, To, decltype(f)::value, decltype(w)::value, decltype(n)::value>,
                                        gr.ctas, kThreads, s, static_cast<const Ti *>(gate), ld_gate,
                                        static_cast<const Ti *>(up), ld_up, static_cast<To *>(h), ld_h, cg, cu,
                                        ckpt_ld(cols), cols, gr.nb, gr.parts, gr.work);
                };
                if (fmt == kNone) go(Int<kNone>());
                else by_format(fmt, go);
            });
        });
    });
    return e;
}

cudaError_t launch_swiglu_bwd(const void *dh, int dh_dtype, int64_t ld_dh, const Ckpt &cg, const Ckpt &cu, int fmt,
                              int64_t rows, int64_t cols, void *dgate, int64_t ld_dgate, void *dup, int64_t ld_dup,
                              int out_dtype, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const Grid g = grid_of(rows, cols, {{dh, ld_dh, dh_dtype}, {dgate, ld_dgate, out_dtype}, {dup, ld_dup, out_dtype}});
    by_type(dh_dtype, [&](auto *td) {
        using Td = Elem<decltype(td)>;
        by_type(out_dtype, [&](auto *to) {
            using To = Elem<decltype(to)>;
            by_format(fmt, [&](auto f) {
                by_layout(g, [&](auto w, auto n) {
                    constexpr int kL = decltype(w)::value, N = decltype(n)::value;
                    e = launch_in_order(k_swiglu_bwd<Td, To, decltype(f)::value, kL, N>, g.ctas, kThreads, s,
                                        static_cast<const Td *>(dh), ld_dh, cg, cu, ckpt_ld(cols),
                                        static_cast<To *>(dgate), ld_dgate, static_cast<To *>(dup), ld_dup, cols, g.nb,
                                        g.parts, g.work);
                });
            });
        });
    });
    return e;
}

}  // namespace ufp4
