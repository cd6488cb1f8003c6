// activation.cu -- the gated activation of an expert's feed-forward layer and
// the 8-bit checkpoints its backward pass reads.  The contract (formats,
// layouts, formulas) is in include/ufp4.h; the pages give no kernels for it.
//
// The dual quantizer already leaves the GEMM operands of the backward pass in
// 4 bits; what the gated activation's own gradient needs is gate and up,
// 8 bytes an element pair in fp32.  At 8 bits and a scale byte per 32 they
// cost 2.06 bytes, written by the pass that reads them anyway.
//
// Two layouts of the work, chosen by alignment:
//  * quads: a thread owns 8 consecutive elements (16-byte accesses), four
//    neighbouring lanes one 32-element block, whose maximum takes two shuffles;
//  * lanes (rows that are not 16-byte aligned or not a multiple of 8 long): a
//    warp owns a block, a lane one element.
#include "common.cuh"
#include "internal.h"
#include "rowops.cuh"

#include <type_traits>

namespace ufp4 {

namespace {

constexpr int kThreads = 256;
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
    if constexpr (FMT == kInt8)
        // adding 1.5 * 2^23 rounds to an integer, ties to even, whose two's
        // complement is then in the low mantissa bits (a NaN becomes -127;
        // non-finite blocks are cleared by the caller)
        return __float_as_uint(__fadd_rn(fminf(fmaxf(x, -127.0f), 127.0f), 12582912.0f)) & 0xFFu;
    else
        return e4m3_from_f32(x);
}

// Codes of 8 elements, first element in the lowest byte.
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], uint32_t b) {
    const float inv = scale_inv(b);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = code_of<FMT>(x[4 * h + i] * inv);
        w[h] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    }
    return b == 255u ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

template <int FMT>
__device__ __forceinline__ float value_of(uint32_t code, float scale) {
    if constexpr (FMT == kInt8) return (float)(int8_t)code * scale;
    else return e4m3_to_f32(code) * scale;
}

template <int FMT>
__device__ __forceinline__ void values8(uint2 w, float scale, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = value_of<FMT>(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu, scale);
}

// ------------------------------------------------------------- activation
// 1 / (1 + exp(-g)).  EXACT (fp32 results): the library's exp and division;
// otherwise the fast forms, whose relative error (below 2^-20 where the
// result is not tiny) disappears in the rounding to bf16.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float g) {
    if constexpr (EXACT) return 1.0f / (1.0f + expf(-g));
    else return __fdividef(1.0f, 1.0f + __expf(-g));
}
template <bool EXACT>
__device__ __forceinline__ float silu(float g) {
    if constexpr (EXACT) return g / (1.0f + expf(-g));
    else return __fdividef(g, 1.0f + __expf(-g));
}

// ------------------------------------------------------------------- work
// A flat index over (row, block of 32, part): parts are 4 quad lanes or 32
// lanes.  Every lane of a block is in or out together.
struct Place {
    int64_t row;
    uint32_t blk, col;
};
template <int V>
__device__ __forceinline__ bool place(uint64_t blocks, RowDiv nb, Place &p) {
    constexpr uint32_t kParts = 32 / V;
    const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    const uint64_t b = i / kParts;
    if (b >= blocks) return false;
    p.row = (int64_t)row_of(b, nb);
    p.blk = (uint32_t)(b - (uint64_t)p.row * nb.d);
    p.col = p.blk * 32 + (uint32_t)(i % kParts) * V;
    return true;
}
// Maximum over the lanes of a block.
template <int V>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
    if constexpr (V == 1) {
        return __reduce_max_sync(0xFFFFFFFFu, m);
    } else {
        const uint32_t quad = 0xFu << (threadIdx.x & 28u);
        m = max(m, __shfl_xor_sync(quad, m, 1));
        return max(m, __shfl_xor_sync(quad, m, 2));
    }
}

// Writes the checkpoint of a block: x[] are this lane's elements (zeros where
// it has none, `in` false).
template <int FMT, int V>
__device__ __forceinline__ void keep(const float (&x)[V], bool in, const Place &p, uint32_t nb, int64_t ld,
                                     const Ckpt &c) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, abs_bits(x[i]));
    const uint32_t b = scale_byte<FMT>(block_max<V>(m));
    if ((p.col & 31u) == 0) c.scales[p.row * nb + p.blk] = (uint8_t)b;
    if (!in) return;
    uint8_t *at = c.codes + p.row * ld + p.col;
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(at) = codes8<FMT>(x, b);
    else *at = b == 255u ? 0 : (uint8_t)code_of<FMT>(x[0] * scale_inv(b));
}
template <int FMT, int V>
__device__ __forceinline__ void restore(const Ckpt &c, const Place &p, uint32_t nb, int64_t ld, float (&x)[V]) {
    const float s = scale_of(__ldg(c.scales + p.row * nb + p.blk));
    const uint8_t *at = c.codes + p.row * ld + p.col;
    if constexpr (V == 8) values8<FMT>(__ldg(reinterpret_cast<const uint2 *>(at)), s, x);
    else x[0] = value_of<FMT>(__ldg(at), s);
}

// ---------------------------------------------------------------- kernels
template <class T, int FMT, int V>
__global__ void __launch_bounds__(kThreads) k_ckpt_save(const T *x, int64_t ld, Ckpt c, int64_t ldc, uint32_t cols,
                                                        RowDiv nb, uint64_t blocks) {
    Place p;
    if (!place<V>(blocks, nb, p)) return;
    const bool in = p.col < cols;
    float v[V] = {};
    if (in) load_f32<V>(x + p.row * ld + p.col, v);
    keep<FMT, V>(v, in, p, nb.d, ldc, c);
}

template <class T, int FMT, int V>
__global__ void __launch_bounds__(kThreads) k_ckpt_load(Ckpt c, int64_t ldc, T *x, int64_t ld, uint32_t cols,
                                                        RowDiv nb, uint64_t blocks) {
    Place p;
    if (!place<V>(blocks, nb, p) || p.col >= cols) return;
    float v[V];
    restore<FMT, V>(c, p, nb.d, ldc, v);
    store_f32<V>(x + p.row * ld + p.col, v);
}

template <class Ti, class To, int FMT, int V>
__global__ void __launch_bounds__(kThreads) k_swiglu(const Ti *gate, int64_t ld_gate, const Ti *up, int64_t ld_up,
                                                     To *h, int64_t ld_h, Ckpt cg, Ckpt cu, int64_t ldc,
                                                     uint32_t cols, RowDiv nb, uint64_t blocks) {
    constexpr bool kExact = std::is_same<To, float>::value;
    Place p;
    if (!place<V>(blocks, nb, p)) return;
    const bool in = p.col < cols;
    float g[V] = {}, u[V] = {};
    if (in) {
        load_f32<V>(gate + p.row * ld_gate + p.col, g);
        load_f32<V>(up + p.row * ld_up + p.col, u);
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = silu<kExact>(g[i]) * u[i];
        store_f32<V>(h + p.row * ld_h + p.col, o);
    }
    if constexpr (FMT != kNone) {
        keep<FMT, V>(g, in, p, nb.d, ldc, cg);
        keep<FMT, V>(u, in, p, nb.d, ldc, cu);
    }
}

template <class Td, class To, int FMT, int V>
__global__ void __launch_bounds__(kThreads) k_swiglu_bwd(const Td *dh, int64_t ld_dh, Ckpt cg, Ckpt cu, int64_t ldc,
                                                         To *dgate, int64_t ld_dgate, To *dup, int64_t ld_dup,
                                                         uint32_t cols, RowDiv nb, uint64_t blocks) {
    constexpr bool kExact = std::is_same<To, float>::value;
    Place p;
    if (!place<V>(blocks, nb, p) || p.col >= cols) return;
    float d[V], g[V], u[V];
    load_f32<V>(dh + p.row * ld_dh + p.col, d);
    restore<FMT, V>(cg, p, nb.d, ldc, g);
    restore<FMT, V>(cu, p, nb.d, ldc, u);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = sigmoid<kExact>(g[i]), gs = g[i] * s;
        u[i] = d[i] * u[i] * fmaf(gs, 1.0f - s, s);
        g[i] = d[i] * gs;
    }
    store_f32<V>(dgate + p.row * ld_dgate + p.col, u);
    store_f32<V>(dup + p.row * ld_dup + p.col, g);
}

// -------------------------------------------------------------- launching
struct Grid {
    RowDiv nb;
    uint64_t blocks;
    unsigned ctas;
};
Grid grid_of(int64_t rows, int64_t cols, bool v8) {
    const uint32_t nb = (uint32_t)((cols + 31) / 32);
    const uint64_t blocks = (uint64_t)rows * nb, lanes = blocks * (v8 ? 4 : 32);
    return Grid{make_rowdiv(nb), blocks, (unsigned)((lanes + kThreads - 1) / kThreads)};
}
template <int N>
using Int = std::integral_constant<int, N>;
template <class F>
void by_width(bool v8, F f) {
    if (v8) f(Int<8>());
    else f(Int<1>());
}
template <class F>
void by_format(int fmt, F f) {
    if (fmt == kInt8) f(Int<kInt8>());
    else f(Int<kE4M3>());
}
template <class P>
using Elem = std::remove_pointer_t<P>;
inline size_t size_of(int dtype) { return dtype == 0 ? 2 : 4; }

}  // namespace

cudaError_t launch_ckpt_save(const void *x, int dtype, int64_t ld, const Ckpt &c, int fmt, int64_t rows, int64_t cols,
                             cudaStream_t s) {
    const bool v8 = vec8(x, ld, cols, size_of(dtype));
    const Grid g = grid_of(rows, cols, v8);
    by_type(dtype, [&](auto *t) {
        using T = Elem<decltype(t)>;
        by_format(fmt, [&](auto f) {
            by_width(v8, [&](auto v) {
                k_ckpt_save<T, decltype(f)::value, decltype(v)::value><<<g.ctas, kThreads, 0, s>>>(
                    static_cast<const T *>(x), ld, c, ckpt_ld(cols), (uint32_t)cols, g.nb, g.blocks);
            });
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_ckpt_load(const Ckpt &c, int fmt, int64_t rows, int64_t cols, void *x, int dtype, int64_t ld,
                             cudaStream_t s) {
    const bool v8 = vec8(x, ld, cols, size_of(dtype));
    const Grid g = grid_of(rows, cols, v8);
    by_type(dtype, [&](auto *t) {
        using T = Elem<decltype(t)>;
        by_format(fmt, [&](auto f) {
            by_width(v8, [&](auto v) {
                k_ckpt_load<T, decltype(f)::value, decltype(v)::value><<<g.ctas, kThreads, 0, s>>>(
                    c, ckpt_ld(cols), static_cast<T *>(x), ld, (uint32_t)cols, g.nb, g.blocks);
            });
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_swiglu(const void *gate, int64_t ld_gate, const void *up, int64_t ld_up, int in_dtype,
                          int64_t rows, int64_t cols, void *h, int h_dtype, int64_t ld_h, const Ckpt &cg,
                          const Ckpt &cu, int fmt, cudaStream_t s) {
    const bool v8 = vec8(gate, ld_gate, cols, size_of(in_dtype)) && vec8(up, ld_up, cols, size_of(in_dtype)) &&
                    vec8(h, ld_h, cols, size_of(h_dtype));
    const Grid gr = grid_of(rows, cols, v8);
    by_type(in_dtype, [&](auto *ti) {
        using Ti = Elem<decltype(ti)>;
        by_type(h_dtype, [&](auto *to) {
            using To = Elem<decltype(to)>;
            by_width(v8, [&](auto v) {
                auto go = [&](auto f) {
                    k_swiglu<Ti, To, decltype(f)::value, decltype(v)::value><<<gr.ctas, kThreads, 0, s>>>(
                        static_cast<const Ti *>(gate), ld_gate, static_cast<const Ti *>(up), ld_up,
                        static_cast<To *>(h), ld_h, cg, cu, ckpt_ld(cols), (uint32_t)cols, gr.nb, gr.blocks);
                };
                if (fmt == kNone) go(Int<kNone>());
                else by_format(fmt, go);
            });
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const void *dh, int dh_dtype, int64_t ld_dh, const Ckpt &cg, const Ckpt &cu, int fmt,
                              int64_t rows, int64_t cols, void *dgate, int64_t ld_dgate, void *dup, int64_t ld_dup,
                              int out_dtype, cudaStream_t s) {
    const bool v8 = vec8(dh, ld_dh, cols, size_of(dh_dtype)) && vec8(dgate, ld_dgate, cols, size_of(out_dtype)) &&
                    vec8(dup, ld_dup, cols, size_of(out_dtype));
    const Grid g = grid_of(rows, cols, v8);
    by_type(dh_dtype, [&](auto *td) {
        using Td = Elem<decltype(td)>;
        by_type(out_dtype, [&](auto *to) {
            using To = Elem<decltype(to)>;
            by_format(fmt, [&](auto f) {
                by_width(v8, [&](auto v) {
                    k_swiglu_bwd<Td, To, decltype(f)::value, decltype(v)::value><<<g.ctas, kThreads, 0, s>>>(
                        static_cast<const Td *>(dh), ld_dh, cg, cu, ckpt_ld(cols), static_cast<To *>(dgate), ld_dgate,
                        static_cast<To *>(dup), ld_dup, (uint32_t)cols, g.nb, g.blocks);
                });
            });
        });
    });
    return cudaGetLastError();
}

}  // namespace ufp4
