// gemv.cu -- products of a few unquantized tokens with a quantized matrix:
// y[t][n] = S sum_k (v e)[n][k] x'[t][k], x' the token or its rotation; dense,
// and by expert for a routed batch.  (include/ufp4.h: ufp4_gemv,
// ufp4_gemv_grouped.)
//
// Bound by reading the weights (9 bits for 2 flops a token), so everything is
// laid out for loads of 16 bytes that go straight to registers and stay in
// flight, and the tensor cores do what arithmetic there is (mma.sync: with 8
// columns of which one is a token's, tcgen05's 128-row tiles would only add a
// trip through shared memory).
//
//  * The weights are the 16-row operand.  A lane reads 16 bytes (two scale
//    blocks) of a row; the inner index of the products is permuted so that
//    these are its operands of eight m16n8k16, and all of a lane's elements
//    of a row share two scales.  A chunk is 128 elements of a row, 4 lanes.
//  * A tile's rows are r, r + 32, r + 64, r + 96: 16 bytes of the scale layout
//    hold 4 blocks of exactly these rows, so scales too are read once, in
//    16-byte loads.
//  * A CTA's 8 warps share a tile's inner dimension (wk) and rows (8 / wk);
//    partial sums meet in shared memory, in a fixed order.
//  * The tokens are staged once per CTA in shared memory as FP16 operands, in
//    the order in which lanes read them.  Each chunk of a token has its own
//    power of two (its largest magnitude below 2^15), so BF16 tokens are exact
//    down to 2^-29 of the chunk's largest; rotated or FP32 tokens are the sum
//    of two FP16 values, within 2^-22 of each element.  The sum of a chunk's
//    products is scaled by that power and the weights' S when it is added to
//    the fp32 sum.
//  * Where the tokens do not fit, the inner dimension is gone through in
//    phases, the sums of a CTA's rows waiting in shared memory.
#include "common.cuh"
#include "dequant.cuh"
#include "internal.h"
#include "rowops.cuh"

#include <algorithm>

namespace ufp4 {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kChunk = 128;                    // elements of a row that 4 lanes hold
constexpr uint32_t kStageBudget = 64 * 1024;   // staged tokens: two CTAs on an SM
constexpr uint32_t kSumsBudget = 16 * 1024;    // sums that wait between phases

struct GemvArgs {
    const void *x;
    int64_t ld_x;
    int32_t x_fp32, x_wide;      // wide: 16-byte loads
    int32_t rht;
    uint64_t rht_seed;
    const uint8_t *codes, *scales;
    const float *tensor_scale;
    int32_t k, kpad;
    int32_t rows, atoms;         // of a matrix; 128-row atoms of it
    void *y;
    int64_t ld_y;
    int32_t y_fp32;
    int32_t tokens;              // dense: rows of x
    // by expert: first place of each (n_experts + 1), slots and their tokens
    const int64_t *offsets;
    const int32_t *src;
    int32_t n_experts, slots, topk, gather;
    int32_t wk, chunks, phase;   // warps along k; chunks of a row, and of a phase
    int32_t cpad;                // columns of a pass (power of two below 8, else 8 i)
    int32_t units;               // steps (wr tiles) of a matrix
    int32_t sums;                // steps a CTA may hold sums of (0: one phase)
};

template <int MT>
struct Frag {
    uint4 c[2 * MT];
    uint32_t s[2 * MT];
};

// Weights are read once: they do not displace the tokens in L1.
__device__ __forceinline__ uint4 load_stream(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A step's columns: tokens [first, first + n) of its matrix, n <= 8 NT.
struct Cols {
    int32_t first, n, pad;       // pad: staged columns (power of two below 8, else 8 i)
};
__host__ __device__ __forceinline__ int pad_cols(int n) { return n >= 8 ? (n + 7) & ~7 : n > 4 ? 8 : n > 2 ? 4 : n; }

template <int GRID, int MT, int NT, int PL>
__global__ void __launch_bounds__(kThreads, 2) k_gemv(GemvArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int32_t seg_unit[kMaxGroups + 1];     // by expert: steps before each
    __shared__ int32_t warp_sum[kWarps];
    const uint32_t zero = begin_in_order();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wk = a.wk, wr = kWarps / wk, my_k = warp % wk, my_r = warp / wk;
    constexpr int kCols = 8 * NT, kRows = 16 * MT, kPitch = kRows + 4;

    uint4 *xs = reinterpret_cast<uint4 *>(smem);                            // [PL][phase][4][cpad][4] x 16 bytes
    const uint32_t plane = (uint32_t)a.phase * 16u * a.cpad;                // 16-byte units
    float *fac = reinterpret_cast<float *>(smem + (size_t)PL * plane * 16); // [phase][kCols]
    float *red = fac + a.phase * kCols;                                     // [2][kWarps][kCols][kPitch]
    float *sums = red + 2 * kWarps * kCols * kPitch;                        // [sums][wr][kCols][kRows]

    const int nseg = a.offsets ? a.n_experts : 1;
    int total;
    if (a.offsets) {
        // steps of each expert: passes over its tokens times steps of a matrix
        int carry = 0;
        for (int base = 0; base < nseg; base += kThreads) {
            const int e = base + tid;
            int v = 0;
            if (e < nseg) {
                const int64_t n = a.offsets[zero + e + 1] - a.offsets[zero + e];
                v = (int)((n + a.cpad - 1) / a.cpad) * a.units;
            }
            int incl = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            if (lane == 31) warp_sum[warp] = incl;
            __syncthreads();
            int before = carry, all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += warp_sum[w];
                all += warp_sum[w];
            }
            if (e < nseg) seg_unit[e] = before + incl - v;
            carry += all;
            __syncthreads();
        }
        if (tid == 0) seg_unit[nseg] = carry;
        __syncthreads();
        total = carry;
        // rows of dropped slots: zeros
        const int64_t routed = a.offsets[zero + nseg];
        const int64_t rest = (a.slots - routed) * (int64_t)a.rows;
        for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < rest; i += (int64_t)gridDim.x * kThreads) {
            const int64_t at = (routed + i / a.rows) * a.ld_y + i % a.rows;
            if (a.y_fp32) static_cast<float *>(a.y)[at] = 0.0f;
            else static_cast<uint16_t *>(a.y)[at] = 0;
        }
    } else {
        total = (a.tokens + a.cpad - 1) / a.cpad * a.units;
    }
    const int begin = (int)((int64_t)total * blockIdx.x / gridDim.x);
    const int end = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
    if (begin >= end) return;
    const uint32_t signs = a.rht ? rht_sign_mask(a.rht_seed) : 0u;
    const int nkt = a.kpad >> 6;
    const int64_t row_bytes = a.kpad >> 1;

    int seg = 0;
    if (a.offsets) {
        int lo = 0, hi = nseg;          // the last expert that begins at or before `begin`
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seg_unit[mid] <= begin) lo = mid;
            else hi = mid;
        }
        seg = lo;
    }
    int parity = 0;
    for (int u0 = begin; u0 < end;) {
        int pass;
        int64_t first_place;             // of the segment
        int seg_tokens, in_seg;
        if (a.offsets) {
            while (seg_unit[seg + 1] <= u0) ++seg;
            in_seg = u0 - seg_unit[seg];
            first_place = a.offsets[zero + seg];
            seg_tokens = (int)(a.offsets[zero + seg + 1] - first_place);
        } else {
            in_seg = u0;
            first_place = 0;
            seg_tokens = a.tokens;
        }
        pass = in_seg / a.units;
        const int step0 = in_seg - pass * a.units;
        const int steps = min(end - u0, a.units - step0);
        Cols cols;
        cols.first = pass * a.cpad;
        cols.n = min(seg_tokens - cols.first, a.cpad);
        cols.pad = pad_cols(cols.n);
        const float ts = a.tensor_scale[zero + seg] * kDecoded<GRID>;
        const int64_t atom0 = (int64_t)seg * a.atoms;

        for (int p0 = 0; p0 < a.chunks; p0 += a.phase) {
            const int pch = min(a.phase, a.chunks - p0);
            const int per = (pch + wk - 1) / wk;             // chunks of a warp
            const int items = steps * per;
            Frag<MT> f[2];
            auto load = [&](Frag<MT> &d, int it) {
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    d.c[i] = make_uint4(0, 0, 0, 0);
                    d.s[i] = 0;
                }
                if (it >= items) return;
                const int st = it / per, c = it - st * per;
                const int in_phase = c * wk + my_k, chunk = p0 + in_phase;
                if (in_phase >= pch || chunk * 2 + (t >> 1) >= nkt) return;
                const int sub = (step0 + st) * wr + my_r;
                const int atom = sub / (8 / MT), w8 = (sub & 3) * 8 + g, i0 = MT == 1 ? (sub >> 2 & 1) * 2 : 0;
                if (atom >= a.atoms) return;
                const uint8_t *cp = a.codes + ((atom0 + atom) * 128 + w8 + i0 * 32) * row_bytes + chunk * 64 + t * 16;
                const int row = atom * 128 + w8 + i0 * 32;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i)
                    if (row + 32 * i < a.rows) d.c[i] = load_stream(cp + (int64_t)(32 * i) * row_bytes);
                const uint8_t *sp = a.scales + (((atom0 + atom) * nkt + chunk * 2 + (t >> 1)) << 9) + w8 * 16;
                if constexpr (MT == 2) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(sp);
                    d.s[0] = v.x; d.s[1] = v.y; d.s[2] = v.z; d.s[3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(sp + i0 * 4);
                    d.s[0] = v.x; d.s[1] = v.y;
                }
            };
            load(f[0], 0);
            load(f[1], 1);

            // ---- the tokens' part of this phase
            __syncthreads();
            for (int i = tid; i < cols.n * pch * 8; i += kThreads) {
                const int b = i & 7, rest = i >> 3, col = rest / pch, ch = rest - col * pch;
                const int k0 = (p0 + ch) * kChunk + b * 16;
                float v[16];
                if (k0 < a.k) {
                    int64_t row = first_place + cols.first + col;
                    if (a.gather) row = a.src[row] / a.topk;
                    const int64_t at = row * a.ld_x + k0;
                    if (a.x_fp32) {
                        const float *p = static_cast<const float *>(a.x) + at;
                        if (a.x_wide) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float4 w = reinterpret_cast<const float4 *>(p)[q];
                                v[4 * q] = w.x; v[4 * q + 1] = w.y; v[4 * q + 2] = w.z; v[4 * q + 3] = w.w;
                            }
                        } else {
#pragma unroll
                            for (int q = 0; q < 16; ++q) v[q] = p[q];
                        }
                    } else {
                        const uint16_t *p = static_cast<const uint16_t *>(a.x) + at;
                        if (a.x_wide) {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint4 w = reinterpret_cast<const uint4 *>(p)[q];
                                v[8 * q] = bf16lo(w.x); v[8 * q + 1] = bf16hi(w.x);
                                v[8 * q + 2] = bf16lo(w.y); v[8 * q + 3] = bf16hi(w.y);
                                v[8 * q + 4] = bf16lo(w.z); v[8 * q + 5] = bf16hi(w.z);
                                v[8 * q + 6] = bf16lo(w.w); v[8 * q + 7] = bf16hi(w.w);
                            }
                        } else {
#pragma unroll
                            for (int q = 0; q < 16; ++q) v[q] = __uint_as_float((uint32_t)p[q] << 16);
                        }
                    }
                    if (a.rht) rotate16(v, signs);
                } else {
#pragma unroll
                    for (int q = 0; q < 16; ++q) v[q] = 0.0f;
                }
                uint32_t top = 0;
#pragma unroll
                for (int q = 0; q < 16; ++q) top = max(top, finite_bits(v[q]));
                const uint32_t group = 0xffu << (lane & 24);     // the chunk's 8 lanes
                top = max(top, __shfl_xor_sync(group, top, 1));
                top = max(top, __shfl_xor_sync(group, top, 2));
                top = max(top, __shfl_xor_sync(group, top, 4));
                const int e = top_exponent(top);
                const float m = exp2i(14 - e);
                if (b == 0) fac[ch * kCols + col] = exp2i(e - 14) * ts;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float p = v[8 * h + code_order<GRID>(2 * q)] * m;
                        const float r = v[8 * h + code_order<GRID>(2 * q + 1)] * m;
                        hi[q] = f16_pair(p, r);
                        if constexpr (PL == 2) lo[q] = f16_rest(p, r, hi[q]);
                    }
                    const uint32_t to = ((uint32_t)(ch * 4 + (b & 1) * 2 + h) * cols.pad + col) * 4 + (b >> 1);
                    xs[to] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (PL == 2) xs[plane + to] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            __syncthreads();

            // ---- the weights
            float sum[MT][NT][4] = {};
            const int bcol = cols.pad < 8 ? g & (cols.pad - 1) : g;
            int st = 0, c = 0;
            auto use = [&](const Frag<MT> &d) {
                const int ch = c * wk + my_k;
                if (ch < pch) {
                    float acc[MT][NT][4] = {};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t sel = ((t & 1) * 2 + (u >> 1)) * 0x11u;
                        uint32_t h[2 * MT][4];
#pragma unroll
                        for (int i = 0; i < 2 * MT; ++i) {
                            const uint32_t s = scale_pair(d.s[i], sel);
                            decode8<GRID>(u == 0 ? d.c[i].x : u == 1 ? d.c[i].y : u == 2 ? d.c[i].z : d.c[i].w, h[i]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) h[i][q] = mul_pair(h[i][q], s);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n > 0 && n * 8 >= cols.pad) break;
                            const uint32_t at = ((uint32_t)(ch * 4 + u) * cols.pad + n * 8 + bcol) * 4 + t;
#pragma unroll
                            for (int p = 0; p < PL; ++p) {
                                const uint4 b = xs[p * plane + at];
#pragma unroll
                                for (int m = 0; m < MT; ++m) {
                                    const uint32_t(&r)[4] = h[2 * m];
                                    const uint32_t(&s)[4] = h[2 * m + 1];
                                    mma_f16(acc[m][n], r[0], s[0], r[1], s[1], b.x, b.y);
                                    mma_f16(acc[m][n], r[2], s[2], r[3], s[3], b.z, b.w);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 w = *reinterpret_cast<const float2 *>(fac + ch * kCols + n * 8 + 2 * t);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            sum[m][n][0] += acc[m][n][0] * w.x;
                            sum[m][n][1] += acc[m][n][1] * w.y;
                            sum[m][n][2] += acc[m][n][2] * w.x;
                            sum[m][n][3] += acc[m][n][3] * w.y;
                        }
                    }
                }
                if (++c < per) return;
                // ---- the end of a step: the warps' sums together
                float *mine = red + (size_t)(parity * kWarps + warp) * kCols * kPitch;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int col = n * 8 + 2 * t + (j & 1);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            if (col < cols.n) mine[col * kPitch + m * 16 + g + (j >> 1) * 8] = sum[m][n][j];
                            sum[m][n][j] = 0.0f;
                        }
                    }
                __syncthreads();
                for (int i = tid; i < wr * cols.n * kRows; i += kThreads) {
                    const int r = i % kRows, rest = i / kRows, col = rest % cols.n, part = rest / cols.n;
                    const float *from = red + (size_t)(parity * kWarps + part * wk) * kCols * kPitch + col * kPitch + r;
                    float v = from[0];
                    for (int w = 1; w < wk; ++w) v += from[(size_t)w * kCols * kPitch];
                    if (a.sums) {
                        float *kept = sums + ((size_t)(st * wr + part) * kCols + col) * kRows + r;
                        if (p0 > 0) v += *kept;
                        if (p0 + a.phase < a.chunks) {
                            *kept = v;
                            continue;
                        }
                    }
                    const int sub = (step0 + st) * wr + part;
                    const int atom = sub / (8 / MT), i0 = MT == 1 ? (sub >> 2 & 1) * 2 : 0;
                    // of a tile's rows, r / 8 is which 32 of the atom
                    const int row = atom * 128 + (i0 + r / 8) * 32 + (sub & 3) * 8 + (r & 7);
                    if (row >= a.rows) continue;
                    const int64_t at = (first_place + cols.first + col) * a.ld_y + row;
                    if (a.y_fp32) static_cast<float *>(a.y)[at] = v;
                    else static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
                }
                parity ^= 1;
                c = 0;
                ++st;
            };
            for (int it = 0; it < items; it += 2) {
                use(f[0]);
                load(f[0], it + 2);
                if (it + 1 < items) {
                    use(f[1]);
                    load(f[1], it + 3);
                }
            }
        }
        u0 += steps;
    }
}

template <int GRID, int MT, int NT, int PL>
cudaError_t launch(GemvArgs a, int most_cols, cudaStream_t s) {
    constexpr int kCols = 8 * NT, kRows = 16 * MT, kPitch = kRows + 4;
    const int wr = kWarps / a.wk;
    const int64_t steps = ((int64_t)a.atoms * (8 / MT) + wr - 1) / wr;
    a.units = (int)steps;
    a.cpad = pad_cols(std::min(most_cols, kCols));
    const uint32_t per_chunk = 256u * a.cpad * PL;
    a.phase = std::max<int>(1, std::min<int>(a.chunks, kStageBudget / per_chunk));
    if (a.phase < a.chunks && a.phase > a.wk) a.phase = a.phase / a.wk * a.wk;
    // upper bound on the steps of all passes (the device knows the counts)
    int64_t passes;
    if (a.offsets) passes = std::min<int64_t>(a.slots, (int64_t)a.n_experts + a.slots / a.cpad);
    else passes = (a.tokens + a.cpad - 1) / a.cpad;
    const int64_t total = passes * steps;
    if (total > 0x7fffffff) return cudaErrorNotSupported;
    int64_t grid = std::min<int64_t>(total, 2 * (int64_t)num_sms());
    size_t sum_bytes = 0;
    a.sums = 0;
    if (a.phase < a.chunks) {
        const size_t one = (size_t)wr * kCols * kRows * sizeof(float);
        const int64_t fits = std::max<int64_t>(1, kSumsBudget / one);
        grid = std::max(grid, (total + fits - 1) / fits);
        a.sums = (int)((total + grid - 1) / grid);
        sum_bytes = a.sums * one;
    }
    const size_t bytes = (size_t)a.phase * per_chunk + (size_t)a.phase * kCols * 4 +
                         2 * (size_t)kWarps * kCols * kPitch * 4 + sum_bytes;
    cudaError_t e = cudaFuncSetAttribute(k_gemv<GRID, MT, NT, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)bytes);
    if (e != cudaSuccess) return e;
    return launch_in_order_smem(k_gemv<GRID, MT, NT, PL>, dim3((unsigned)grid), kThreads, bytes, s, a);
}

cudaError_t dispatch(const GemvArgs &a, int grid, int most_cols, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    auto with = [&](auto gr, auto mt, auto nt) {
        constexpr int G = decltype(gr)::value, M = decltype(mt)::value, N = decltype(nt)::value;
        if (a.rht || a.x_fp32) e = launch<G, M, N, 2>(a, most_cols, s);
        else e = launch<G, M, N, 1>(a, most_cols, s);
    };
    auto by_cols = [&](auto gr) {
        if (most_cols <= 8) with(gr, Int<2>(), Int<1>());
        else if (most_cols <= 16 || a.offsets) with(gr, Int<2>(), Int<2>());
        else with(gr, Int<1>(), Int<4>());
    };
    if (grid == kE1M2) by_cols(Int<kE1M2>());
    else by_cols(Int<kE2M1>());      // (the clamped grid's codes are E2M1 codes)
    return e;
}

}  // namespace

cudaError_t launch_gemv(const GemvLaunch &l, cudaStream_t s) {
    GemvArgs a{};
    a.x = l.x;
    a.ld_x = l.ld_x;
    a.x_fp32 = l.x_dtype == 1;
    a.x_wide = rows_by(l.x, l.ld_x, type_size(l.x_dtype), a.x_fp32 ? 4 : 8);
    a.rht = l.rht;
    a.rht_seed = l.rht_seed;
    a.codes = l.codes;
    a.scales = l.scales;
    a.tensor_scale = l.tensor_scale;
    a.k = (int)l.k;
    a.kpad = (int)kpad_of(l.k);
    a.rows = (int)l.rows;
    a.atoms = (int)((l.rows + 127) / 128);
    a.y = l.y;
    a.ld_y = l.ld_y;
    a.y_fp32 = l.y_dtype == 1;
    a.tokens = (int)l.tokens;
    a.offsets = l.offsets;
    a.src = l.src;
    a.n_experts = l.n_experts;
    a.slots = (int)l.slots;
    a.topk = l.topk;
    a.gather = l.gather;
    a.chunks = (a.kpad + kChunk - 1) / kChunk;
    // Warps along k: as many as leave at most a quarter of their chunks empty.
    a.wk = 8;
    while (a.wk > 1 && a.chunks * 4 < (a.chunks + a.wk - 1) / a.wk * a.wk * 3) a.wk /= 2;
    // By expert, columns for what one mostly has: a token each.  (One that a
    // token names twice may have more, in further passes.)
    return dispatch(a, l.grid, (int)(l.offsets ? std::min(l.slots, l.tokens) : l.tokens), s);
}

}  // namespace ufp4
