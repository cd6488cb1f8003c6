// gemv.cu -- products of a few unquantized tokens with a quantized matrix:
// y[t][n] = S sum_k (v e)[n][k] x'[t][k], x' the token or its rotation; dense,
// and by expert for a routed batch.  (include/ufp4.h: ufp4_gemv,
// ufp4_gemv_grouped.)
//
// Bound by reading the weights (9 bits for 2 flops a token), and next by
// decoding them: 42 weights arrive per SM and clock at the measured copy
// bandwidth.  So the loads are 16 bytes a lane and stay in flight, and the tensor
// cores do what arithmetic there is (mma.sync: with 8 columns of which one is a
// token's, tcgen05's 128-row tiles would only add a trip through shared memory).
//
//  * The weights are the 16-row operand.  A lane takes 16 bytes (two scale
//    blocks) of a row; the inner index of the products is permuted so that
//    these are its operands of eight m16n8k16, and all of a lane's elements
//    of a row share two scales.  A chunk is 128 elements of a row, 4 lanes.
//  * A tile's rows are r, r + 32, r + 64, r + 96: 16 bytes of the scale layout
//    hold 4 blocks of exactly these rows, so scales too are read once, in
//    16-byte pieces.
//  * Chunks come by cp.async, two ahead, into places of the lane's own: no
//    barrier, and 40 registers less than loads held in registers.
//  * A CTA's 8 warps share a tile's inner dimension (wk) and rows (8 / wk);
//    partial sums meet in shared memory, in a fixed order.
//  * The tokens are staged once per CTA in shared memory as FP16 operands, in
//    the order in which lanes read them.  Each chunk of a token has its own
//    power of two (its largest magnitude below 2^15), so BF16 tokens are exact
//    down to 2^-29 of the chunk's largest (less where its products come near
//    fp32's lower end).  Rotated or FP32 tokens are, for an
//    FP32 result, the sum of two FP16 values, within 2^-22 of each element; for
//    a BF16 result (8 bits) one FP16 value (11 bits).  The sum of a chunk's
//    products is scaled by that power and the weights' S when it is added to
//    the fp32 sum.
//  * Where the tokens do not fit, the inner dimension is gone through in
//    phases, the sums of a CTA's rows waiting in shared memory.
//
// Measured (graph replay, inputs past L2): 131072 x 8192 E2M1, one token, 123 us
// (4.9 TB/s, 72 % of the copy bandwidth; 114 us with the decoding and the products
// left out, so what is left is the loads: their start, the steps' joins and the
// last, uneven round).  Other splits of the same: warps along k 8 / 4 / 2: 126 /
// 122 / 138 us; tiles of 16 rows 149; one CTA of 16 warps an SM 128; three chunks
// ahead 121; consecutive steps a CTA instead of every gridDim.x-th 125 (all of
// these beside 121).  2048 x 2048, one token, 4.8 us; 64 tokens x 6 of 64 experts
// of 2048 x 1408 59 us.
#include "common.cuh"
#include "dequant.cuh"
#include "internal.h"
#include "rowops.cuh"

#include <algorithm>

namespace ufp4 {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kChunk = 128;                    // elements of a row that 4 lanes hold
constexpr int kAhead = 2;                      // chunks of a warp under way
constexpr uint32_t kSharedBudget = 110 * 1024; // two CTAs on an SM, with 1 KB each that is not dynamic, and the system's
constexpr uint32_t kSumsBudget = 16 * 1024;    // sums that wait between phases

struct GemvArgs {
    const void *x;
    int64_t ld_x;
    int32_t x_fp32, x_wide;      // wide: 16-byte loads
    int32_t rht;
    uint32_t signs;              // of the rotation
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
    int32_t factors;             // floats for the chunks' factors
    int32_t red_two;             // whether the sums to be joined alternate between two places
    int32_t ring;                // where the chunks in flight lie in shared memory
    int32_t cpad;                // columns of a pass (power of two below 8, else 8 i)
    int32_t units;               // steps (wr tiles) of a matrix
    int32_t sums;                // steps a CTA may hold sums of (0: one phase)
};

template <int MT>
struct Frag {
    uint4 c[2 * MT];
    uint32_t s[2 * MT];
};

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
    float *fac = reinterpret_cast<float *>(smem + (size_t)PL * plane * 16); // [chunks of a phase][columns, 8 at least]
    float *red = fac + a.factors;                                           // [1 or 2][kWarps][cpad][kPitch]
    const int red_warp = a.cpad * kPitch;
    float *sums = red + (a.red_two ? 2 : 1) * kWarps * red_warp;            // [sums][wr][kCols][kRows]
    // the lane's own pieces of its warp's chunks in flight
    constexpr int kSlot = (2 * MT + 1) * 512;
    uint8_t *const ring = smem + a.ring + warp * kAhead * kSlot + lane * 16;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);

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
        total = (a.tokens + a.cpad - 1) / a.cpad;        // passes
    }
    // By expert a CTA has consecutive steps, of few experts; else, of every
    // pass, every gridDim.x-th: neighbouring rows are read at the same time
    // (131072 x 8192: 7 us less).
    const int begin = a.offsets ? (int)((int64_t)total * blockIdx.x / gridDim.x) : 0;
    const int end = a.offsets ? (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x) : total;
    if (begin >= end) return;
    const int nkt = a.kpad >> 6;
    const int64_t row_bytes = a.kpad >> 1, row_step = 32 * row_bytes;

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
        int pass, step0, stride, steps;
        int64_t first_place;             // of the segment
        int seg_tokens;
        if (a.offsets) {
            while (seg_unit[seg + 1] <= u0) ++seg;
            first_place = a.offsets[zero + seg];
            seg_tokens = (int)(a.offsets[zero + seg + 1] - first_place);
            pass = (u0 - seg_unit[seg]) / a.units;
            step0 = u0 - seg_unit[seg] - pass * a.units;
            stride = 1;
            steps = min(end - u0, a.units - step0);
            u0 += steps;
        } else {
            first_place = 0;
            seg_tokens = a.tokens;
            pass = u0++;
            step0 = blockIdx.x;
            stride = gridDim.x;
            steps = (a.units - step0 + stride - 1) / stride;
        }
        Cols cols;
        cols.first = pass * a.cpad;
        cols.n = min(seg_tokens - cols.first, a.cpad);
        cols.pad = pad_cols(cols.n);
        const float ts = a.tensor_scale[zero + seg] * kDecoded<GRID>;
        const int64_t atom0 = (int64_t)seg * a.atoms;

        // chunks that fit beside this many columns, evenly over the phases
        int phase = min(a.chunks, a.phase * a.cpad / cols.pad);
        if (phase < a.chunks) {
            const int n = (a.chunks + phase - 1) / phase, even = ((a.chunks + n - 1) / n + wk - 1) / wk * wk;
            phase = min(phase, even);
        }
        const int fpitch = max(cols.pad, 8);
        for (int p0 = 0; p0 < a.chunks; p0 += phase) {
            const int pch = min(phase, a.chunks - p0);
            const int per = (pch + wk - 1) / wk;             // chunks of a warp
            const int items = steps * per;
            // Where the next chunk to load lies: of the lane's rows of a step
            // (row_count of 2 MT), chunk my_k + wk lc of the phase.
            const int lane_chunks = (nkt + 1 - (t >> 1)) / 2 - p0;          // (a row may end with half a chunk)
            const int lane_count = (min(pch, lane_chunks) - my_k + wk - 1) / wk;
            int lc = 0, lst = 0;
            bool whole = true;                       // all rows of the step exist
            int row_count = 2 * MT;
            const uint8_t *cp = nullptr, *sp = nullptr;
            const auto enter = [&] {
                const int sub = (step0 + lst * stride) * wr + my_r;
                const int atom = sub / (8 / MT), w8 = (sub & 3) * 8 + g, i0 = MT == 1 ? (sub >> 2 & 1) * 2 : 0;
                const int row = atom * 128 + w8 + i0 * 32;
                whole = (atom + 1) * 128 <= a.rows;
                row_count = atom < a.atoms ? (a.rows - row + 31) >> 5 : 0;
                cp = a.codes + (atom0 * 128 + row) * row_bytes + (p0 + my_k) * 64 + t * 16;
                sp = a.scales + (((atom0 + atom) * nkt + (p0 + my_k) * 2 + (t >> 1)) << 9) + w8 * 16;
            };
            enter();
            // (a chunk that is past the phase, for the whole warp, is not used)
            const int warp_count = (pch - my_k + wk - 1) / wk;
            const auto copy = [&](int slot) {
                if (lst < steps && lc < warp_count) {
                    const uint32_t to = ring_s + slot * kSlot;
                    const bool real = lc < lane_count;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 2 * MT; ++i) copy16(to + i * 512, cp + i * row_step, real);
                        copy16(to + 2 * MT * 512, sp, real);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2 * MT; ++i) copy16(to + i * 512, cp + i * row_step, real && i < row_count);
                        copy16(to + 2 * MT * 512, sp, real && row_count > 0);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                cp += wk * 64;
                sp += wk * 1024;
                if (++lc == per) {
                    lc = 0;
                    if (++lst < steps) enter();
                }
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) copy(i);

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
                    if (a.rht) rotate16(v, a.signs);
                } else {
#pragma unroll
                    for (int q = 0; q < 16; ++q) v[q] = 0.0f;
                }
                uint32_t top = top_bits(v);
                const uint32_t group = 0xffu << (lane & 24);     // the chunk's 8 lanes
                top = max(top, __shfl_xor_sync(group, top, 1));
                top = max(top, __shfl_xor_sync(group, top, 2));
                top = max(top, __shfl_xor_sync(group, top, 4));
                // (small tokens by small weights: up to 2^16 less for the tokens'
                // FP16 values, of which the largest keep their bits, rather
                // than bits of the factor, which all products share)
                int e = top_exponent(top);
                if (e < -32) {
                    asm volatile("");            // (a branch: other tokens do not wait for the scale)
                    e = max(e, min(e + 16, -112 - ((int)(__float_as_uint(ts) >> 23 & 0xFFu) - 127)));
                }
                const float m = exp2i(14 - e);
                if (b == 0) fac[ch * fpitch + col] = exp2i(e - 14) * ts;
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
            const int x_word = cols.pad * 4;                 // 16-byte units from one word of the lanes to the next
            const uint4 *const x_first = xs + my_k * 4 * x_word + (cols.pad < 8 ? g & (cols.pad - 1) : g) * 4 + t;
            const uint4 *xp = x_first;
            int st = 0, c = 0;
            const auto use = [&](int slot) {
                const int ch = c * wk + my_k;
                if (ch < pch) {
                    Frag<MT> d;
                    const uint8_t *from = ring + slot * kSlot;
#pragma unroll
                    for (int i = 0; i < 2 * MT; ++i) d.c[i] = *reinterpret_cast<const uint4 *>(from + i * 512);
                    const uint4 v = *reinterpret_cast<const uint4 *>(from + 2 * MT * 512);
                    if constexpr (MT == 2) {
                        d.s[0] = v.x; d.s[1] = v.y; d.s[2] = v.z; d.s[3] = v.w;
                    } else {
                        const bool upper = ((step0 + st * stride) * wr + my_r) & 4;      // which 64 rows of the atom
                        d.s[0] = upper ? v.z : v.x;
                        d.s[1] = upper ? v.w : v.y;
                    }
                    float acc[PL][MT][NT][4] = {};
                    uint32_t scale[2 * MT];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t h[2 * MT][4];
#pragma unroll
                        for (int i = 0; i < 2 * MT; ++i) {
                            if (u % 2 == 0) scale[i] = scale_pair(d.s[i], ((t & 1) * 2 + u / 2) * 0x11u);
                            const uint32_t s = scale[i];
                            decode8<GRID>(u == 0 ? d.c[i].x : u == 1 ? d.c[i].y : u == 2 ? d.c[i].z : d.c[i].w, h[i]);
#pragma unroll
                            for (int q = 0; q < 4; ++q) h[i][q] = mul_pair(h[i][q], s);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n > 0 && n * 8 >= cols.pad) break;
#pragma unroll
                            for (int p = 0; p < PL; ++p) {
                                const uint4 b = xp[p * plane + u * x_word + n * 32];
#pragma unroll
                                for (int m = 0; m < MT; ++m) {
                                    const uint32_t(&r)[4] = h[2 * m];
                                    const uint32_t(&s)[4] = h[2 * m + 1];
                                    mma_f16(acc[p][m][n], r[0], s[0], r[1], s[1], b.x, b.y);
                                    mma_f16(acc[p][m][n], r[2], s[2], r[3], s[3], b.z, b.w);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 w = *reinterpret_cast<const float2 *>(fac + ch * fpitch + n * 8 + 2 * t);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float v = acc[0][m][n][j];
                                if constexpr (PL == 2) v += acc[1][m][n][j];
                                sum[m][n][j] += v * (j & 1 ? w.y : w.x);
                            }
                    }
                }
                xp += wk * 4 * x_word;
                if (++c < per) return;
                // ---- the end of a step: the warps' sums together
                float *mine = red + (parity * kWarps + warp) * red_warp;
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
                // a warp takes a column (two of 16 rows) of one of the step's tiles
                constexpr int kPer = 32 / kRows;
                const int r = lane % kRows;
                for (int i = warp * kPer + lane / kRows, part = 0; part < wr; i += kWarps * kPer) {
                    for (; i >= cols.n && part < wr; i -= cols.n) ++part;
                    if (part >= wr) break;
                    const int col = i;
                    const float *from = red + (parity * kWarps + part * wk) * red_warp + col * kPitch + r;
                    float v = from[0];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w)
                        if (w < wk) v += from[w * red_warp];
                    if (a.sums) {
                        float *kept = sums + ((size_t)(st * wr + part) * kCols + col) * kRows + r;
                        if (p0 > 0) v += *kept;
                        if (p0 + phase < a.chunks) {
                            *kept = v;
                            continue;
                        }
                    }
                    const int sub = (step0 + st * stride) * wr + part;
                    const int atom = sub / (8 / MT), i0 = MT == 1 ? (sub >> 2 & 1) * 2 : 0;
                    // of a tile's rows, r / 8 is which 32 of the atom
                    const int row = atom * 128 + (i0 + r / 8) * 32 + (sub & 3) * 8 + (r & 7);
                    if (row >= a.rows) continue;
                    const int64_t at = (first_place + cols.first + col) * a.ld_y + row;
                    if (a.y_fp32) static_cast<float *>(a.y)[at] = v;
                    else static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v);
                }
                if (a.red_two) parity ^= 1;
                else __syncthreads();
                c = 0;
                xp = x_first;
                ++st;
            };
            for (int it = 0; it < items; it += kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (it + i >= items) break;
                    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                    use(i);
                    copy(i);
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");     // (the next phase's copies go to the same places)
        }
    }
}

template <int GRID, int MT, int NT, int PL>
cudaError_t launch(GemvArgs a, int most_cols, cudaStream_t s) {
    constexpr int kCols = 8 * NT, kRows = 16 * MT, kPitch = kRows + 4;
    a.cpad = pad_cols(std::min(most_cols, kCols));
    a.red_two = a.cpad <= 8;
    const uint32_t per_chunk = 256u * a.cpad * PL;
    const size_t red_bytes = (size_t)(a.red_two ? 2 : 1) * kWarps * a.cpad * kPitch * 4, slot = (2 * MT + 1) * 512;
    // What the chunks in flight leave holds the tokens and their factors: all
    // of them, or as many as go beside the sums that then wait.
    const auto room = [&](size_t others) {
        const int64_t left = (int64_t)kSharedBudget - (int64_t)(kWarps * kAhead * slot + red_bytes + others + 512);
        return (int)std::max<int64_t>(1, left / (per_chunk + 36 * a.cpad));
    };
    a.phase = room(0) >= a.chunks ? a.chunks : room(kSumsBudget);
    // upper bound on the steps of all passes (the device knows the counts)
    int64_t passes;
    if (a.offsets) passes = std::min<int64_t>(a.slots, (int64_t)a.n_experts + a.slots / a.cpad);
    else passes = (a.tokens + a.cpad - 1) / a.cpad;
    const int64_t ctas = 2 * (int64_t)num_sms(), tiles = (int64_t)a.atoms * (8 / MT);
    if (passes * tiles > 0x7fffffff) return cudaErrorNotSupported;
    // Warps along k: what makes the CTAs' steps times the chunks of a warp,
    // and the joining of the sums (about 3/4 of a chunk's time), the least.
    // (Of whole rows: that some warps wait where a phase has fewer chunks than
    // wk, or no multiple of it, is not priced.)
    const int64_t likely = a.offsets ? std::min<int64_t>(a.slots, a.n_experts) : passes;
    int64_t least = INT64_MAX;
    for (int wk = kWarps; wk >= 1; wk /= 2) {
        const int64_t steps = likely * ((tiles * wk + kWarps - 1) / kWarps);
        const int64_t cost = (steps + ctas - 1) / ctas * (4 * ((a.chunks + wk - 1) / wk) + 3);
        if (cost < least) {
            least = cost;
            a.wk = wk;
        }
    }
    const int wr = kWarps / a.wk;
    const int64_t steps = (tiles + wr - 1) / wr;
    const int64_t total = a.offsets ? passes * steps : steps;        // (a pass takes every CTA)
    a.units = (int)steps;
    int64_t grid = std::min<int64_t>(total, ctas);
    size_t sum_bytes = 0;
    a.sums = 0;
    if (a.phase < a.chunks) {
        const size_t one = (size_t)wr * kCols * kRows * sizeof(float);
        const int64_t fits = std::max<int64_t>(1, kSumsBudget / one);
        grid = std::max(grid, (total + fits - 1) / fits);
        a.sums = (int)((total + grid - 1) / grid);
        sum_bytes = a.sums * one;
    }
    // (a pass over fewer columns has as many more chunks in a phase)
    a.factors = 8 * std::min(a.chunks, a.phase * a.cpad) + a.phase * a.cpad;
    a.ring = (int)((a.phase * (size_t)per_chunk + a.factors * 4 + red_bytes + sum_bytes + 15) / 16 * 16);
    const size_t bytes = a.ring + kWarps * kAhead * slot;
    if (bytes > kSharedBudget) return cudaErrorNotSupported;       // (room() allows for none)
    // The whole budget, at every call: a call of another thread leaves the
    // kernel as this one needs it.
    cudaError_t e = cudaFuncSetAttribute(k_gemv<GRID, MT, NT, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSharedBudget);
    if (e != cudaSuccess) return e;
    return launch_in_order_smem(k_gemv<GRID, MT, NT, PL>, dim3((unsigned)grid), kThreads, bytes, 1, s, a);
}

cudaError_t dispatch(const GemvArgs &a, int grid, int most_cols, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    auto with = [&](auto gr, auto mt, auto nt) {
        constexpr int G = decltype(gr)::value, M = decltype(mt)::value, N = decltype(nt)::value;
        if (a.y_fp32 && (a.rht || a.x_fp32)) e = launch<G, M, N, 2>(a, most_cols, s);
        else e = launch<G, M, N, 1>(a, most_cols, s);
    };
    // Columns of a pass.  16384 x 4096 E1M2, rotated BF16 tokens, us: 8 tokens
    // 23; 16 tokens 36 as 16 columns, 46 as two passes of 8; 32 tokens 67 as
    // 32 columns of 16-row tiles (more would not leave registers for 32), 77 as
    // two passes of 16, 137 as four of 8.  By expert, where columns are what an
    // expert happens to have and passes after the first read L2, 8: 256 tokens x
    // 6 of 64 experts of 2048 x 2048 157, with 16 columns 171.
    auto by_cols = [&](auto gr) {
        if (most_cols <= 8 || a.offsets) with(gr, Int<2>(), Int<1>());
        else if (most_cols <= 16) with(gr, Int<2>(), Int<2>());
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
    a.signs = l.rht ? host_rht_sign_mask(l.rht_seed) : 0u;
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
    // By expert: no more columns than tokens.  (An expert that a token names
    // twice may have more, in further passes.)
    return dispatch(a, l.grid, (int)(l.offsets ? std::min(l.slots, l.tokens) : l.tokens), s);
}

}  // namespace ufp4
