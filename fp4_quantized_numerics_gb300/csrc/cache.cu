// cache.cu -- keys and values kept in 4 bits: written row by row as they
// come, read back, and attended over by new tokens.  (include/ufp4.h:
// ufp4_cache_append, ufp4_cache_load, ufp4_cache_attn.)
#include "attn.cuh"
#include "common.cuh"
#include "dequant.cuh"
#include "internal.h"
#include "rowops.cuh"

#include <algorithm>

namespace ufp4 {
namespace {

// ------------------------------------------------------------ write and read
// A row (one token's key or value of one head) is quantized by itself: its
// largest magnitude takes the place of the tensor's in ufp4_quantize.  A
// thread has one 16-block, the 4, 8 or 16 threads of a row exchange their
// maxima.  2 or 4 bytes an element in, 0.6 out: bound by memory for FP32 (32768
// tokens of 8 heads of 128, written and read back: 108 us, 84 % of the copy
// bandwidth), by the instructions of the rotation and of the rounding for BF16
// (262144 tokens rotated, E1M2: written in 490 us, 490 instructions a thread and
// 80 % of the issue slots; read in 335 us, 4.2 TB/s).
struct RowArgs {
    CacheHalf half[2];
    const void *x[2];            // append: k and v; load: unused
    void *y[2];
    int64_t ld_token[2], ld_head[2];
    int32_t fp32, wide;          // wide: rows of x / y in 32-byte accesses
    const int64_t *slots;
    int64_t places;              // pages x page
    int32_t heads, page_shift, dim, blocks, grid, rht;
    uint32_t signs;              // of the rotation
    RowDiv by_heads;
    uint64_t rows;               // tokens x heads
};

// Index of the cache's row for head h of a place.
__device__ __forceinline__ int64_t cache_row(int64_t slot, int32_t h, int32_t heads, int32_t page_shift) {
    const int64_t page = slot >> page_shift;
    return ((page * heads + h) << page_shift) + (slot & ((1 << page_shift) - 1));
}

template <class T>
__device__ __forceinline__ void load16(const T *p, bool wide, float (&v)[16]) {
    if (wide) {
        load_whole<16>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = load_one(p + i);
    }
}
template <class T>
__device__ __forceinline__ void store16(T *p, bool wide, const float (&v)[16]) {
    if (wide) {
        store_whole<16>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) store_one(p + i, v[i]);
    }
}

template <class T, int G, int GRID>       // G threads a row
__global__ void __launch_bounds__(128) k_append(RowArgs a) {
    const uint32_t zero = begin_in_order();
    const int which = blockIdx.y;
    const uint64_t at = (uint64_t)blockIdx.x * 128 + threadIdx.x;
    const uint64_t row = at / G;
    const int b = (int)(at % G);
    if (row >= a.rows) return;
    const uint64_t token = row_of(row, a.by_heads);
    const int32_t h = (int32_t)(row - token * a.heads);
    const int64_t slot = a.slots[zero + token];
    if (slot < 0 || slot >= a.places) return;
    float v[16] = {};
    const bool mine = b * 16 < a.dim;
    if (mine) {
        const T *p = static_cast<const T *>(a.x[which]) + token * a.ld_token[which] + h * a.ld_head[which] + b * 16;
        load16(p, a.wide, v);
        if (a.rht) rotate16(v, a.signs);
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max3_nan(top, fabsf(v[i]), fabsf(v[i + 1]));
    float all = top;
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t group = (G == 32 ? 0xffffffffu : ((1u << (G & 31)) - 1u)) << (lane & ~(G - 1u));
#pragma unroll
    for (int d = 1; d < G; d <<= 1) all = max_nan(all, __shfl_xor_sync(group, all, d));
    const bool finite = all < __uint_as_float(0x7F800000u);
    const float qmax = grid_qmax(a.grid), range = 448.0f * qmax;
    const float enc = all > 0.0f ? fminf(__fdiv_rn(range, all), kFltMax) : 1.0f;
    const float dec = all > 0.0f ? __fdiv_rn(all, range) : 1.0f;
    uint32_t e = e4m3_from_f32(__fmul_rn(__fdiv_rn(top, qmax), enc));
    if (!finite) e = 0;
    const float ev = e4m3_to_f32(e), r = e ? __fdiv_rn(enc, ev) : 0.0f;
    uint32_t w[2] = {0u, 0u};
    if (e) {
        const float most = (float)grid_top(a.grid);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            uint32_t two;
            if constexpr (GRID == kE2M1) {
                two = e2m1x2_rn(__fmul_rn(v[i], r), __fmul_rn(v[i + 1], r));
            } else {
                two = e1m2_rn(__fmul_rn(v[i], r), most) | (e1m2_rn(__fmul_rn(v[i + 1], r), most) << 4);
            }
            w[i / 8] |= two << (4 * (i % 8));
        }
    }
    if (b >= a.blocks) return;
    const CacheHalf c = a.half[which];
    const int64_t to = cache_row(slot, h, a.heads, a.page_shift);
    *reinterpret_cast<uint2 *>(c.codes + to * (a.blocks * 8) + b * 8) = make_uint2(w[0], w[1]);
    c.scales[to * a.blocks + b] = (uint8_t)e;
    if (b == 0) c.row_scale[to] = finite ? dec : __uint_as_float(0x7FC00000u);
}

template <class T, int G, int GRID>
__global__ void __launch_bounds__(128) k_load(RowArgs a) {
    const uint32_t zero = begin_in_order();
    const int which = blockIdx.y;
    const uint64_t at = (uint64_t)blockIdx.x * 128 + threadIdx.x;
    const uint64_t row = at / G;
    const int b = (int)(at % G);
    if (row >= a.rows || b * 16 >= a.dim) return;
    const uint64_t token = row_of(row, a.by_heads);
    const int32_t h = (int32_t)(row - token * a.heads);
    const int64_t slot = a.slots[zero + token];
    float v[16] = {};
    if (slot >= 0 && slot < a.places) {
        const CacheHalf c = a.half[which];
        const int64_t from = cache_row(slot, h, a.heads, a.page_shift);
        const uint2 w = *reinterpret_cast<const uint2 *>(c.codes + from * (a.blocks * 8) + b * 8);
        // value times block scale is exact in FP16; one rounding, by the row's scale
        const uint32_t e = scale_pair(c.scales[from * a.blocks + b], 0u);
        const float s = c.row_scale[from] * kDecoded<GRID>;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t p[4];
            decode8<GRID>(i ? w.y : w.x, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = f16_unpair(mul_pair(p[j], e));
                v[8 * i + code_order<GRID>(2 * j)] = __fmul_rn(f.x, s);
                v[8 * i + code_order<GRID>(2 * j + 1)] = __fmul_rn(f.y, s);
            }
        }
        if (a.rht) rotate16_back(v, a.signs);
    }
    T *p = static_cast<T *>(a.y[which]) + token * a.ld_token[which] + h * a.ld_head[which] + b * 16;
    store16(p, a.wide, v);
}

// ---------------------------------------------------------------- attention
// out = softmax(scale q K^T) V over a sequence's rows of the cache, for the
// `m` new tokens that end it; a group of query heads shares a head of the
// cache, and group x m queries are the columns of both products.
//
// Bound by reading the cache for one token (76 bytes for a row of 128 and 1024
// flops a query head).  A warp takes 32 rows at a time through both products
// by itself, with its own running maximum and sum:
//  * rows come by cp.async, 16 bytes a lane, a few tiles ahead, into shared
//    memory of the warp's own (no barrier in the loop);
//  * S^T = K q^T: keys are the 16-row operand, so a lane decodes 8 to 32 bytes
//    of a row's codes, which share 1 to 4 block scales, and a score's row scale
//    is a factor of the accumulator;
//  * O^T = V^T P^T: a lane decodes the same elements of four keys and pairs
//    them up by permutes; P^T becomes the other operand by movmatrix.
// The probabilities enter the product times their key's row scale, brought
// below 2^15 by a power of two of the query's own, which follows the largest of
// these products that it has seen (no row of values, however large, costs the
// others bits but for the queries in whose sum it counts), as FP16 (11 bits; two
// of them for fp32 results), and the sums are fp32.  Keys of a
// sequence are spread over warps, and over CTAs (splits) where sequences and
// heads are too few; the parts are joined in a fixed order, by a cluster for up
// to 8, else by a second kernel.
//
// Measured: one token of 31 sequences of 4096 to 8192 keys, 64 heads over 8,
// E1M2 rotated, 98 us (2.4 TB/s, 35 % of the copy bandwidth); of one sequence of
// 262111 keys, 32 heads over 4, E2M1, 60 us (39 %); 93 and 57 before the weights
// of the values followed each query and the second values had sums of their own.
// Bound by the instructions of decoding: some 1100 for 32 keys and values (57 % of
// the issue slots while all SMs work, the integer pipe fullest: an E1M2 code costs
// 10 operations a word of 8, an E2M1 one 4), where the copy bandwidth leaves 840;
// and by uneven lengths.
constexpr int kAttnWarps = 4, kTileKeys = 32;
constexpr int kCluster = 8;              // splits that a cluster joins

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// *p of the cluster's CTA `rank` (its y is its rank), p in this CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_at(const float *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_at(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_load4(const float *p, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_at(p, rank))
                 : "memory");
    return v;
}


__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Ends a row: O / l, back from the rotation, rounded once.  A lane has the 8
// elements 8 lane .. 8 lane + 7 (lanes past the row none).
__device__ __forceinline__ void finish_row(const AttnArgs &a, float (&o)[8], float m2, float l, int b, int q, int kvh,
                                           int lane) {
    const int node = q / a.group, head = kvh * a.group + q % a.group;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;      // (NaN stays)
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= inv;
    if (a.rht) {
        // the butterflies of 16 over two neighbouring lanes
        const uint32_t signs = a.signs >> (lane & 1) * 8;
        fwht8(o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, o[i], 1);
            const float v = (lane & 1 ? other - o[i] : o[i] + other) * 0.25f;
            o[i] = __uint_as_float(__float_as_uint(v) ^ ((signs << (31 - i)) & 0x80000000u));
        }
    }
    const int64_t token = (int64_t)b * a.m + node;
    const int64_t at = token * a.o_token + head * a.o_head + lane * 8;
    if (lane * 8 < a.dim) {
        if (a.out_fp32) {
            float *p = static_cast<float *>(a.out) + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = o[i];
        } else {
            __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(a.out) + at;
            if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
                store_words(p, w);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16_rn(o[i]);
            }
        }
    }
    if (a.lse && lane == 0)
        a.lse[token * a.heads + head] = (m2 + log2f(l)) * 0.6931471805599453f;   // no key: -inf + -inf
}

// DC: 64-element pieces of a padded row (1, 2 or 4); NT: groups of 8 queries.
template <int GRID, int DC, int NT>
__global__ void __launch_bounds__(kAttnWarps * 32, NT == 1 && DC <= 2 ? 4 : 2) k_attn(AttnArgs a) {
    constexpr int kDim = 64 * DC, kQ = 8 * NT, kRow = kDim / 2, kBlocks = kDim / 16;
    constexpr int kCodes = kTileKeys * kRow, kScales = kTileKeys * kBlocks, kRs = kTileKeys * 4;
    constexpr int kStage = 2 * (kCodes + kScales + kRs);
    // a stage: codes and scales of the keys, row scales of keys and values,
    // codes and scales of the values
    constexpr int kKeyRs = kCodes + kScales, kValRs = kKeyRs + kRs, kVal = kValRs + kRs;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4 *qs = reinterpret_cast<uint4 *>(smem);                       // [2][2 DC][kQ][4] x 16 bytes
    float *qf = reinterpret_cast<float *>(qs + 2 * 2 * DC * kQ * 4);   // [kQ]
    uint64_t *qm = reinterpret_cast<uint64_t *>(qf + kQ);              // [kQ]
    uint8_t *stages = reinterpret_cast<uint8_t *>(qm + kQ);
    const uint32_t zero = begin_in_order();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    const int qt = blockIdx.x % a.qtiles, bh = blockIdx.x / a.qtiles, kvh = bh % a.kv, b = bh / a.kv;
    const int most = a.width << a.page_shift;
    const int len = min(max(a.lens[zero + b], 0), most);
    int first, last;
    split_range(len, blockIdx.y, a.splits, first, last);
    if (a.splits > 1 && first >= last && !a.clustered) return;        // (the join does not look)
    const int q0 = qt * kQ, nq = min(a.group * a.m - q0, kQ);

    // ---- the rows' copies
    uint8_t *my = stages + warp * 2 * kStage;
    const uint32_t my_s = (uint32_t)__cvta_generic_to_shared(my);
    const int tiles = (last - first + kTileKeys - 1) / kTileKeys;
    const int32_t *table = a.table + b * a.ld_table;
    int next[2];                                      // pages of the next tile's two halves
    const auto look = [&](int tile) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = first + tile * kTileKeys + h * 16;
            next[h] = tile < tiles && pos < last ? table[zero + (pos >> a.page_shift)] : -1;
        }
    };
    int64_t row[2];                                   // the cache's rows of the tile being copied
    bool real[2];
    const auto copy_keys = [&](int tile, int slot) {
        const uint32_t to = my_s + slot * kStage;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = first + tile * kTileKeys + h * 16;
            real[h] = next[h] >= 0 && next[h] < a.pages;
            row[h] = real[h] ? (((int64_t)next[h] * a.kv + kvh) << a.page_shift) + (pos & ((1 << a.page_shift) - 1)) : 0;
        }
        if (tile < tiles) {
#pragma unroll
            for (int j = 0; j < 2 * DC; ++j) {
                const int h = j / DC;
                copy16(to + (j * 32 + lane) * 16, a.k.codes + row[h] * kRow + ((j % DC) * 32 + lane) * 16, real[h]);
            }
            if (lane < 8 * DC) {
                const int h = lane / (4 * DC);
                copy16(to + kCodes + lane * 16, a.k.scales + (h ? row[1] : row[0]) * kBlocks + lane % (4 * DC) * 16,
                       h ? real[1] : real[0]);
            }
            if (lane < 16) {
                const int h = lane / 4 % 2;
                copy16(to + kKeyRs + lane * 16,
                       (lane < 8 ? a.k.row_scale : a.v.row_scale) + (h ? row[1] : row[0]) + lane % 4 * 4,
                       h ? real[1] : real[0]);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const auto copy_values = [&](int tile, int slot) {
        const uint32_t to = my_s + slot * kStage + kVal;
        if (tile < tiles) {
#pragma unroll
            for (int j = 0; j < 2 * DC; ++j) {
                const int h = j / DC;
                copy16(to + (j * 32 + lane) * 16, a.v.codes + row[h] * kRow + ((j % DC) * 32 + lane) * 16, real[h]);
            }
            if (lane < 8 * DC) {
                const int h = lane / (4 * DC);
                copy16(to + kCodes + lane * 16, a.v.scales + (h ? row[1] : row[0]) * kBlocks + lane % (4 * DC) * 16,
                       h ? real[1] : real[0]);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look(warp);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        copy_keys(warp + i * kAttnWarps, i);
        copy_values(warp + i * kAttnWarps, i);
        look(warp + (i + 1) * kAttnWarps);
    }

    // ---- the queries as operands: [plane][word of a lane's elements][query][lane % 4]
    uint64_t seen = 0;
    for (int i = tid; i < kQ * kBlocks; i += kAttnWarps * 32) {
        const int col = i / kBlocks, blk = i % kBlocks, q = q0 + col;
        float v[16] = {};
        if (col < nq && blk * 16 < a.dim) {
            const int64_t at = ((int64_t)b * a.m + q / a.group) * a.q_token +
                               (kvh * a.group + q % a.group) * a.q_head + blk * 16;
            if (a.q_fp32) {
                const float *p = static_cast<const float *>(a.q) + at;
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = p[j];
            } else {
                const uint16_t *p = static_cast<const uint16_t *>(a.q) + at;
                if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[4];
                        load_words(p + 8 * h, w);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[8 * h + 2 * j] = bf16lo(w[j]);
                            v[8 * h + 2 * j + 1] = bf16hi(w[j]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float((uint32_t)p[j] << 16);
                }
            }
            if (a.rht) rotate16(v, a.signs);
        }
        uint32_t top = top_bits(v);
#pragma unroll
        for (int d = 1; d < kBlocks; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        const int e = top_exponent(top);
        const float up = exp2i(14 - e);
        if (blk == 0) {
            qf[col] = exp2i(e - 14) * kDecoded<GRID> * a.scale * 1.4426950408889634f;
            const int node = q / a.group;
            qm[col] = col >= nq ? 0ull : a.mask ? a.mask[(int64_t)b * a.m + node] : ~0ull >> (63 - node);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = v[8 * h + code_order<GRID>(2 * j)] * up, y = v[8 * h + code_order<GRID>(2 * j + 1)] * up;
                hi[j] = f16_pair(x, y);
                lo[j] = f16_rest(x, y, hi[j]);
            }
            const int at = (((blk % DC) * 2 + h) * kQ + col) * 4 + blk / DC;
            qs[at] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            qs[2 * DC * kQ * 4 + at] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    __syncthreads();
    for (int i = 0; i < nq; ++i) seen |= qm[i];

    float o[4 * DC][NT][4] = {};
    float mx[NT][2], l[NT][2] = {};
    float up[NT][2], limit[NT][2];                   // 2^(11 - we), and we + 3
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        mx[n][0] = mx[n][1] = -INFINITY;
        limit[n][0] = limit[n][1] = kLeastExponent + 3;
        up[n][0] = up[n][1] = exp2i(11 - kLeastExponent);
    }
    float qscale[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        qscale[n][0] = qf[n * 8 + 2 * t];
        qscale[n][1] = qf[n * 8 + 2 * t + 1];
    }

    int slot = 0;
    for (int tile = warp; tile < tiles; tile += kAttnWarps, slot ^= 1) {
        // (after these keys, the tile's values and the next tile's two groups are under way)
        asm volatile("cp.async.wait_group 3;" ::: "memory");
        __syncwarp();
        uint8_t *const ks = my + slot * kStage, *const vs = ks + kVal;
        const int pos0 = first + tile * kTileKeys;
        const bool edge = pos0 + kTileKeys > len - (a.m > 1 || a.mask ? a.m : 0);
        // rows that nobody sees may never have been written: their scales
        // become zero, so that whatever codes stand there count for nothing
        const int lane_rel = pos0 + lane - (len - a.m);
        const bool unseen = edge && (pos0 + lane >= last || (lane_rel >= 0 && !(seen >> lane_rel & 1)));
        const auto blank = [&](uint8_t *scales) {
            if (unseen)
#pragma unroll
                for (int j = 0; j < kBlocks / 4; ++j) reinterpret_cast<uint32_t *>(scales + lane * kBlocks)[j] = 0;
            __syncwarp();
        };
        if (edge) {
            if (unseen) {
                reinterpret_cast<float *>(ks + kKeyRs)[lane] = 0.0f;
                reinterpret_cast<float *>(ks + kValRs)[lane] = 0.0f;
            }
            blank(ks + kCodes);
        }

        // ---- scores: keys 16 i + g (and + 8) by queries 8 n + 2 t (and + 1)
        float s[2][NT][4] = {}, s2[2][NT][4] = {};      // s2: of the queries' second values
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t kw[2][2 * DC], kb[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int key = 16 * i + 8 * r + g;
                const uint8_t *p = ks + key * kRow + t * (kRow / 4), *sp = ks + kCodes + key * kBlocks + t * DC;
                if constexpr (DC == 1) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(p);
                    kw[r][0] = w.x; kw[r][1] = w.y;
                    kb[r] = *sp;
                } else {
#pragma unroll
                    for (int j = 0; j < DC / 2; ++j) {
                        const uint4 w = reinterpret_cast<const uint4 *>(p)[j];
                        kw[r][4 * j] = w.x; kw[r][4 * j + 1] = w.y; kw[r][4 * j + 2] = w.z; kw[r][4 * j + 3] = w.w;
                    }
                    if constexpr (DC == 2) kb[r] = *reinterpret_cast<const uint16_t *>(sp);
                    else kb[r] = *reinterpret_cast<const uint32_t *>(sp);
                }
            }
#pragma unroll
            for (int u = 0; u < 2 * DC; ++u) {
                uint32_t h[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t sc = scale_pair(kb[r], (u / 2) * 0x11u);
                    decode8<GRID>(kw[r][u], h[r]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[r][j] = mul_pair(h[r][j], sc);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 x = qs[(u * kQ + n * 8 + g) * 4 + t];
                    mma_f16(s[i][n], h[0][0], h[1][0], h[0][1], h[1][1], x.x, x.y);
                    mma_f16(s[i][n], h[0][2], h[1][2], h[0][3], h[1][3], x.z, x.w);
                    if (a.planes == 2) {
                        const uint4 y = qs[2 * DC * kQ * 4 + (u * kQ + n * 8 + g) * 4 + t];
                        mma_f16(s2[i][n], h[0][0], h[1][0], h[0][1], h[1][1], y.x, y.y);
                        mma_f16(s2[i][n], h[0][2], h[1][2], h[0][3], h[1][3], y.z, y.w);
                    }
                }
            }
        }
        float krs[4], vrs[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            krs[r] = reinterpret_cast<const float *>(ks + kKeyRs)[8 * r + g];
            vrs[r] = reinterpret_cast<const float *>(ks + kValRs)[8 * r + g];
        }
        __syncwarp();
        copy_keys(tile + 2 * kAttnWarps, slot);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][n][j] = (s[i][n][j] + s2[i][n][j]) * (krs[2 * i + (j >> 1)] * qscale[n][j & 1]);
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint64_t bits = qm[n * 8 + 2 * t + c];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int pos = pos0 + 8 * r + g, rel = pos - (len - a.m);
                        const bool hidden = pos >= last || (rel >= 0 && !(bits >> rel & 1));
                        if (hidden) s[r / 2][n][(r & 1) * 2 + c] = -INFINITY;
                    }
                }
        }

        // ---- running maximum and sum; weights of the values.  The maximum
        // follows the scores when one passes it by more than 2^3, and so does
        // the exponent of the weights: until then probabilities are up to 8,
        // and weights times 2^(11 - we) below 2^15.  Only what passed is moved:
        // a query's results do not depend on the others.
        float top[NT][2], wtop[NT][2];
        uint32_t vmost = 0, vleast = ~0u;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            vmost = max(vmost, __float_as_uint(vrs[r]));
            vleast = min(vleast, __float_as_uint(vrs[r]));
        }
        const float vexp = bits_exponent(vmost & 0x7FFFFFFFu);
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                top[n][c] = fmaxf(fmaxf(s[0][n][c], s[0][n][2 + c]), fmaxf(s[1][n][c], s[1][n][2 + c]));
                wtop[n][c] = vexp;
            }
        if (vmost - vleast > (uint32_t)kEvenScales << 23) {       // (NaN, too, unless all are)
            seldom();
            float own[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) own[r] = scale_exponent(vrs[r]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    wtop[n][c] = fmaxf(
                        fmaxf(s[0][n][c] - top[n][c] + own[0], s[0][n][2 + c] - top[n][c] + own[1]),
                        fmaxf(s[1][n][c] - top[n][c] + own[2], s[1][n][2 + c] - top[n][c] + own[3]));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                rise |= passes(mx[n][c], limit[n][c], top[n][c], wtop[n][c], 3.0f);
        if (__any_sync(0xffffffffu, rise)) {
            // (where the tile's scales are close, the largest of all serves)
            const uint32_t most = __reduce_max_sync(0xffffffffu, vmost & 0x7FFFFFFFu);
            const bool close = most - __reduce_min_sync(0xffffffffu, vleast) <= (uint32_t)kEvenScales << 23;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = top[n][c];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                    float w = bits_exponent(most);
                    if (!close) {
                        seldom();
                        w = top[n][c] - v + wtop[n][c];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, d));
                    }
                    const Rise to = rise_to(mx[n][c], 11 - power_of(up[n][c]), v, w, 3.0f);
                    mx[n][c] = to.mx;
                    up[n][c] = exp2i(11 - to.we);
                    limit[n][c] = (float)(to.we + 3);
                    l[n][c] *= to.l_back;
#pragma unroll
                    for (int i = 0; i < 4 * DC; ++i) {
                        o[i][n][c] *= to.o_back;
                        o[i][n][2 + c] *= to.o_back;
                    }
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float base = mx[n][c] == -INFINITY ? 0.0f : mx[n][c];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float &x = s[r / 2][n][(r & 1) * 2 + c];
                    const bool hidden = x == -INFINITY;
                    const float p = exp2_fast(x - base);
                    l[n][c] += p;
                    x = hidden ? 0.0f : p * up[n][c] * vrs[r];
                }
            }

        asm volatile("cp.async.wait_group 3;" ::: "memory");
        __syncwarp();
        if (edge) blank(vs + kCodes);

        // ---- values: elements of key 16 i + 2 t, + 1, + 8, + 9
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t h = f16_pair(s[i][n][2 * r], s[i][n][2 * r + 1]);
                    ph[n][r] = transpose8x8(h);
                    if (a.two_p) pl[n][r] = transpose8x8(f16_rest(s[i][n][2 * r], s[i][n][2 * r + 1], h));
                }
            uint32_t vw[4][DC], vb[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = 16 * i + 2 * t + (r & 1) + (r >> 1) * 8;
                const uint8_t *p = vs + key * kRow + g * (kRow / 8), *sp = vs + kCodes + key * kBlocks;
                if constexpr (DC == 1) {
                    vw[r][0] = *reinterpret_cast<const uint32_t *>(p);
                    vb[r] = sp[g >> 1];
                } else if constexpr (DC == 2) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(p);
                    vw[r][0] = w.x; vw[r][1] = w.y;
                    vb[r] = sp[g];
                } else {
                    const uint4 w = *reinterpret_cast<const uint4 *>(p);
                    vw[r][0] = w.x; vw[r][1] = w.y; vw[r][2] = w.z; vw[r][3] = w.w;
                    vb[r] = *reinterpret_cast<const uint16_t *>(sp + 2 * g);
                }
            }
#pragma unroll
            for (int u = 0; u < DC; ++u) {
                uint32_t h[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t sc = scale_pair(vb[r], DC == 4 ? (u / 2) * 0x11u : 0u);
                    decode8<GRID>(vw[r][u], h[r]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[r][j] = mul_pair(h[r][j], sc);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t a0 = __byte_perm(h[0][j], h[1][j], 0x5410), a1 = __byte_perm(h[0][j], h[1][j], 0x7632);
                    const uint32_t a2 = __byte_perm(h[2][j], h[3][j], 0x5410), a3 = __byte_perm(h[2][j], h[3][j], 0x7632);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16(o[4 * u + j][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
                        if (a.two_p) mma_f16(o[4 * u + j][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
                    }
                }
            }
        }
        __syncwarp();
        copy_values(tile + 2 * kAttnWarps, slot);
        look(tile + 3 * kAttnWarps);
    }

    // ---- the warps' parts together, in the stages' memory
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float *po = reinterpret_cast<float *>(stages);                 // [warp][query][kDim]
    float *pm = po + kAttnWarps * kQ * kDim, *pl = pm + kAttnWarps * kQ;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float down = exp2i(-power_of(up[n][c])) * kDecoded<GRID>;
            float sum = l[n][c];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const int col = n * 8 + 2 * t + c;
            if (g == 0) {
                pm[warp * kQ + col] = mx[n][c];
                pl[warp * kQ + col] = sum;
            }
            float *row = po + (warp * kQ + col) * kDim + g * (kDim / 8);
#pragma unroll
            for (int u = 0; u < DC; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        row[u * 8 + code_order<GRID>(2 * j + e)] = o[4 * u + j][n][2 * e + c] * down;
        }
    __syncthreads();
    for (int col = warp; col < nq; col += kAttnWarps) {
        float top = -INFINITY, sum = 0.0f, v[8] = {};
        for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, pm[w * kQ + col]);
        const float base = top == -INFINITY ? 0.0f : top;
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = exp2f(pm[w * kQ + col] - base);
            sum += pl[w * kQ + col] * f;
            if (lane * 8 < kDim) {
                const float *row = po + (w * kQ + col) * kDim + lane * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += row[i] * f;
            }
        }
        if (a.splits == 1) {
            finish_row(a, v, top, sum, b, q0 + col, kvh, lane);
        } else if (a.clustered) {
            // (in the place of the first warp's part, which these lanes have read)
            __syncwarp();
            if (lane * 8 < kDim) {
                float4 *to = reinterpret_cast<float4 *>(po + col * kDim + lane * 8);
                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                to[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
            if (lane == 0) {
                pm[col] = top;
                pl[col] = sum;
            }
        } else {
            const int64_t r = ((int64_t)blockIdx.y * a.batch * a.kv + bh) * (a.group * a.m) + q0 + col;
            if (lane * 8 < kDim) {
                float4 *to = reinterpret_cast<float4 *>(a.part_o + r * kDim + lane * 8);
                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                to[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
            if (lane == 0) {
                a.part_m[r] = top;
                a.part_l[r] = sum;
            }
        }
    }
    if (!a.clustered) return;
    // ---- the cluster's parts together: each CTA joins some of the queries
    cluster_sync();
    for (int col = blockIdx.y * kAttnWarps + warp; col < nq; col += a.splits * kAttnWarps) {
        float top = -INFINITY, sum = 0.0f, v[8] = {};
        for (int s = 0; s < a.splits; ++s) top = fmaxf(top, cluster_load(pm + col, s));
        const float base = top == -INFINITY ? 0.0f : top;
        for (int s = 0; s < a.splits; ++s) {
            const float f = exp2f(cluster_load(pm + col, s) - base);
            sum += cluster_load(pl + col, s) * f;
            if (lane * 8 < kDim) {
                const float4 x = cluster_load4(po + col * kDim + lane * 8, s),
                             y = cluster_load4(po + col * kDim + lane * 8 + 4, s);
                v[0] += x.x * f; v[1] += x.y * f; v[2] += x.z * f; v[3] += x.w * f;
                v[4] += y.x * f; v[5] += y.y * f; v[6] += y.z * f; v[7] += y.w * f;
            }
        }
        finish_row(a, v, top, sum, b, q0 + col, kvh, lane);
    }
    cluster_sync();                       // (the others have read this CTA's)
}

// Joins the splits' parts: W warps a query (of 8 in a CTA), each some of its
// parts, in a fixed order.
template <int W>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a, int kdim) {
    __shared__ float part[8][256 + 1];
    const uint32_t zero = begin_in_order();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % W;
    const int64_t queries = (int64_t)a.batch * a.kv * a.group * a.m;
    const int64_t r = (int64_t)blockIdx.x * (8 / W) + warp / W;
    float top = -INFINITY, sum = 0.0f, v[8] = {};
    int bh = 0, q = 0;
    if (r < queries) {
        const int per = a.group * a.m;
        bh = (int)(r / per);
        q = (int)(r % per);
        const int len = min(max(a.lens[zero + bh / a.kv], 0), a.width << a.page_shift);
        const int keys = split_keys(len, a.splits), parts = (len + keys - 1) / keys;
        for (int s = lane; s < parts; s += 32) top = fmaxf(top, a.part_m[s * queries + r + zero]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int s = mine; s < parts; s += W) {
            const float f = exp2f(a.part_m[s * queries + r + zero] - base);
            sum += a.part_l[s * queries + r + zero] * f;
            if (lane * 8 < kdim) {
                const float4 *from =
                    reinterpret_cast<const float4 *>(a.part_o + (s * queries + r + zero) * kdim + lane * 8);
                const float4 x = from[0], y = from[1];
                v[0] += x.x * f; v[1] += x.y * f; v[2] += x.z * f; v[3] += x.w * f;
                v[4] += y.x * f; v[5] += y.y * f; v[6] += y.z * f; v[7] += y.w * f;
            }
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[warp][i * 32 + lane] = v[i];
        if (lane == 0) part[warp][256] = sum;
        __syncthreads();
        if (mine) return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
            sum += part[warp + w][256];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += part[warp + w][i * 32 + lane];
        }
    }
    if (r < queries) finish_row(a, v, top, sum, bh / a.kv, q, bh % a.kv, lane);
}
cudaError_t join(const AttnArgs &a, int kdim, cudaStream_t s) {
    const int64_t queries = (int64_t)a.batch * a.kv * a.group * a.m;
    const auto with = [&](auto w) {
        constexpr int W = decltype(w)::value, per = 8 / W;
        return launch_in_order(k_attn_join<W>, (uint64_t)(queries + per - 1) / per, 256, s, a, kdim);
    };
    return a.splits <= 8 ? with(Int<1>()) : a.splits <= 32 ? with(Int<4>()) : with(Int<8>());
}

// The kernel's groups of queries (nt of 8; 0: the wide kernel's 128), how many
// of its CTAs share an SM, and the keys' time that its start and end take.
// Measured, 8 sequences of 8192 to 16384 keys of 8 heads of 128, E1M2, us, for 16
// / 20 / 32 queries a head: groups of 16 101 / 155 / 162, groups of 8 97 / 130 /
// 171, wide 142 / 141 / 145.  (256-element rows leave no registers for 16, and
// the wide kernel no TMEM.)  The wide kernel's start and end take 8 us, as long
// as 400 to 500 keys.  The number decides little: of 12 shapes (1 to 16 sequences
// of 1000 to 131072 keys, 32 to 512 queries a head) two differ between 128 and
// 1536: 8 of 8192 to 16384 keys with 64 queries take 139 us up to 256 and 146
// from 512 on, one of 131072 keys with 512, fp32, 318 up to 512 and 310 from 768.
struct Shape {
    int nt, qtiles, resident, start;
};
Shape shape_of(int64_t queries, int64_t padded) {
    if (queries > 16 && padded <= 128) return Shape{0, (int)((queries + kWideQueries - 1) / kWideQueries), 1, 768};
    const int nt = queries <= 8 || padded > 128 ? 1 : 2;
    return Shape{nt, (int)((queries + 8 * nt - 1) / (8 * nt)), nt == 1 && padded <= 128 ? 4 : 2, 64};
}
// Whether `splits` are joined within the kernel, by a cluster: one sequence of
// 1000 keys 8.2 us, with a second kernel 10.0 and a workspace.
bool clusters(int64_t splits, const Shape &shape) { return shape.nt && splits > 1 && splits <= kCluster; }
// Splits of a sequence: what makes an SM's CTAs times the keys of one, its start
// and end among them, the least; fewer CTAs than share an SM
// leave it idle, and every split is read again when they are joined.
int splits_of(int64_t batch, int64_t kv, const Shape &shape, int64_t most_keys) {
    const int64_t ctas = batch * kv * shape.qtiles, sms = num_sms();
    int64_t best = 1, least = INT64_MAX;
    for (int64_t s = 1; s <= 512 && (s == 1 || (s - 1) * kSplitKeys < most_keys); ++s) {
        const int64_t keys = (most_keys + s * kSplitKeys - 1) / (s * kSplitKeys) * kSplitKeys;
        const int64_t joined = s == 1 || clusters(s, shape) ? 0 : 1600 + 6 * s;
        const int64_t cost = std::max<int64_t>((ctas * s + sms - 1) / sms, shape.resident) * (keys + shape.start) + joined;
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return (int)best;
}

template <int GRID, int DC, int NT>
cudaError_t attn(const AttnArgs &a, cudaStream_t s) {
    constexpr int kDim = 64 * DC, kQ = 8 * NT;
    constexpr size_t kStage = 2 * (kTileKeys * (kDim / 2) + kTileKeys * (kDim / 16) + kTileKeys * 4);
    constexpr size_t parts = kAttnWarps * kQ * (kDim + 2) * sizeof(float);
    constexpr size_t bytes = 2 * 2 * DC * kQ * 4 * 16 + kQ * 12 + std::max(kAttnWarps * 2 * kStage, parts);
    cudaError_t e = cudaFuncSetAttribute(k_attn<GRID, DC, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    e = launch_in_order_smem(k_attn<GRID, DC, NT>, dim3((unsigned)(a.batch * a.kv * a.qtiles), (unsigned)a.splits),
                             kAttnWarps * 32, bytes, a.clustered ? a.splits : 1, s, a);
    if (e != cudaSuccess || a.splits == 1 || a.clustered) return e;
    return join(a, kDim, s);
}

template <class F>
cudaError_t by_threads(int blocks, F f) {
    return blocks <= 4 ? f(Int<4>()) : blocks <= 8 ? f(Int<8>()) : f(Int<16>());
}

RowArgs row_args(const CacheRows &l) {
    RowArgs a{};
    a.half[0] = l.cache.k;
    a.half[1] = l.cache.v;
    for (int i = 0; i < 2; ++i) {
        a.x[i] = l.x[i];
        a.y[i] = l.y[i];
        a.ld_token[i] = l.ld_token[i];
        a.ld_head[i] = l.ld_head[i];
    }
    a.fp32 = l.dtype == 1;
    const size_t size = type_size(l.dtype);
    a.wide = 1;
    for (int i = 0; i < 2; ++i) {
        const void *p = l.x[i] ? l.x[i] : l.y[i];
        a.wide = a.wide && rows_by(p, l.ld_token[i], size, 16) && rows_by(p, l.ld_head[i], size, 16);
    }
    a.slots = l.slots;
    a.places = l.cache.pages << l.cache.page_shift;
    a.heads = l.cache.heads;
    a.page_shift = l.cache.page_shift;
    a.dim = l.cache.dim;
    a.blocks = l.cache.padded / 16;
    a.grid = l.cache.grid;
    a.rht = l.cache.rht;
    a.signs = l.cache.rht ? host_rht_sign_mask(l.cache.rht_seed) : 0u;
    a.by_heads = make_rowdiv((uint32_t)l.cache.heads);
    a.rows = (uint64_t)l.tokens * l.cache.heads;
    return a;
}

}  // namespace

cudaError_t launch_cache_append(const CacheRows &l, cudaStream_t s) {
    const RowArgs a = row_args(l);
    return by_threads(a.blocks, [&](auto g) {
        constexpr int G = decltype(g)::value;
        const dim3 grid((unsigned)((a.rows * G + 127) / 128), 2);
        const auto with = [&](auto gr) {
            constexpr int K = decltype(gr)::value;
            return a.fp32 ? launch_in_order_smem(k_append<float, G, K>, grid, 128, 0, 1, s, a)
                          : launch_in_order_smem(k_append<__nv_bfloat16, G, K>, grid, 128, 0, 1, s, a);
        };
        // (the clamped grid rounds as the uniform one does)
        return a.grid == kE2M1 ? with(Int<kE2M1>()) : with(Int<kE1M2>());
    });
}

cudaError_t launch_cache_load(const CacheRows &l, cudaStream_t s) {
    const RowArgs a = row_args(l);
    return by_threads(a.blocks, [&](auto g) {
        constexpr int G = decltype(g)::value;
        const dim3 grid((unsigned)((a.rows * G + 127) / 128), 2);
        const auto with = [&](auto gr) {
            constexpr int K = decltype(gr)::value;
            return a.fp32 ? launch_in_order_smem(k_load<float, G, K>, grid, 128, 0, 1, s, a)
                          : launch_in_order_smem(k_load<__nv_bfloat16, G, K>, grid, 128, 0, 1, s, a);
        };
        return a.grid == kE1M2 ? with(Int<kE1M2>()) : with(Int<kE2M1>());
    });
}

size_t cache_attn_workspace(int64_t batch, int64_t m, int64_t heads, int64_t kv, int64_t padded, int64_t most_keys) {
    const int64_t queries = heads / kv * m;
    const Shape shape = shape_of(queries, padded);
    const int64_t splits = splits_of(batch, kv, shape, most_keys);
    return splits == 1 || clusters(splits, shape) ? 0 : (size_t)(splits * batch * m * heads * (padded + 2)) * sizeof(float);
}

cudaError_t launch_cache_attn(const CacheAttn &l, cudaStream_t s) {
    AttnArgs a{};
    a.q = l.q;
    a.q_token = l.q_token;
    a.q_head = l.q_head;
    a.q_fp32 = l.q_dtype == 1;
    a.planes = a.q_fp32 || l.cache.rht ? 2 : 1;      // (a BF16 query is an FP16 value times a power of two)
    a.k = l.cache.k;
    a.v = l.cache.v;
    a.table = l.table;
    a.ld_table = l.ld_table;
    a.width = (int)l.width;
    a.pages = (int)l.cache.pages;
    a.page_shift = l.cache.page_shift;
    a.lens = l.lens;
    a.mask = l.mask;
    a.batch = (int)l.batch;
    a.m = l.m;
    a.heads = l.heads;
    a.kv = l.cache.heads;
    a.group = l.heads / l.cache.heads;
    a.dim = l.cache.dim;
    a.rht = l.cache.rht;
    a.signs = l.cache.rht ? host_rht_sign_mask(l.cache.rht_seed) : 0u;
    a.scale = l.scale;
    a.out = l.out;
    a.o_token = l.o_token;
    a.o_head = l.o_head;
    a.out_fp32 = a.two_p = l.out_dtype == 1;
    a.lse = l.lse;
    const int64_t queries = (int64_t)a.group * a.m;
    const Shape shape = shape_of(queries, l.cache.padded);
    a.qtiles = shape.qtiles;
    a.splits = splits_of(a.batch, a.kv, shape, l.width << a.page_shift);
    a.clustered = clusters(a.splits, shape);
    const int64_t all = (int64_t)a.batch * a.kv * queries * a.splits;
    a.part_o = static_cast<float *>(l.workspace);
    a.part_m = a.part_o + all * l.cache.padded;
    a.part_l = a.part_m + all;
    if (shape.nt == 0) {
        const cudaError_t e = launch_attn_wide(a, l.cache.grid, l.cache.padded, s);
        return e != cudaSuccess || a.splits == 1 ? e : join(a, l.cache.padded, s);
    }
    const auto with = [&](auto gr, auto dc) {
        constexpr int G = decltype(gr)::value, D = decltype(dc)::value;
        if constexpr (D <= 2)
            if (shape.nt == 2) return attn<G, D, 2>(a, s);
        return attn<G, D, 1>(a, s);
    };
    const auto by_dim = [&](auto gr) {
        return l.cache.padded == 64 ? with(gr, Int<1>()) : l.cache.padded == 128 ? with(gr, Int<2>()) : with(gr, Int<4>());
    };
    return l.cache.grid == kE1M2 ? by_dim(Int<kE1M2>()) : by_dim(Int<kE2M1>());
}

}  // namespace ufp4
