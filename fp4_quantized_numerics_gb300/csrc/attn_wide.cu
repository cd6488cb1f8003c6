// attn_wide.cu -- attention over the 4-bit cache for many queries a head of
// the cache (a tree of drafted tokens times a group of query heads), on the
// tensor cores' 128-row tiles (tcgen05, accumulators in TMEM).
//
// With 128 queries a row of the cache takes part in 32768 multiply-adds for 152
// bytes, so the decoding and the softmax bound it, not memory; both are done
// once for all queries:
//  * 8 warps copy rows (cp.async, a few tiles ahead), decode them and write them
//    as FP16 into the 128-byte swizzled tiles that the MMAs read: keys K-major,
//    values in the same form, read as the N-major operand, so nothing is
//    transposed;
//  * one thread issues S = Q K^T (a second time for the queries' second FP16
//    value) of the next tile before O += P V of this one.  Q and P are the
//    operands from TMEM: from shared memory their 4 KB an MMA would take two to
//    three times the MMA's own time;
//  * 8 warps do the softmax, two threads a query (a tile's chain of dependent
//    steps, not the number of instructions, is what it takes), two keys an
//    instruction where there is one: S from TMEM, the row scale of its key as a
//    factor, the probabilities times their row's scale (and the query's own
//    power of two) as FP16 to TMEM.  O stays there; it is scaled, and the two
//    threads of a query speak, only when the largest score or weight of a query
//    rises by more than 2^8 (2^3 for fp32 results).
// Measured: trees of 32 tokens, 8 sequences of 8192 to 16384 keys, 32 heads over
// 8, E1M2 rotated, 152 us (353 TFLOP/s of the definition's; twice the queries'
// product in fact); 143 before the weights of the values followed each query
// (attn.cuh), and then 114 without the decoding.  A tile of 64 keys took some 5400
// instructions there (softmax 2200, decoding 1600, copies 400, the CTA's start 600)
// at 1.9 an SM and clock.  A CTA's start and end take 8 us, three times over.
// Steps on the way: operands in shared memory, one group of softmax warps 271 us;
// Q and P in TMEM 168; a pair of threads a query that agree only when a maximum
// rises 147; the MMAs issued by an elected lane rather than by lane 0 139 (its
// operands then need no moves to uniform registers).
//
// Waits are bounded: one that gives up raises the library's timeout flag, every
// role leaves, and the CTA waits for the MMAs that it issued and ends.
#include "attn.cuh"
#include "common.cuh"
#include "dequant.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rowops.cuh"

#include <algorithm>

namespace ufp4 {
namespace {

constexpr int kQ = kWideQueries, kKeys = 64, kStages = 3, kRing = 3;
constexpr int kSoftWarps = 8, kDecodeWarps = 8, kThreads = (kSoftWarps + kDecodeWarps + 1) * 32;
constexpr int kGroups = 2, kGroupWarps = kDecodeWarps / kGroups;   // decoding warps take every second tile,
constexpr int kWarpKeys = kKeys / kGroupWarps;                     // 16 rows of it each
// Keys whose scales are 2^80 and more: their products, up to 2^34, would leave
// fp32 times the scales.  A decoding warp marks their tile.
constexpr uint32_t kFarKeys = (80u + 127u) << 23;
constexpr int kFarMark = 1 << 16;
constexpr float kFarScores = 0x1p20f;                     // scores that fp32 holds to within 2^-4
constexpr long long kWaitBudget = 2000000000LL;          // SM clocks: about a second
// What the waits are given (and the test-only stall switch); a test-only build
// of the library can change them, libufp4 keeps the defaults.
long long g_attn_wait_budget = kWaitBudget;
int g_attn_stall = 0;
// TMEM: O, S of two tiles, Q's two FP16 values, P's of two tiles.
constexpr uint32_t kTmemCols = 512, kColS = 128, kColQ = 256, kColP = 384;

template <int DC>
struct Smem {
    static constexpr int kDim = 64 * DC, kRow = kDim / 2, kBlocks = kDim / 16;
    static constexpr int kPanel = kKeys * 128;                                      // 64 elements of every row
    static constexpr int kHalf = DC * kPanel, kStage = 2 * kHalf;                   // keys, then values
    static constexpr int kRaw = 2 * kWarpKeys * (kRow + kBlocks + 4);               // a warp's rows of a tile as copied
    // before the first tile, the queries: rows of two FP16 values, off each other's banks
    static constexpr int kQRow = kDim * 2 + 16, kQPlane = kQ * kQRow;
    static constexpr int kKvBytes = kStages * kStage > 2 * kQPlane ? kStages * kStage : 2 * kQPlane;
    static constexpr int kOffRaw = kKvBytes, kOffMeta = kOffRaw + kDecodeWarps * kRing * kRaw;
    // of each stage: row scales of the keys and values, the decoding warps' largest and least exponents of the latter
    static constexpr int kMeta = kKeys * 8 + kGroupWarps * 8;
    static constexpr int kOffRow = kOffMeta + kStages * kMeta;                      // of each query: mask, scale,
    static constexpr int kOffTop = kOffRow + kQ * 12;                               // its two threads' maxima or sums
    static constexpr int kOffBar = kOffTop + kQ * 16;
    static constexpr int kBars = 2 * kStages + 7;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16;
};

// The thread sleeps up to 10 us for the phase: a warp that polls takes issue
// slots and shared-memory accesses from those that work.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// D[tmem] (+)= A[tmem] B[smem]: A's row i in lane i, two FP16 a column.
template <bool ADD>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0)
                 : "memory");
}
__device__ __forceinline__ bool rows_of_16_bytes(const void *p, int64_t token, int64_t head) {     // of BF16
    return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)token * 2 | (uint64_t)head * 2) & 15) == 0;
}
// Two fp32 at a time.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor of kind::f16: fp32 accumulators, FP16 operands,
// 128 x n; b_n_major: B's rows (its inner index) lie apart, its columns together.
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_n_major) {
    return 1u << 4 | (b_n_major ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(kQ >> 4) << 24;
}

// TWO: the probabilities are two FP16 values (fp32 results).
template <int GRID, int DC, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) k_attn_wide(AttnArgs a, uint32_t *timeout, long long budget, int stall) {
    using M = Smem<DC>;
    constexpr int kDim = M::kDim, kRow = M::kRow, kBlocks = M::kBlocks;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *const smem = raw_smem + ((1024u - (ptx::smem_u32(raw_smem) & 1023u)) & 1023u);
    const uint32_t smem_s = ptx::smem_u32(smem);
    uint64_t *const qm = reinterpret_cast<uint64_t *>(smem + M::kOffRow);
    float *const qf = reinterpret_cast<float *>(qm + kQ);
    const uint32_t bars = smem_s + M::kOffBar;
    const auto full = [&](int s) { return bars + s * 8; };                          // a stage is decoded
    const auto empty = [&](int s) { return bars + (kStages + s) * 8; };             // its MMAs are done
    const auto s_full = [&](int i) { return bars + (2 * kStages + i) * 8; };        // scores are in TMEM
    // of every second tile: its probabilities are in TMEM; O has them
    const auto p_ready = [&](int i) { return bars + (2 * kStages + 2 + (i & 1)) * 8; };
    const auto pv_done = [&](int i) { return bars + (2 * kStages + 4 + (i & 1)) * 8; };
    const uint32_t drained = bars + (2 * kStages + 6) * 8;                          // after a failure: all MMAs are done
    uint32_t *const slot = reinterpret_cast<uint32_t *>(smem + M::kOffBar + M::kBars * 8);
    volatile uint32_t *const stop = slot + 1;
    const uint32_t zero = begin_in_order();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int qt = blockIdx.x % a.qtiles, bh = blockIdx.x / a.qtiles, kvh = bh % a.kv, b = bh / a.kv;
    const int len = min(max(a.lens[zero + b], 0), a.width << a.page_shift);
    int first, last;
    split_range(len, blockIdx.y, a.splits, first, last);
    if (a.splits > 1 && first >= last) return;
    const int q0 = qt * kQ, nq = min(a.group * a.m - q0, kQ);
    const int tiles = (last - first + kKeys - 1) / kKeys;

    if (warp == kSoftWarps + kDecodeWarps) {
        ptx::tmem_alloc(ptx::smem_u32(slot), kTmemCols);
        ptx::tmem_relinquish();
        if (ptx::elect_one()) {
            *stop = 0;
            for (int s = 0; s < kStages; ++s) {
                ptx::mbar_init(full(s), kGroupWarps);
                ptx::mbar_init(empty(s), 1);
            }
            for (int i = 0; i < 2; ++i) {
                ptx::mbar_init(s_full(i), 1);
                ptx::mbar_init(p_ready(i), kSoftWarps * 32);
                ptx::mbar_init(pv_done(i), 1);
            }
            ptx::mbar_init(drained, 1);
            ptx::fence_mbar_init();
        }
    }
    const auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (try_wait_long(bar, parity)) return true;
        const long long t0 = clock64();
        while (!*stop) {
            if (try_wait_long(bar, parity)) return true;
            if (clock64() - t0 > budget) {
                atomicOr(timeout, 1u);
                *stop = 1;
            }
        }
        return false;
    };

    // ---- the decoding warps' copies of rows; the first ones under way before all else
    const bool decodes = warp >= kSoftWarps && warp < kSoftWarps + kDecodeWarps;
    const int w = (warp - kSoftWarps) % kGroupWarps, grp = (warp - kSoftWarps) / kGroupWarps;
            uint8_t *const mine = smem + M::kOffRaw + (decodes ? warp - kSoftWarps : 0) * kRing * M::kRaw;
            const uint32_t mine_s = ptx::smem_u32(mine);
            constexpr int kCodes = kWarpKeys * kRow, kScales = kWarpKeys * kBlocks, kRs = kWarpKeys * 4;
            constexpr int kVal = kCodes + kScales + kRs;        // the values' part
            const int32_t *table = a.table + b * a.ld_table;
            const auto page_of = [&](int tile) -> int {
                const int pos = first + tile * kKeys + w * kWarpKeys;
                return tile < tiles && pos < last ? table[zero + (pos >> a.page_shift)] : -1;
            };
            int next = decodes ? page_of(grp) : -1;
            const auto copy = [&](int tile, int at) {
                if (tile < tiles) {
                    const bool real = next >= 0 && next < a.pages;
                    const int pos = first + tile * kKeys + w * kWarpKeys;
                    const int64_t row =
                        real ? (((int64_t)next * a.kv + kvh) << a.page_shift) + (pos & ((1 << a.page_shift) - 1)) : 0;
                    const uint32_t to = mine_s + at * M::kRaw + lane * 16;
                    const uint8_t *k = a.k.codes + row * kRow + lane * 16, *v = a.v.codes + row * kRow + lane * 16;
    #pragma unroll
                    for (int j = 0; j < kCodes / 512; ++j) {
                        copy16(to + j * 512, k + j * 512, real);
                        copy16(to + kVal + j * 512, v + j * 512, real);
                    }
                    constexpr int kS = kScales / 16, kR = kRs / 16;
                    if (lane < 2 * kS) {
                        const int v = lane / kS, i = lane % kS;
                        copy16(mine_s + at * M::kRaw + v * kVal + kCodes + i * 16,
                               (v ? a.v.scales : a.k.scales) + row * kBlocks + i * 16, real);
                    } else if (lane < 2 * (kS + kR)) {
                        const int v = (lane - 2 * kS) / kR, i = (lane - 2 * kS) % kR;
                        copy16(mine_s + at * M::kRaw + v * kVal + kCodes + kScales + i * 16,
                               (v ? a.v.row_scale : a.k.row_scale) + row + i * 4, real);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                next = page_of(tile + kGroups);
            };
    if (decodes)
        for (int i = 0; i < kRing; ++i) copy(grp + i * kGroups, i);
    const int tail = a.m > 1 || a.mask ? a.m : 0;

    // ---- the queries as the 128-row operand: through shared memory to TMEM
    {
        const uint32_t group = ((1u << kBlocks) - 1u) << (lane & ~(kBlocks - 1));
        constexpr int kTasks = (kQ * kBlocks + kThreads - 1) / kThreads;
        const auto place = [&](int i) -> int64_t {
            const int q = q0 + i / kBlocks;
            return ((int64_t)b * a.m + q / a.group) * a.q_token + (kvh * a.group + q % a.group) * a.q_head +
                   i % kBlocks * 16;
        };
        const bool wide = !a.q_fp32 && rows_of_16_bytes(a.q, a.q_token, a.q_head);
        uint32_t early[kTasks][8];                          // all loads under way before the first is used
#pragma unroll
        for (int n = 0; n < kTasks; ++n) {
            const int i = tid + n * kThreads;
#pragma unroll
            for (int j = 0; j < 8; ++j) early[n][j] = 0;
            if (wide && i / kBlocks < nq && i % kBlocks * 16 < a.dim) {
                uint32_t x[4], y[4];
                const uint16_t *p = static_cast<const uint16_t *>(a.q) + place(i);
                load_words(p, x);
                load_words(p + 8, y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    early[n][j] = x[j];
                    early[n][4 + j] = y[j];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kTasks; ++n) {
            const int i = tid + n * kThreads;
            if (i >= kQ * kBlocks) break;                   // (whole groups of lanes)
            const int r = i / kBlocks, blk = i % kBlocks, q = q0 + r;
            float v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[2 * j] = bf16lo(early[n][j]);
                v[2 * j + 1] = bf16hi(early[n][j]);
            }
            if (!wide && r < nq && blk * 16 < a.dim) {
                if (a.q_fp32) {
                    const float *p = static_cast<const float *>(a.q) + place(i);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = p[j];
                } else {
                    const uint16_t *p = static_cast<const uint16_t *>(a.q) + place(i);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float((uint32_t)p[j] << 16);
                }
            }
            if (a.rht) rotate16(v, a.signs);
            uint32_t top = top_bits(v);
#pragma unroll
            for (int d = 1; d < kBlocks; d <<= 1) top = max(top, __shfl_xor_sync(group, top, d));
            const int e = top_exponent(top);
            // (the scale's sign, or its being zero, goes with the queries)
            const float up = a.scale == 0.0f ? 0.0f : copysignf(exp2i(14 - e), a.scale);
            if (blk == 0) {
                // (not zero, by which a hidden key's -infinity would become NaN: where the factor underflows, 2^-149
                // in its place moves no score by more than 2^-21)
                qf[r] = a.scale == 0.0f ? 1.0f
                                        : fmaxf(exp2i(e - 14) * kDecoded<GRID> * fabsf(a.scale) * 1.4426950408889634f,
                                                __uint_as_float(1u));
                const int node = q / a.group;
                qm[r] = r >= nq ? 0ull : a.mask ? a.mask[(int64_t)b * a.m + node] : ~0ull >> (63 - node);
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
                uint8_t *to = smem + r * M::kQRow + blk * 32 + h * 16;
                *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(to + M::kQPlane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    if (warp < 4) {
#pragma unroll 1
        for (int p = 0; p < a.planes; ++p)
#pragma unroll 1
            for (int h = 0; h < DC; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 v =
                        *reinterpret_cast<const uint4 *>(smem + p * M::kQPlane + tid * M::kQRow + h * 128 + j * 16);
                    w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
                }
                tc_st_32x32b_x32(tmem + lanes + kColQ + (p * DC + h) * 32, w);
            }
        tc_wait_st();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::tc_fence_after();

    if (decodes) {
        // ------------------------------------------------- rows to operands
        const int r = lane >> 2, t = lane & 3;
        const uint64_t four = qm[lane] | qm[lane + 32] | qm[lane + 64] | qm[lane + 96];      // (rows past nq: 0)
        const uint64_t seen = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(four >> 32)) << 32 |
                              __reduce_or_sync(0xffffffffu, (uint32_t)four);
        int at = 0, stage = grp, round = 0;                  // round: how often the stage was filled before
        for (int i = grp; i < tiles; i += kGroups) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            if (round > 0 && !__all_sync(0xffffffffu, wait(empty(stage), (round - 1) & 1))) break;
            const uint8_t *from = mine + at * M::kRaw;
            uint8_t *const meta = smem + M::kOffMeta + stage * M::kMeta;
            const int pos0 = first + i * kKeys + w * kWarpKeys;
            const bool edge = pos0 + kWarpKeys > len - tail || pos0 + kWarpKeys > last;
            uint32_t vtop = 0, vleast = ~0u;                 // (a scale of zero weighs nothing)
            bool far = false;
#pragma unroll
            for (int part = 0; part < kWarpKeys / 8; ++part) {
                const int key = part * 8 + r;
                bool unseen = false;
                if (edge) {
                    // rows that nobody sees may never have been written: their
                    // scales become zero, and whatever codes stand there count
                    // for nothing
                    const int pos = pos0 + key, rel = pos - (len - a.m);
                    unseen = pos >= last || (rel >= 0 && !(seen >> rel & 1));
                }
                uint8_t *const tile = smem + stage * M::kStage + (w * (kWarpKeys / 8) + part) * 1024 + r * 128;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint8_t *p = from + half * kVal + key * kRow + t * (kRow / 4);
                    const uint8_t *sp = from + half * kVal + kCodes + key * kBlocks + t * DC;
                    uint32_t c[2 * DC], sb;
                    if constexpr (DC == 1) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(p);
                        c[0] = v.x; c[1] = v.y;
                        sb = *sp;
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4 *>(p);
                        // (the second panel's lanes start with their second
                        // piece, for the banks that their stores meet)
                        const bool turn = t >> 1;
                        c[0] = turn ? v.y : v.x; c[1] = turn ? v.x : v.y;
                        c[2] = turn ? v.w : v.z; c[3] = turn ? v.z : v.w;
                        sb = *reinterpret_cast<const uint16_t *>(sp);
                    }
                    if (unseen) sb = 0;
                    uint32_t sc[DC];
#pragma unroll
                    for (int j = 0; j < DC; ++j) sc[j] = scale_pair(sb, j * 0x11u);
#pragma unroll
                    for (int u = 0; u < 2 * DC; ++u) {
                        uint32_t h[4];
                        decode8<GRID>(c[u], h);
#pragma unroll
                        for (int j = 0; j < 4; ++j) h[j] = mul_pair(h[j], sc[u / 2]);
                        const int piece = DC == 1 ? 2 * t + u : (t & 1) * 4 + (u ^ (t >> 1));
                        const int panel = DC == 1 ? 0 : t >> 1;
                        *reinterpret_cast<uint4 *>(tile + half * M::kHalf + panel * M::kPanel + ((piece ^ r) & 7) * 16) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
                // the row scales (a lane the key's, the next the value's)
                float rs = *reinterpret_cast<const float *>(from + (t & 1) * kVal + kCodes + kScales + key * 4);
                if (unseen) rs = 0.0f;
                if (t < 2) reinterpret_cast<float *>(meta)[t * kKeys + w * kWarpKeys + key] = rs;
                const uint32_t bits = finite_bits(rs), value = t & 1 ? bits : 0u;
                vtop = max(vtop, value);
                vleast = min(vleast, value - 1);
                far |= !(t & 1) && bits >= kFarKeys;
            }
            vtop = __reduce_max_sync(0xffffffffu, vtop);
            vleast = __reduce_min_sync(0xffffffffu, vleast);
            far = __any_sync(0xffffffffu, far);
            if (lane == 0) {
                int *const exps = reinterpret_cast<int *>(meta + kKeys * 8);
                exps[w] = (int)(vtop >> 23) - 127 + (far ? kFarMark : 0);
                exps[kGroupWarps + w] = (int)(vleast >> 23) - 127;
            }
            ptx::fence_proxy_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full(stage));
            copy(i + kRing * kGroups, at);
            if (++at == kRing) at = 0;
            if ((stage += kGroups) >= kStages) {
                stage -= kStages;
                ++round;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp == kSoftWarps + kDecodeWarps) {
        // ------------------------------------------------------- the products
        if (ptx::elect_one()) {
            // Descriptors of the first stage; a stage, panel or step further
            // is an addition (of 16-byte units) to the low word.
            const uint64_t keys = ptx::sdesc(smem_s, 16, 1024, 2);
            const uint64_t values = ptx::sdesc(smem_s + M::kHalf, M::kPanel, 1024, 2);
            const auto scores = [&](int i, int stage, uint32_t parity) -> bool {
                if (!wait(full(stage), parity)) return false;
                ptx::tc_fence_after();
                const uint64_t kd = keys + (uint32_t)stage * (M::kStage / 16);
                const uint32_t d_col = tmem + kColS + (i & 1) * kKeys;
                const auto plane = [&](uint32_t q_col, bool add) {
#pragma unroll
                    for (int d = 0; d < DC; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (d == 0 && k == 0 && !add)
                                mma_f16_ts<false>(d_col, q_col, kd, idesc(kKeys, false));
                            else
                                mma_f16_ts<true>(d_col, q_col + d * 32 + k * 8, kd + d * (M::kPanel / 16) + k * 2,
                                                 idesc(kKeys, false));
                };
                // (the second values first: their sums are small, and the accumulator truncates)
                if (a.planes == 2) plane(tmem + kColQ + DC * 32, false);
                plane(tmem + kColQ, a.planes == 2);
                ptx::tc_commit(s_full(i & 1));
                return true;
            };
            bool ok = true;
#ifdef UFP4_PROBE
            // test-only build: a wait that nothing ends (`drained` is committed
            // only below), so that the way out runs
            if (stall) ok = wait(drained, 0);
#endif
            ok = ok && (tiles == 0 || scores(0, 0, 0));
            int stage = 0, ahead = 1 % kStages, ahead_round = 0;
            for (int i = 0; ok && i < tiles; ++i) {
                // (the place of S of the next tile: read before the probabilities of the last were ready)
                if (i + 1 < tiles && !(ok = scores(i + 1, ahead, ahead_round & 1))) break;
                if (++ahead == kStages) {
                    ahead = 0;
                    ++ahead_round;
                }
                if (!(ok = wait(p_ready(i), (i >> 1) & 1))) break;
                ptx::tc_fence_after();
                const uint64_t vd = values + (uint32_t)stage * (M::kStage / 16);
                const uint32_t p_col = tmem + kColP + (i & 1) * 64;
                if (i == 0) mma_f16_ts<false>(tmem, p_col, vd, idesc(kDim, true));
                else mma_f16_ts<true>(tmem, p_col, vd, idesc(kDim, true));
#pragma unroll
                for (int k = 1; k < kKeys / 16; ++k)
                    mma_f16_ts<true>(tmem, p_col + k * 8, vd + k * 128, idesc(kDim, true));
                if constexpr (TWO)
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_f16_ts<true>(tmem, p_col + 32 + k * 8, vd + k * 128, idesc(kDim, true));
                ptx::tc_commit(empty(stage));
                ptx::tc_commit(pv_done(i));
                if (++stage == kStages) stage = 0;
            }
            if (!ok) {       // TMEM is given back, and the operands' memory, when what was issued has ended
                ptx::tc_commit(drained);
                const long long t0 = clock64();
                while (!try_wait_long(drained, 0) && clock64() - t0 <= kWaitBudget) {}
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- the softmax
        const int half = warp >> 2, r = tid & (kQ - 1);          // keys 32 half .. of a tile
        constexpr int kMine = kKeys / 2;
        const uint32_t tm = tmem + lanes;
        const float qscale = qf[r];
        float mx = -INFINITY, l = 0.0f;
        int stage = 0, round = 0;
        bool ok = true;
        float *const tops = reinterpret_cast<float *>(smem + M::kOffTop), *const wtops = tops + 2 * kQ;     // [2][kQ] each
        // over the two warps that have the same queries; a barrier of whole warps
        const auto either = [&](bool v) -> bool {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
                         "barrier.cta.red.or.pred.aligned q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(r)
                         : "r"((uint32_t)v), "r"(1 + (warp & 3))
                         : "memory");
            return r != 0;
        };
        // The lanes of a warp come out of a wait together: what accesses TMEM
        // behind it are instructions of the whole warp.
        const auto wait_warp = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait(bar, parity));
        };
        // How far a maximum may pass the one that counts (exponents of 2), of
        // the scores and of the weights (attn.cuh): probabilities are up to
        // 2^slack, and FP16's normal numbers reach down to 2^(slack - 28) of the
        // query's largest weight.  A rise costs a pass over O, which BF16
        // results save more often (8 trees of 32 tokens: in most tiles some query
        // of 128 rises by 3).
        constexpr int slack = TWO ? 3 : 8;
        int we = kLeastExponent;                             // of the query's weights
        bool large = false;                                  // some maximum of the warp's is 2^20 or more
        // Scores times their key's scale (-infinity where hidden), the running
        // maximum, and the probabilities.  kAll: of any tile; else of one without
        // hidden or far keys, and given back where scores of 2^20 and more raise a
        // maximum.  vmost: the largest exponent of the tile's row scales.
        constexpr int kFailed = 0, kDone = 1, kOther = 2;
        const auto soften = [&](int i, int vmost, bool far, auto all_t) -> int {
            constexpr bool kAll = decltype(all_t)::value != 0;
            const uint8_t *meta = smem + M::kOffMeta + stage * M::kMeta;
            const float *krs = reinterpret_cast<const float *>(meta) + half * kMine, *vrs = krs + kKeys;
            const int4 least = *reinterpret_cast<const int4 *>(meta + kKeys * 8 + 16);
            const bool even = vmost - min(min(least.x, least.y), min(least.z, least.w)) <= kEvenScales;
            // (far keys: a factor of 2^64 goes from the products to the query's)
            const float qs = kAll && far ? qscale * 0x1p64f : qscale;
            const uint64_t qs2 = pack2(qs, qs);
            uint64_t z[kMine / 2];
            {
                uint32_t raw[kMine];
                ptx::tc_ld_32x32b_x32(tm + kColS + (i & 1) * kKeys + half * kMine, raw);
                ptx::tc_wait_ld();
                if (kAll && far) {
                    seldom();
#pragma unroll
                    for (int j = 0; j < kMine; ++j) raw[j] = __float_as_uint(__uint_as_float(raw[j]) * 0x1p-64f);
                }
#pragma unroll
                for (int j = 0; j < kMine; j += 4) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(krs + j);
                    const auto s = [&](int e) { return __uint_as_float(raw[j + e]); };
                    z[j / 2] = mul2(pack2(s(0), s(1)), pack2(k4.x, k4.y));
                    z[j / 2 + 1] = mul2(pack2(s(2), s(3)), pack2(k4.z, k4.w));
                }
            }
            if constexpr (kAll) {
                const uint64_t bits = qm[r];
                const int pos0 = first + i * kKeys + half * kMine;
#pragma unroll
                for (int j = 0; j < kMine; j += 2) {
                    float2 v = unpack2(z[j / 2]);
                    const int rel = pos0 + j - (len - a.m);
                    if (pos0 + j >= last || (rel >= 0 && !(bits >> rel & 1))) v.x = -INFINITY;
                    if (pos0 + j + 1 >= last || (rel >= -1 && !(bits >> (rel + 1) & 1))) v.y = -INFINITY;
                    z[j / 2] = pack2(v.x, v.y);
                }
            }
            float top = -INFINITY, other = -INFINITY;
#pragma unroll
            for (int j = 0; j < kMine / 2; j += 2) {
                const float2 u = unpack2(z[j]), v = unpack2(z[j + 1]);
                top = max3(top, u.x, u.y);
                other = max3(other, v.x, v.y);
            }
            top = fmaxf(top, other) * qs;
            float wtop = (float)vmost;
            if (!even) {
                seldom();
                wtop = -INFINITY;
#pragma unroll
                for (int j = 0; j < kMine; j += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(vrs + j), u = unpack2(z[j / 2]);
                    // (scores rounded as the largest was)
                    wtop = max3(wtop, __fadd_rn(__fmul_rn(u.x, qs), -top) + scale_exponent(v.x),
                                __fadd_rn(__fmul_rn(u.y, qs), -top) + scale_exponent(v.y));
                }
            }
            // the place of the probabilities was the last but one tile's
            // (or the scores never came)
            ok = ok && (i < 2 || wait_warp(pv_done(i), ((i >> 1) - 1) & 1));
            const bool rise = either(passes(mx, (float)(we + slack), top, wtop, (float)slack) || !ok);
            ptx::tc_fence_after();
            if (rise) {
                tops[half * kQ + r] = top;
                wtops[half * kQ + r] = wtop;
                const bool other = !kAll && fabsf(top) >= kFarScores;
                if (either(!ok || other)) return either(!ok) ? kFailed : kOther;
                const float best = fmaxf(tops[r], tops[kQ + r]);
                const Rise to = rise_to(mx, we, best, fmaxf(tops[r] - best + wtops[r], tops[kQ + r] - best + wtops[kQ + r]),
                                        (float)slack);
                mx = to.mx;
                we = to.we;
                if constexpr (kAll) large = __any_sync(0xffffffffu, fabsf(mx) >= kFarScores && mx != -INFINITY);
                l *= to.l_back;
                if (i > 0) {
                    // O has the last tile's product first
                    if (either(!wait_warp(pv_done(i - 1), ((i - 1) >> 1) & 1))) return kFailed;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int h = 0; h < kDim / 64; ++h) {
                        uint32_t o[32];
                        const uint32_t col = tm + (half * (kDim / 64) + h) * 32;
                        ptx::tc_ld_32x32b_x32(col, o);
                        ptx::tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * to.o_back);
                        tc_st_32x32b_x32(col, o);
                    }
                }
            }
            const float base = mx == -INFINITY ? 0.0f : -mx, up = exp2i(14 - slack - we);
            const uint64_t base2 = pack2(base, base), up2 = pack2(up, up);
            uint64_t sums[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
            for (int c = 0; c < kMine; c += 16) {
                uint32_t hi[8];
                [[maybe_unused]] uint32_t lo[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(vrs + c + 2 * j);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // (kAll: rounded as the maximum was, before that is taken off, which matters far from 0)
                        float2 y;
                        if constexpr (kAll) {
                            const float2 u = unpack2(z[c / 2 + j + e]);
                            y = make_float2(__fadd_rn(__fmul_rn(u.x, qs), base), __fadd_rn(__fmul_rn(u.y, qs), base));
                        } else {
                            y = unpack2(fma2(z[c / 2 + j + e], qs2, base2));
                        }
                        const uint64_t p = pack2(exp2_fast(y.x), exp2_fast(y.y));
                        sums[e] = add2(sums[e], p);
                        float2 x = unpack2(mul2(mul2(p, up2), e ? pack2(v4.z, v4.w) : pack2(v4.x, v4.y)));
                        if constexpr (kAll) {
                            if (y.x == -INFINITY) x.x = 0.0f;
                            if (y.y == -INFINITY) x.y = 0.0f;
                        }
                        hi[j + e] = f16_pair(x.x, x.y);
                        if constexpr (TWO) lo[j + e] = f16_rest(x.x, x.y, hi[j + e]);
                    }
                }
                const uint32_t to = tm + kColP + (i & 1) * 64 + half * 16 + c / 2;
                tc_st_32x32b_x8(to, hi);
                if constexpr (TWO) tc_st_32x32b_x8(to + 32, lo);
            }
            const float2 two = unpack2(add2(sums[0], sums[1]));
            l += two.x + two.y;
            tc_wait_st();
            return kDone;
        };
        for (int i = 0; i < tiles; ++i) {
            ok = wait(full(stage), round & 1) && wait(s_full(i & 1), (i >> 1) & 1);
            if (!(ok = __all_sync(0xffffffffu, ok))) *stop = 1;  // (the others stop at their next wait)
            ptx::tc_fence_after();
            const int end = first + (i + 1) * kKeys;
            const int4 exps = *reinterpret_cast<const int4 *>(smem + M::kOffMeta + stage * M::kMeta + kKeys * 8);
            int vmost = max(max(exps.x, exps.y), max(exps.z, exps.w));
            const bool far = vmost >= kFarMark / 2;
            if (far) {
                seldom();
                const auto bare = [](int e) { return e >= kFarMark / 2 ? e - kFarMark : e; };
                vmost = max(max(bare(exps.x), bare(exps.y)), max(bare(exps.z), bare(exps.w)));
            }
            int did = kOther;
            if (end <= len - tail && end <= last && !far && !large) did = soften(i, vmost, false, Int<0>());
            if (did == kOther) did = soften(i, vmost, far, Int<1>());
            if (did != kDone) {
                ok = false;
                break;
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(p_ready(i));
            if (++stage == kStages) {
                stage = 0;
                ++round;
            }
        }
        if (ok && tiles > 0) ok = wait_warp(pv_done(tiles - 1), ((tiles - 1) >> 1) & 1);
        tops[half * kQ + r] = l;
        ok = !either(!ok);
        ptx::tc_fence_after();
        if (ok) {
            const float sum = tops[r] + tops[kQ + r];
            const float down = exp2i(we - 14 + slack) * kDecoded<GRID>;
            const float inv = sum > 0.0f || sum != sum ? down / sum : 0.0f;
            const int q = q0 + r, node = q / a.group, head = kvh * a.group + q % a.group;
            const int64_t token = (int64_t)b * a.m + node;
            const int64_t part = ((int64_t)blockIdx.y * a.batch * a.kv + bh) * (a.group * a.m) + q;
#pragma unroll 1
            for (int h = half * DC; h < (half + 1) * DC; ++h) {
                uint32_t o[32];
                __syncwarp();
                ptx::tc_ld_32x32b_x32(tm + h * 32, o);
                ptx::tc_wait_ld();
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    if (r >= nq) break;
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j / 8 * 8 + code_order<GRID>(j % 8)] =
                            tiles == 0 ? 0.0f : __uint_as_float(o[blk * 16 + j]) * (a.splits > 1 ? down : inv);
                    const int col = h * 32 + blk * 16;
                    if (a.splits > 1) {
                        float4 *to = reinterpret_cast<float4 *>(a.part_o + part * kDim + col);   // (16-byte aligned)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        continue;
                    }
                    if (col >= a.dim) continue;
                    if (a.rht) rotate16_back(v, a.signs);
                    const int64_t at = token * a.o_token + head * a.o_head + col;
                    if (a.out_fp32) {
                        float *p = static_cast<float *>(a.out) + at;
                        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
                            store_whole<16>(p, v);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) p[j] = v[j];
                        }
                    } else {
                        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(a.out) + at;
                        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
                            store_whole<16>(p, v);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) p[j] = __float2bfloat16_rn(v[j]);
                        }
                    }
                }
            }
            if (r < nq && half == 0) {
                if (a.splits > 1) {
                    a.part_m[part] = mx;
                    a.part_l[part] = sum;
                } else if (a.lse) {
                    a.lse[token * a.heads + head] = (mx + log2f(sum)) * 0.6931471805599453f;
                }
            }
        }
        ptx::tc_fence_before();
    }
    __syncthreads();
    if (warp == kSoftWarps + kDecodeWarps) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int GRID, int DC, bool TWO>
cudaError_t wide(const AttnArgs &a, cudaStream_t s) {
    constexpr int bytes = Smem<DC>::kBytes + 1024;
    static_assert(bytes <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(k_attn_wide<GRID, DC, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    uint32_t *timeout = nullptr;         // raised by a wait that gives up (read by ufp4_check)
    if (e == cudaSuccess) e = timeout_flag(&timeout);
    if (e != cudaSuccess) return e;
    return launch_in_order_smem(k_attn_wide<GRID, DC, TWO>,
                                dim3((unsigned)(a.batch * a.kv * a.qtiles), (unsigned)a.splits), kThreads, bytes, 1, s, a,
                                timeout, g_attn_wait_budget, g_attn_stall);
}

}  // namespace

cudaError_t launch_attn_wide(const AttnArgs &a, int grid, int padded, cudaStream_t s) {
    const auto with = [&](auto gr, auto dc) {
        constexpr int G = decltype(gr)::value, D = decltype(dc)::value;
        return a.two_p ? wide<G, D, true>(a, s) : wide<G, D, false>(a, s);
    };
    const auto by_dim = [&](auto gr) { return padded == 64 ? with(gr, Int<1>()) : with(gr, Int<2>()); };
    return grid == kE1M2 ? by_dim(Int<kE1M2>()) : by_dim(Int<kE2M1>());
}

}  // namespace ufp4

#ifdef UFP4_PROBE
#include "probe_attn.inc"
#endif
