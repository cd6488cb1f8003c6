// attn_wide.cu -- attention over the 4-bit cache for many queries a head of
// the cache (a tree of drafted tokens times a group of query heads), on the
// tensor cores' 128-row tiles (tcgen05, accumulators in TMEM).
//
// With 128 queries a row of the cache takes part in 32768 multiply-adds for 152
// bytes, so the decoding and the softmax bound it, not memory; both are done
// once for all queries:
//  * 8 warps copy rows (cp.async, three tiles ahead), decode them and write them as
//    FP16 into the 128-byte swizzled tiles that the MMAs read: keys K-major,
//    values in the same form, read as the N-major operand, so nothing is
//    transposed;
//  * one thread issues S = Q K^T (a second time for the queries' second FP16
//    value) of the next tile before O += P V of this one;
//  * 4 warps do the softmax, a thread a query: S from TMEM, the scales of its
//    key as factors, probabilities times their row's scale as FP16 into shared
//    memory; O stays in TMEM and is scaled only when the maximum rises by
//    more than 2^3 or a larger row scale appears.
// Waits are bounded: one that gives up raises the library's timeout flag, the
// CTA drains its MMAs and ends.
#include "attn.cuh"
#include "common.cuh"
#include "dequant.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "rowops.cuh"

#include <algorithm>

namespace ufp4 {

// Raised by a wait that gave up (read by ufp4_check).
__device__ uint32_t g_ufp4_attn_timeout;

cudaError_t read_attn_timeout_flag(uint32_t *flag, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(flag, g_ufp4_attn_timeout, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *flag) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbolAsync(g_ufp4_attn_timeout, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

namespace {

constexpr int kQ = kWideQueries, kKeys = 64, kStages = 3, kRing = 3;
constexpr int kSoftWarps = 4, kDecodeWarps = 8, kThreads = (kSoftWarps + kDecodeWarps + 1) * 32;
constexpr int kWarpKeys = kKeys / kDecodeWarps;          // rows of a tile that a warp decodes: one swizzle atom
constexpr long long kWaitBudget = 2000000000LL;          // SM clocks: about a second
constexpr uint32_t kTmemCols = 256;

template <int DC>
struct Smem {
    static constexpr int kDim = 64 * DC, kRow = kDim / 2, kBlocks = kDim / 16;
    static constexpr int kQPanel = kQ * 128, kPanel = kKeys * 128;                  // 64 elements of every row
    static constexpr int kHalf = DC * kPanel, kStage = 2 * kHalf;                   // keys, then values
    static constexpr int kP = kQ * 128;
    static constexpr int kRaw = 2 * kWarpKeys * (kRow + kBlocks + 4);               // a warp's rows of a tile as copied
    static constexpr int kOffQ = 0, kOffKv = kOffQ + 2 * DC * kQPanel, kOffP = kOffKv + kStages * kStage,
                         kOffRaw = kOffP + 2 * kP, kOffMeta = kOffRaw + kDecodeWarps * kRing * kRaw;
    // of each stage: row scales of the keys and values, the warps' largest exponents
    static constexpr int kMeta = kKeys * 8 + kDecodeWarps * 4;
    static constexpr int kOffRow = kOffMeta + kStages * kMeta;                      // of each query: mask, scale
    static constexpr int kOffBar = kOffRow + kQ * 12;
    static constexpr int kBars = 2 * kStages + 4;
    static constexpr int kBytes = kOffBar + kBars * 8 + 16;
};

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
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
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor of kind::f16: fp32 accumulators, FP16 operands,
// 128 x n; b_n_major: B's rows (its inner index) lie apart, its columns together.
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool b_n_major) {
    return 1u << 4 | (b_n_major ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(kQ >> 4) << 24;
}
// Byte offset of 16-byte piece c of row r of a swizzled tile (rows of 128 bytes).
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u + (uint32_t)((c ^ r) & 7) * 16u;
}

template <int GRID, int DC>
__global__ void __launch_bounds__(kThreads, 1) k_attn_wide(AttnArgs a) {
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
    const uint32_t p_ready = bars + (2 * kStages + 2) * 8, pv_done = p_ready + 8;
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
        if (lane == 0) {
            *stop = 0;
            for (int s = 0; s < kStages; ++s) {
                ptx::mbar_init(full(s), kDecodeWarps);
                ptx::mbar_init(empty(s), 1);
            }
            ptx::mbar_init(s_full(0), 1);
            ptx::mbar_init(s_full(1), 1);
            ptx::mbar_init(p_ready, kSoftWarps * 32);
            ptx::mbar_init(pv_done, 1);
            ptx::fence_mbar_init();
        }
    }
    const auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        const long long t0 = clock64();
        while (!*stop) {
#pragma unroll 1
            for (int i = 0; i < 256; ++i)
                if (ptx::mbar_try_wait(bar, parity)) return true;
            if (clock64() - t0 > kWaitBudget) {
                atomicOr(&g_ufp4_attn_timeout, 1u);
                *stop = 1;
            }
        }
        return false;
    };

    // ---- the queries as the 128-row operand
    {
        const uint32_t signs = a.rht ? rht_sign_mask(a.rht_seed) : 0u;
        const uint32_t group = ((1u << kBlocks) - 1u) << (lane & ~(kBlocks - 1));
        for (int i = tid; i < kQ * kBlocks; i += kThreads) {
            const int r = i / kBlocks, blk = i % kBlocks, q = q0 + r;
            float v[16] = {};
            if (r < nq && blk * 16 < a.dim) {
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
                if (a.rht) rotate16(v, signs);
            }
            uint32_t top = top_bits(v);
#pragma unroll
            for (int d = 1; d < kBlocks; d <<= 1) top = max(top, __shfl_xor_sync(group, top, d));
            const int e = top_exponent(top);
            const float up = exp2i(14 - e);
            if (blk == 0) {
                qf[r] = exp2i(e - 14) * kDecoded<GRID> * a.scale * 1.4426950408889634f;
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
                uint8_t *to = smem + M::kOffQ + blk / 4 * M::kQPanel + swizzled(r, blk % 4 * 2 + h);
                *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(to + DC * M::kQPanel) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
    }
    ptx::fence_proxy_async();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t o_col = tmem, s_col = tmem + 128;

    if (warp >= kSoftWarps && warp < kSoftWarps + kDecodeWarps) {
        // ------------------------------------------------- rows to operands
        const int w = warp - kSoftWarps, r = lane >> 2, t = lane & 3;
        uint64_t seen = 0;
        for (int i = 0; i < nq; ++i) seen |= qm[i];
        uint8_t *const mine = smem + M::kOffRaw + w * kRing * M::kRaw;
        const uint32_t mine_s = ptx::smem_u32(mine);
        constexpr int kCodes = kWarpKeys * kRow, kScales = kWarpKeys * kBlocks, kRs = kWarpKeys * 4;
        constexpr int kVal = kCodes + kScales + kRs;        // the values' part
        const int32_t *table = a.table + b * a.ld_table;
        const auto page_of = [&](int tile) -> int {
            const int pos = first + tile * kKeys + w * kWarpKeys;
            return tile < tiles && pos < last ? table[zero + (pos >> a.page_shift)] : -1;
        };
        int next = page_of(0);
        const auto copy = [&](int tile, int at) {
            if (tile < tiles) {
                const bool real = next >= 0 && next < a.pages;
                const int pos = first + tile * kKeys + w * kWarpKeys;
                const int64_t row =
                    real ? (((int64_t)next * a.kv + kvh) << a.page_shift) + (pos & ((1 << a.page_shift) - 1)) : 0;
                const uint32_t to = mine_s + at * M::kRaw;
                if (lane < kCodes / 16) {
                    copy16(to + lane * 16, a.k.codes + row * kRow + lane * 16, real);
                    copy16(to + kVal + lane * 16, a.v.codes + row * kRow + lane * 16, real);
                }
                constexpr int kS = kScales / 16, kR = kRs / 16;
                if (lane < 2 * kS) {
                    const int v = lane / kS, i = lane % kS;
                    copy16(to + v * kVal + kCodes + i * 16, (v ? a.v.scales : a.k.scales) + row * kBlocks + i * 16, real);
                } else if (lane < 2 * (kS + kR)) {
                    const int v = (lane - 2 * kS) / kR, i = (lane - 2 * kS) % kR;
                    copy16(to + v * kVal + kCodes + kScales + i * 16,
                           (v ? a.v.row_scale : a.k.row_scale) + row + i * 4, real);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            next = page_of(tile + 1);
        };
        for (int i = 0; i < kRing; ++i) copy(i, i);
        int at = 0, stage = 0;
        for (int i = 0; i < tiles; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            if (i >= kStages && !__all_sync(0xffffffffu, wait(empty(stage), (i / kStages - 1) & 1))) break;
            const uint8_t *from = mine + at * M::kRaw;
            const int pos = first + i * kKeys + w * kWarpKeys + r, rel = pos - (len - a.m);
            // rows that nobody sees may never have been written: their scales
            // become zero, and whatever codes stand there count for nothing
            const bool unseen = pos >= last || (rel >= 0 && !(seen >> rel & 1));
            uint8_t *const tile = smem + M::kOffKv + stage * M::kStage + w * 1024 + r * 128;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint8_t *p = from + half * kVal + r * kRow + t * (kRow / 4);
                const uint8_t *sp = from + half * kVal + kCodes + r * kBlocks + t * DC;
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
            // the row scales, and the exponent of the largest one of the values
            uint8_t *const meta = smem + M::kOffMeta + stage * M::kMeta;
            const float rs = unseen ? 0.0f : *reinterpret_cast<const float *>(from + (t & 1) * kVal + kCodes + kScales + r * 4);
            if (t < 2) reinterpret_cast<float *>(meta)[t * kKeys + w * kWarpKeys + r] = rs;
            const uint32_t top = __reduce_max_sync(0xffffffffu, t & 1 ? finite_bits(rs) : 0u);
            if (lane == 0) reinterpret_cast<int *>(meta + kKeys * 8)[w] = top_exponent(top);
            ptx::fence_proxy_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full(stage));
            copy(i + kRing, at);
            if (++at == kRing) at = 0;
            if (++stage == kStages) stage = 0;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp == kSoftWarps + kDecodeWarps) {
        // ------------------------------------------------------- the products
        if (lane == 0) {
            const auto scores = [&](int i) -> bool {
                const int stage = i % kStages;
                if (!wait(full(stage), (i / kStages) & 1)) return false;
                ptx::tc_fence_after();
                const uint32_t kt = smem_s + M::kOffKv + stage * M::kStage;
                uint32_t acc = 0;
                for (int p = 0; p < a.planes; ++p)
#pragma unroll
                    for (int d = 0; d < DC; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            mma_f16_ss(s_col + (i & 1) * kKeys,
                                       ptx::sdesc(smem_s + M::kOffQ + (p * DC + d) * M::kQPanel + k * 32, 16, 1024, 2),
                                       ptx::sdesc(kt + d * M::kPanel + k * 32, 16, 1024, 2), idesc(kKeys, false), acc);
                            acc = 1;
                        }
                ptx::tc_commit(s_full(i & 1));
                return true;
            };
            bool ok = tiles == 0 || scores(0);
            for (int i = 0; ok && i < tiles; ++i) {
                if (i + 1 < tiles && !(ok = scores(i + 1))) break;
                if (!(ok = wait(p_ready, i & 1))) break;
                ptx::tc_fence_after();
                const uint32_t vt = smem_s + M::kOffKv + (i % kStages) * M::kStage + M::kHalf;
                for (int p = 0; p < (a.two_p ? 2 : 1); ++p)
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_f16_ss(o_col, ptx::sdesc(smem_s + M::kOffP + p * M::kP + k * 32, 16, 1024, 2),
                                   ptx::sdesc(vt + k * 2048, M::kPanel, 1024, 2), idesc(kDim, true),
                                   i > 0 || p > 0 || k > 0);
                ptx::tc_commit(empty(i % kStages));
                ptx::tc_commit(pv_done);
            }
            if (!ok) {
                // what was issued ends before TMEM is given back: the first
                // tile's pair of barriers is nobody's any more
                ptx::tc_commit(s_full(0));
                const long long t0 = clock64();
                while (clock64() - t0 < kWaitBudget / 100) {}
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- the softmax
        const int r = tid;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const float qscale = qf[r];
        float mx = -INFINITY, l = 0.0f;
        int ve = -110, stage = 0;
        bool ok = true;
        for (int i = 0; i < tiles; ++i) {
            ok = wait(full(stage), (i / kStages) & 1) && wait(s_full(i & 1), (i >> 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint8_t *meta = smem + M::kOffMeta + stage * M::kMeta;
            const float *krs = reinterpret_cast<const float *>(meta), *vrs = krs + kKeys;
            const int *exps = reinterpret_cast<const int *>(meta + kKeys * 8);
            if (++stage == kStages) stage = 0;
            int ve_new = ve;
#pragma unroll
            for (int j = 0; j < kDecodeWarps; ++j) ve_new = max(ve_new, exps[j]);
            uint32_t raw[kKeys / 32][32];
#pragma unroll
            for (int h = 0; h < kKeys / 32; ++h) ptx::tc_ld_32x32b_x32(lanes + s_col + (i & 1) * kKeys + h * 32, raw[h]);
            ptx::tc_wait_ld();
            float s[kKeys];
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < kKeys; j += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(krs + j);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j + e] = __uint_as_float(raw[(j + e) / 32][(j + e) % 32]) * (kk[e] * qscale);
            }
            const int pos0 = first + i * kKeys;
            if (pos0 + kKeys > len - (a.m > 1 || a.mask ? a.m : 0)) {
                const uint64_t bits = qm[r];
#pragma unroll
                for (int j = 0; j < kKeys; ++j) {
                    const int rel = pos0 + j - (len - a.m);
                    if (pos0 + j >= last || (rel >= 0 && !(bits >> rel & 1))) s[j] = -INFINITY;
                }
            }
#pragma unroll
            for (int j = 0; j < kKeys; ++j) top = fmaxf(top, s[j]);
            // O and the place of the probabilities are the previous tile's until its product is done
            if (i > 0) {
                ok = wait(pv_done, (i - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
            }
            const bool rise = top > mx + 3.0f;
            if (__any_sync(0xffffffffu, rise || ve_new > ve)) {
                const float v = fmaxf(mx, top);
                const float back = exp2f(mx - (v == -INFINITY ? 0.0f : v));
                const float ob = back * exp2f((float)(ve - ve_new));
                mx = v;
                l *= back;
                ve = ve_new;
                if (i > 0) {
#pragma unroll
                    for (int h = 0; h < kDim / 32; ++h) {
                        uint32_t o[32];
                        ptx::tc_ld_32x32b_x32(lanes + o_col + h * 32, o);
                        ptx::tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * ob);
                        tc_st_32x32b_x32(lanes + o_col + h * 32, o);
                    }
                    tc_wait_st();
                }
            }
            const float base = mx == -INFINITY ? 0.0f : mx, vup = exp2i(11 - ve);
            uint8_t *const prow = smem + M::kOffP + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
            for (int c = 0; c < kKeys / 8; ++c) {
                float x[8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 v4 = *reinterpret_cast<const float4 *>(vrs + c * 8 + h * 4);
                    const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = s[c * 8 + h * 4 + e], p = exp2_fast(y - base);
                        l += p;
                        x[h * 4 + e] = y == -INFINITY ? 0.0f : p * (vv[e] * vup);
                    }
                }
                uint32_t hi[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) hi[e] = f16_pair(x[2 * e], x[2 * e + 1]);
                *reinterpret_cast<uint4 *>(prow + ((c ^ r) & 7) * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (a.two_p) {
                    uint32_t lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) lo[e] = f16_rest(x[2 * e], x[2 * e + 1], hi[e]);
                    *reinterpret_cast<uint4 *>(prow + M::kP + ((c ^ r) & 7) * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            ptx::fence_proxy_async();
            ptx::tc_fence_before();
            ptx::mbar_arrive(p_ready);
        }
        if (ok && tiles > 0) {
            ok = wait(pv_done, (tiles - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
        }
        if (ok) {
            const float down = exp2i(ve - 11) * kDecoded<GRID>;
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            const int q = q0 + r, node = q / a.group, head = kvh * a.group + q % a.group;
            const int64_t token = (int64_t)b * a.m + node;
            const int64_t part = ((int64_t)blockIdx.y * a.batch * a.kv + bh) * (a.group * a.m) + q;
            const uint32_t signs = a.rht && a.splits == 1 ? rht_sign_mask(a.rht_seed) : 0u;
#pragma unroll
            for (int h = 0; h < kDim / 32; ++h) {
                uint32_t o[32];
                if (tiles > 0) {
                    ptx::tc_ld_32x32b_x32(lanes + o_col + h * 32, o);
                    ptx::tc_wait_ld();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = 0;
                }
                if (r < nq) {
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j / 8 * 8 + code_order<GRID>(j % 8)] = __uint_as_float(o[blk * 16 + j]) * down;
                        const int col = h * 32 + blk * 16;
                        if (a.splits > 1) {
                            store_whole<16>(a.part_o + part * kDim + col, v);
                            continue;
                        }
                        if (col >= a.dim) continue;
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] *= inv;
                        if (a.rht) rotate16_back(v, signs);
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
            }
            if (r < nq) {
                if (a.splits > 1) {
                    a.part_m[part] = mx;
                    a.part_l[part] = l;
                } else if (a.lse) {
                    a.lse[token * a.heads + head] = (mx + log2f(l)) * 0.6931471805599453f;
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

template <int GRID, int DC>
cudaError_t wide(const AttnArgs &a, cudaStream_t s) {
    constexpr int bytes = Smem<DC>::kBytes + 1024;
    static_assert(bytes <= 232448, "shared memory of a CTA");
    const cudaError_t e =
        cudaFuncSetAttribute(k_attn_wide<GRID, DC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_in_order_smem(k_attn_wide<GRID, DC>,
                                dim3((unsigned)(a.batch * a.kv * a.qtiles), (unsigned)a.splits), kThreads, bytes, s, a);
}

}  // namespace

cudaError_t launch_attn_wide(const AttnArgs &a, int grid, int padded, cudaStream_t s) {
    if (grid == kE1M2) return padded == 64 ? wide<kE1M2, 1>(a, s) : wide<kE1M2, 2>(a, s);
    return padded == 64 ? wide<kE2M1, 1>(a, s) : wide<kE2M1, 2>(a, s);
}

}  // namespace ufp4
