// moe.cu -- tokens into expert order and back, for the grouped GEMMs of an
// MoE layer ([HP] hotpaper.ai card, technical approach: MoE 7.9B and 124B
// models; the pages give no kernels for this).  The contract is in
// include/ufp4.h.
//
// Every kernel but the sort reads or writes each row element once and does
// fewer than two operations a byte, so memory bounds them; the sort moves 16
// bytes a slot and is bound by its steps' latency.  Times below: one GB300,
// 16384 tokens x top-6 of 64 experts (98304 slots), rows of 2048, unless
// stated; "of measured" is of the 6676 GB/s of a plain copy.
#include "common.cuh"
#include "internal.h"
#include "rowops.cuh"

#include <algorithm>
#include <type_traits>

namespace ufp4 {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- sort
// Stable counting sort of n expert ids (bucket E = dropped) by one cluster.
// Every warp of the cluster owns a contiguous range of slots, in order.
//   1. A histogram per warp in shared memory, summed over the CTA's warps.
//   2. The CTAs read each other's sums over distributed shared memory: a
//      bucket's first place in the order is the sum of all smaller buckets,
//      a CTA's the sums of the CTAs before it, a warp's those of the warps
//      before it.
//   3. A warp takes 32 slots at a time; lanes of one expert find each other
//      by one ballot per bit of the expert's number, and a lane's place is
//      the warp's running place plus the number of such lanes before it.
// One launch and no scratch memory: 98304 slots take 9 us, of which about 4
// are the steps between the passes and the launch; 524288 slots of 256 experts
// 31 us.  The passes are bound by the 16 of 152 SMs that a cluster has, none of
// whose units is full: at 524288 slots the integer pipe is 58 % busy, 54 % of
// the issue slots are used (142 warp instructions per 32 slots), and a third of
// a warp's time it waits for ids.  Measured slower at 98304: one CTA (71 us),
// __match_any_sync for the ballots (2 us more), ranks kept from the first pass
// through pos (2 us more).  Several clusters and two more kernels that join
// them are faster above some 200000 slots (524288: 18 us; 98304: 9 to 10) and
// not built.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxSortCtas = 16;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// *p of the cluster's CTA `rank`, p in this CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t *p, uint32_t rank) {
    uint32_t a, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(a)
        : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

template <class Id>
__device__ __forceinline__ uint32_t bucket_of(const Id *ids, uint32_t i, uint32_t E) {
    const Id id = ids[i];
    return id >= 0 && id < (Id)E ? (uint32_t)id : E;
}

// The lanes of the warp whose b (of `bits` bits) equals this lane's, among
// those of `in`.
__device__ __forceinline__ uint32_t lanes_like(uint32_t b, int bits, bool in) {
    uint32_t same = __ballot_sync(0xFFFFFFFFu, in);
    for (int k = 0; k < bits; ++k) {
        const bool set = (b >> k) & 1u;
        const uint32_t v = __ballot_sync(0xFFFFFFFFu, set);
        same &= set ? v : ~v;
    }
    return same;
}

template <class Id>
__global__ void __launch_bounds__(kSortThreads) k_moe_sort(const Id *ids, uint32_t n, uint32_t E, int32_t *pos,
                                                           int32_t *src, int64_t *counts, int64_t *offsets) {
    __shared__ uint32_t hist[kSortWarps * (kMaxGroups + 1)];   // [warp][bucket]
    __shared__ uint32_t sums[kMaxGroups + 1];                  // this CTA's, read by the others
    __shared__ uint32_t warp_sum[kSortWarps];
    const uint32_t zero = begin_in_order();
    const uint32_t tid = threadIdx.x + zero, lane = tid & 31u, warp = tid >> 5, B = E + 1, W = blockDim.x / 32;
    const uint32_t rank = cluster_rank(), nctas = cluster_size();
    const uint32_t warps = nctas * W;
    const int bits = 32 - __clz((int)E);
    const uint32_t per = ((n + warps - 1u) / warps + 31u) / 32u * 32u;   // slots of a warp: a multiple of 32
    const uint32_t lo = (uint32_t)min((uint64_t)n, (uint64_t)(rank * W + warp) * per), hi = min(n, lo + per);
    uint32_t *mine = hist + warp * B;

    for (uint32_t i = tid; i < W * B; i += blockDim.x) hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (uint32_t i = lo + lane; i < hi; i += 32) atomicAdd(mine + bucket_of(ids, i, E), 1u);
    __syncthreads();

    uint32_t total = 0, before_me = 0;   // of bucket tid: in all CTAs, in those before this one
    if (tid < B) {
#pragma unroll 8
        for (uint32_t w = 0; w < W; ++w) total += hist[w * B + tid];
        sums[tid] = total;
    }
    if (nctas > 1) {
        cluster_arrive();
        cluster_wait();
        if (tid < B) {
            total = 0;
#pragma unroll 8
            for (uint32_t r = 0; r < nctas; ++r) {
                const uint32_t c = cluster_load(sums + tid, r);
                total += c;
                before_me += r < rank ? c : 0u;
            }
        }
        cluster_arrive();   // this CTA has read the others' sums; waited for before it ends
    }
    // exclusive sum of the totals over the buckets
    uint32_t incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= (uint32_t)d) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (tid < B) {
        uint32_t first = incl - total;
        for (uint32_t w = 0; w < warp; ++w) first += warp_sum[w];
        if (rank == 0) {
            offsets[tid] = first;
            if (tid < E) counts[tid] = total;
        }
        first += before_me;
#pragma unroll 8
        for (uint32_t w = 0; w < W; ++w) {
            const uint32_t c = hist[w * B + tid];
            hist[w * B + tid] = first;
            first += c;
        }
    }
    __syncthreads();

    uint32_t next = lo + lane < hi ? bucket_of(ids, lo + lane, E) : 0u;
    for (uint32_t base = lo; base < hi; base += 32) {
        const uint32_t i = base + lane, b = next;
        const bool in = i < hi;
        if (i + 32 < hi) next = bucket_of(ids, i + 32, E);
        const uint32_t same = lanes_like(b, bits, in);
        const uint32_t before = __popc(same & ((1u << lane) - 1u));
        uint32_t p = 0;
        if (in) p = mine[b] + before;
        __syncwarp();
        if (in && before == 0) mine[b] = p + __popc(same);
        __syncwarp();
        if (in) {
            pos[i] = (int32_t)p;
            src[p] = (int32_t)i;
        }
    }
    if (nctas > 1) cluster_wait();
}

// --------------------------------------------------------------- dispatch
// A thread reads its part of a token's row once and writes it topk times (not:
// a thread per result row, which would read x topk times): one 16-byte unit
// where all rows are 16-byte aligned, else eight elements a warp's width
// apart.  Bound by DRAM writes: 71 us, 6.7 TB/s (100 % of measured); rows of
// 1001 BF16 elements 45 us (76 %), bound by the number of 64-byte accesses.
template <class Unit, int N>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch(const Unit *x, int64_t ld_x, Unit *__restrict__ xs,
                                                           int64_t ld_xs, const int32_t *pos,
                                                           const int64_t *routed_at, int topk, uint32_t width,
                                                           RowDiv units, uint64_t work) {
    const uint32_t zero = begin_in_order();
    uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x + zero;
    if constexpr (N > 1) i /= 32;
    if (i >= work) return;
    const uint64_t t = row_of(i, units);
    const uint32_t u = (uint32_t)(i - t * units.d);
    const uint32_t c = N > 1 ? u * (32 * N) + (threadIdx.x & 31u) : u;
    Unit v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = c + 32 * e < width ? x[t * ld_x + c + 32 * e] : Unit{};
    const int32_t routed = (int32_t)routed_at[zero];
    const int32_t *at = pos + t * topk;
    for (int j = 0; j < topk; ++j) {
        const int32_t p = at[j];
        Unit *to = xs + (int64_t)p * ld_xs + c;
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c + 32 * e < width) to[32 * e] = p < routed ? v[e] : Unit{};
    }
}

// ---------------------------------------------------------------- combine
// A thread owns N elements of an output row (32 bytes of y in the whole
// layout); the topk rows are added in ascending order of choice, in fp32, and
// rounded once.  Bound by DRAM reads: fp32 to BF16 124 us, 7.0 TB/s (105 % of
// measured: reads run faster than a copy); 16384 x 8 BF16 rows of 4096 178 us
// (102 %; 203 us with 16-byte accesses).  Loading the rows of several choices
// before adding them takes registers, and so warps: 155 us.  Off the whole
// layout the loop stays rolled: rows of 1002 BF16 43 us (80 %; unrolled 53),
// of 1001 54 us (64 %; two rows at once 74, four 117: neighbouring accesses
// share sectors, which more rows in flight push out of L1).
//
// CTAs of 128 threads are 1-5 % faster, and 4 % slower with 16 elements a
// thread.
template <int N>
constexpr int kCombineThreads = N == 16 ? 256 : 128;

template <class Ty, class To, int L, int N>
__global__ void __launch_bounds__(kCombineThreads<N>)
    k_moe_combine(const Ty *y, int64_t ld_y, const int32_t *pos, const float *weights, const int64_t *routed_at,
                  To *__restrict__ out, int64_t ld_out, int topk, uint32_t hidden, RowDiv parts, uint64_t work) {
    const uint32_t zero = begin_in_order();
    uint64_t i = (uint64_t)blockIdx.x * kCombineThreads<N> + threadIdx.x + zero;
    if (L != kWhole) i /= 32;
    if (i >= work) return;
    const uint64_t t = row_of(i, parts);
    const Part<L, N> part((uint32_t)(i - t * parts.d), hidden);
    const int32_t routed = (int32_t)routed_at[zero];
    float acc[N] = {};
#pragma unroll(L == kWhole ? 4 : 1)
    for (int j = 0; j < topk; ++j) {
        const int32_t p = pos[t * topk + j];
        if (p >= routed) continue;
        const float w = weights ? weights[t * topk + j] : 1.0f;
        float v[N];
        part.load(y + (int64_t)p * ld_y, v);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = fmaf(w, v[e], acc[e]);
    }
    part.store(out + t * ld_out, acc);
}

// ------------------------------------------------------ combine's gradient
// dy[pos[t, j]] = w[t, j] dout[t] and dw[t, j] = <dout[t], y[pos[t, j]]>: both
// need dout's row, so one kernel makes both.  G threads per token read it
// once per kBatch choices, with the choices' rows of y requested together,
// write the scaled copies and keep the dot products in registers; a butterfly
// over the warp that halves the number of sums at each step, then one
// addition per warp in shared memory, joins them in an order that depends on
// nothing but the sizes and the layout.  Bound by DRAM: fp32 y, BF16 dout and
// dy 181 us, 7.0 TB/s (106 % of measured; one choice after the other 245);
// 8192 x 2 rows of 8192 BF16 100 us (101 %); 8192 x 4 rows of 1001 BF16 46 us
// (48 %), of 1002 44 us (51 %).  One token a CTA: with two (256 threads) 188,
// 102 and 58 us.
constexpr int kBatch = 4, kBwdThreads = 128;

// y's elements of one part: raw in the whole layout, else as fp32.
template <class Ty, int L, int N>
struct Held {
    std::conditional_t<L == kWhole, Raw<Ty, N>, float[N]> v;
    __device__ __forceinline__ void load(const Part<L, N> &part, const Ty *row) {
        if constexpr (L == kWhole) v.load(row + part.col);
        else part.load(row, v);
    }
};

template <class Td, class Ty, class To, int L, int N, uint32_t G>
__global__ void __launch_bounds__(kBwdThreads) k_moe_combine_bwd(
    const Td *dout, int64_t ld_dout, const Ty *y, int64_t ld_y, const int32_t *pos, const float *weights,
    const int64_t *routed_at, To *__restrict__ dy, int64_t ld_dy, float *__restrict__ dw, int topk, uint32_t hidden,
    uint32_t parts, uint32_t tokens) {
    __shared__ float sums[kBwdThreads / 32][kBatch];
    const uint32_t zero = begin_in_order();
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x / 32;
    const uint32_t mine = threadIdx.x / G, in_group = threadIdx.x % G;
    const uint32_t t = blockIdx.x * (kBwdThreads / G) + mine + zero;
    const bool live = t < tokens;
    const int32_t routed = (int32_t)routed_at[zero];
    for (int j0 = 0; j0 < topk; j0 += kBatch) {
        int32_t p[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const bool in = live && j0 + j < topk;
            p[j] = in ? pos[(int64_t)t * topk + j0 + j] : -1;
            w[j] = in && p[j] < routed ? weights[(int64_t)t * topk + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        if (live)
            for (uint32_t u = L == kWhole ? in_group : in_group / 32; u < parts; u += L == kWhole ? G : G / 32) {
                const Part<L, N> part(u, hidden);
                Held<Td, L, N> d;
                Held<Ty, L, N> v[kBatch];
                d.load(part, dout + (int64_t)t * ld_dout);
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (p[j] >= 0 && p[j] < routed) v[j].load(part, y + (int64_t)p[j] * ld_y);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (p[j] < 0) continue;
                    float o[N] = {};
                    if (p[j] < routed) {
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            o[e] = w[j] * d.v[e];
                            dot[j] = fmaf(d.v[e], v[j].v[e], dot[j]);
                        }
                    }
                    part.store(dy + (int64_t)p[j] * ld_dy, o);
                }
            }
        // kBatch = 4 sums over 32 lanes: two steps that halve their number,
        // three that add; lanes 0, 8, 16, 24 hold sums 0, 1, 2, 3
        const bool h16 = lane & 16u, h8 = lane & 8u;
        const float a = (h16 ? dot[2] : dot[0]) + __shfl_xor_sync(0xFFFFFFFFu, h16 ? dot[0] : dot[2], 16);
        const float b = (h16 ? dot[3] : dot[1]) + __shfl_xor_sync(0xFFFFFFFFu, h16 ? dot[1] : dot[3], 16);
        float s = (h8 ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, h8 ? a : b, 8);
#pragma unroll
        for (int m = 4; m; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
        const int k = (int)(lane >> 3);
        if (G > 32) {
            if ((lane & 7u) == 0) sums[warp][k] = s;
            __syncthreads();
        }
        if (live && in_group < 32 && (lane & 7u) == 0 && j0 + k < topk) {
#pragma unroll
            for (uint32_t o = 1; o < G / 32; ++o) s += sums[warp + o][k];
            dw[(int64_t)t * topk + j0 + k] = s;
        }
        if (G > 32) __syncthreads();
    }
}

// CTAs of the sort's cluster: the steps between the passes cost 1 us more in
// several, the passes 0.7 us per 1024 slots of a CTA.  Measured over 64
// experts (1 / 8 / 16 CTAs): 512 slots 2.3 / 3.5 / 3.7 us, 2048 slots 4.3 /
// 4.2 / 4.5, 8192 slots 8.3 / 4.4 / 4.5, 98304 slots 71 / 13 / 9.0.
int sort_ctas(uint32_t n) { return n <= 1024 ? 1 : n <= 8192 ? 8 : kMaxSortCtas; }

inline uint64_t ctas(uint64_t work, int threads = kThreads) { return (work + threads - 1) / threads; }

template <class Unit, int N>
cudaError_t dispatch(const void *x, int64_t ldx, void *xs, int64_t ldxs, int64_t row_bytes, const MoePlan &m,
                     cudaStream_t s) {
    const int64_t size = sizeof(Unit);
    const uint32_t width = (uint32_t)(row_bytes / size), units = N > 1 ? parts_of(kSingles, N, width) : width;
    const uint64_t work = (uint64_t)m.tokens * units;
    return launch_in_order(k_moe_dispatch<Unit, N>, ctas(work * (N > 1 ? 32 : 1)), kThreads, s,
                           static_cast<const Unit *>(x), ldx / size, static_cast<Unit *>(xs), ldxs / size, m.pos,
                           m.offsets + m.n_experts, m.topk, width, make_rowdiv(units), work);
}

}  // namespace

cudaError_t launch_moe_sort(const void *ids, int id_bytes, const MoePlan &m, cudaStream_t s) {
    uint32_t n = (uint32_t)(m.tokens * m.topk), E = (uint32_t)m.n_experts;
    int ctas = sort_ctas(n);
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(ctas > 1 ? kSortThreads : 32u * std::max((E + 32u) / 32u, std::min(32u, (n + 31u) / 32u)));
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    auto go = [&](auto *t) {
        using Id = std::remove_pointer_t<decltype(t)>;
        if (ctas > 8) {
            const cudaError_t e =
                cudaFuncSetAttribute(k_moe_sort<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        return cudaLaunchKernelEx(&cfg, k_moe_sort<Id>, static_cast<const Id *>(ids), n, E, m.pos, m.src, m.counts,
                                  m.offsets);
    };
    return id_bytes == 4 ? go(static_cast<int32_t *>(nullptr)) : go(static_cast<int64_t *>(nullptr));
}

cudaError_t launch_moe_dispatch(const void *x, int dtype, int64_t hidden, int64_t ld_x, const MoePlan &m, void *xs,
                                int64_t ld_xs, cudaStream_t s) {
    const int64_t esz = dtype == 0 ? 2 : 4, row = hidden * esz;
    const uint64_t all = (uint64_t)(uintptr_t)x | (uint64_t)(uintptr_t)xs | (uint64_t)(ld_x * esz) |
                         (uint64_t)(ld_xs * esz) | (uint64_t)row;
    if (all % 16 == 0) return dispatch<uint4, 1>(x, ld_x * esz, xs, ld_xs * esz, row, m, s);
    if (esz == 4) return dispatch<uint32_t, 8>(x, ld_x * esz, xs, ld_xs * esz, row, m, s);
    return dispatch<uint16_t, 8>(x, ld_x * esz, xs, ld_xs * esz, row, m, s);
}

cudaError_t launch_moe_combine(const void *y, int y_dtype, int64_t hidden, int64_t ld_y, const MoePlan &m,
                               const float *weights, void *out, int out_dtype, int64_t ld_out, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    auto go = [&](auto *yp, auto *op, auto layout, auto elems) {
        constexpr int L = decltype(layout)::value, N = decltype(elems)::value;
        const uint32_t parts = parts_of(L, N, hidden);
        const uint64_t work = (uint64_t)m.tokens * parts;
        using Ty = Elem<decltype(yp)>;
        using To = Elem<decltype(op)>;
        e = launch_in_order(k_moe_combine<Ty, To, L, N>, ctas(threads_of(L, work), kCombineThreads<N>),
                            kCombineThreads<N>, s,
                            static_cast<const Ty *>(y), ld_y, m.pos, weights, m.offsets + m.n_experts,
                            static_cast<To *>(out), ld_out, m.topk, hidden, make_rowdiv(parts), work);
    };
    const auto by = [&](int n) {
        return hidden % n == 0 && rows_by(y, ld_y, type_size(y_dtype), n) &&
               rows_by(out, ld_out, type_size(out_dtype), n);
    };
    by_type(y_dtype, [&](auto *yp) {
        using Ty = Elem<decltype(yp)>;
        by_type(out_dtype, [&](auto *op) {
            if constexpr (sizeof(Ty) == 2)   // 32 bytes of y a thread where rows allow it
                if (by(16)) return go(yp, op, Int<kWhole>(), Int<16>());
            if (by(8)) go(yp, op, Int<kWhole>(), Int<8>());
            else if (by(2)) go(yp, op, Int<kPairs>(), Int<8>());
            else go(yp, op, Int<kSingles>(), Int<8>());
        });
    });
    return e;
}

cudaError_t launch_moe_combine_bwd(const void *dout, int dout_dtype, int64_t ld_dout, const void *y, int y_dtype,
                                   int64_t ld_y, int64_t hidden, const MoePlan &m, const float *weights, void *dy,
                                   int dy_dtype, int64_t ld_dy, float *dw, cudaStream_t s) {
    const auto by = [&](int n) {
        return hidden % n == 0 && rows_by(dout, ld_dout, type_size(dout_dtype), n) &&
               rows_by(y, ld_y, type_size(y_dtype), n) && rows_by(dy, ld_dy, type_size(dy_dtype), n);
    };
    cudaError_t e = cudaSuccess;
    by_type(dout_dtype, [&](auto *dp) {
        using Td = Elem<decltype(dp)>;
        by_type(y_dtype, [&](auto *yp) {
            using Ty = Elem<decltype(yp)>;
            by_type(dy_dtype, [&](auto *op) {
                using To = Elem<decltype(op)>;
                auto go = [&](auto layout, auto elems) {
                    constexpr int L = decltype(layout)::value, N = decltype(elems)::value;
                    const uint32_t parts = parts_of(L, N, hidden);
                    auto with = [&](auto group) {
                        constexpr uint32_t G = decltype(group)::value;
                        e = launch_in_order(
                            k_moe_combine_bwd<Td, Ty, To, L, N, G>, ctas((uint64_t)m.tokens * G, kBwdThreads),
                            kBwdThreads, s, static_cast<const Td *>(dout), ld_dout, static_cast<const Ty *>(y), ld_y,
                            m.pos, weights, m.offsets + m.n_experts, static_cast<To *>(dy), ld_dy, dw, m.topk, hidden,
                            parts, m.tokens);
                    };
                    // 128 threads a token unless most would idle.  Measured
                    // (32 / 64 / 128): 16384 tokens x 6 of 2048 194 / 187 /
                    // 182 us, 128 tokens 8.5 / 5.2 / 3.8 us, 8192 x 4 of
                    // 1001 BF16 52 / 48 / 46 us.  The count is a constant of
                    // the kernel, which lets its loop over the row be
                    // unrolled (with a variable the last takes 59 us).
                    if (threads_of(L, parts) <= 64) with(Int<32>());
                    else with(Int<128>());
                };
                if constexpr (sizeof(Ty) == 2)   // 32 bytes of y a thread where rows allow it
                    if (by(16)) return go(Int<kWhole>(), Int<16>());
                if (by(8)) go(Int<kWhole>(), Int<8>());
                else if (by(2)) go(Int<kPairs>(), Int<8>());
                else go(Int<kSingles>(), Int<8>());
            });
        });
    });
    return e;
}

}  // namespace ufp4
