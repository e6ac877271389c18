// evict.cu -- eviction from a paged cache by accumulated attention weight: which
// tokens every KV head of a sequence keeps, and their move to blocks of their own.
//
// Of the c tokens of a context n = min(c, keep) stay: the last l = min(keep_last, n),
// the first f = min(keep_first, n - l), and of those between the n - f - l of largest
// weight, the lower index first where weights are equal (NaN counts as -inf).
//   * select: a cluster of CTAs per (sequence, KV head), 8 tokens a thread, weights
//     as integers of the same order.  Four rounds of 8 bits find the smallest weight
//     kept: a histogram per CTA, added up over the cluster through distributed
//     shared memory.  A scan over threads and CTAs then places what is kept, in
//     order.  Contexts above 8 x 4,096 tokens are read again in every round (from L2).
//   * move: a warp per destination block and KV head; its rows are gathered 16 bytes
//     a lane.  In a scaled cache the block's new scale is the largest of the blocks
//     its tokens come from, codes of smaller ones become E4M3(code * old / new).
// Bound by latency for short contexts, by the gather and its writes for long ones.
// Measured (8 heads, D 128, scaled cache): 64 contexts of 1,500..2,600 tokens to 2,048
// 99 us: select 19, move 80, 93 % of a copy's rate; 4 of 16,384..32,768 to 2,048 26 us:
// 16 and 9.  Three rounds of 11 bits, with larger histograms over the cluster: select 57.
#include <cuda_runtime.h>

#include "context_internal.h"
#include "pkv_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 512;                  // at most
constexpr int kFewThreads = 256;               // at least: one for each bin
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;                        // tokens a thread holds
constexpr int kTile = kThreads * kPer;
constexpr int kMaxCluster = 8;
constexpr int kMoveWarps = 8;

// Unsigned integers in the order of the weights.
__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w)
        w = -__builtin_huge_valf();
    const uint32_t u = __float_as_uint(w + 0.f);       // (-0 is 0)
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

// A word of CTA `rank`'s shared memory, at this CTA's address of it.
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, uint32_t rank)
{
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// What a sequence keeps; n < 0: its length or its budget cannot be used.
struct Budget {
    int ctx, n, first, last;
};

__device__ __forceinline__ Budget budget_of(const EvictParams& p, int s)
{
    Budget b;
    b.ctx = __ldg(p.context_lens + s);
    const int keep = __ldg(p.keep_lens + s);
    b.n = min(b.ctx, keep);
    if (b.ctx < 0 || b.ctx > p.max_context_len ||
        (b.ctx + p.block_size - 1) / p.block_size > p.max_blocks_per_seq || keep < 0 ||
        keep > p.max_keep_len)
        b.n = -1;
    b.last = min(p.keep_last, b.n);
    b.first = min(p.keep_first, b.n - b.last);
    return b;
}

// ONE: the CTA's part of the row is one tile, whose weights stay in registers.
template <bool ONE>
__global__ void __launch_bounds__(kThreads, ONE ? 3 : 1) evict_select_kernel(const EvictParams p)
{
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t sums[kWarps];
    __shared__ uint32_t digit, above, inside;  // of the round: the bin, what lies above it and in it
    __shared__ uint32_t counts[2];             // above, equal to the smallest kept weight: this CTA's

    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int lane = tid & 31;
    const int warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int64_t item = blockIdx.x / size;
    const int s = (int)(item / p.num_kv_heads);
    const int h = (int)(item - (int64_t)s * p.num_kv_heads);
    pdl_wait_primary();
    pdl_launch_dependents();
    const Budget b = budget_of(p, s);
    if (h == 0 && rank == 0 && tid == 0) {
        p.lens_out[s] = max(b.n, 0);
        if (b.n < 0)
            flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
    }
    if (b.n < 0)
        return;                                // (the whole cluster)
    const float* row = p.weights + s * p.weights_seq + h * p.weights_head;
    float* out = p.weights_out + s * p.weights_out_seq + h * p.weights_out_head;
    int32_t* kept = p.kept + item * p.most;
    for (int64_t i = (int64_t)b.n + rank * threads + tid; i < p.weights_out_len; i += size * threads)
        out[i] = 0.f;

    // this CTA's tokens [t0, t1); those between the first and the last kept ones
    // compete
    const int part = ((b.ctx + (int)size - 1) / (int)size + kPer - 1) / kPer * kPer;
    const int t0 = min(b.ctx, (int)rank * part), t1 = min(b.ctx, t0 + part);
    const int c0 = b.first, c1 = b.ctx - b.last;
    const bool wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    auto load = [&](int base, uint32_t(&key)[kPer]) {
        const int i0 = base + tid * kPer;
        float w[kPer];
        if (wide && i0 + kPer <= t1) {         // (i0 is a multiple of kPer)
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + i0));
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + i0) + 1);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                w[e] = i0 + e < t1 ? __ldg(row + i0 + e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            key[e] = order_key(w[e]);
    };
    auto competes = [&](int i) { return i >= c0 && i < c1 && i < t1; };

    uint32_t key[kPer];
    // ONE: the thread's tokens (bit e: token e) that may still be on the edge, and those
    // above it
    uint32_t open = 0, won = 0;
    if constexpr (ONE) {
        load(t0, key);
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            open |= (competes(t0 + tid * kPer + e) ? 1u : 0u) << e;
    }
    // the kept weights are those with (key & mask) > edge, and `rest` of those equal
    uint32_t mask = 0, edge = 0;
    uint32_t rest = (uint32_t)(b.n - b.first - b.last);
    const bool choose = rest > 0 && b.n < b.ctx;
    if (!choose)
        rest = b.n < b.ctx ? 0u : 0xffffffffu;         // none, or all, of the equal (mask 0: all are)
    for (int i = tid; i < 4 * 256; i += threads)
        (&hist[0][0])[i] = 0;
    if (tid < kWarps)
        sums[tid] = 0;                         // (of the warps that are not there, too)
    __syncthreads();
    for (int round = 0; choose && round < 4; ++round) {
        const int shift = 24 - 8 * round;
        if constexpr (ONE) {
            if (open != 0)
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if ((open >> e) & 1u)
                        atomicAdd(&hist[round][(key[e] >> shift) & 255u], 1u);
        } else {
            for (int base = t0; base < t1; base += kTile) {
                load(base, key);
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (competes(base + tid * kPer + e) && (key[e] & mask) == edge)
                        atomicAdd(&hist[round][(key[e] >> shift) & 255u], 1u);
            }
        }
        if (size > 1)
            cluster_sync();
        else
            __syncthreads();
        // bin 255 - tid: how many lie in it and above it
        uint32_t mine = 0, incl = 0;
        if (tid < 256) {
            if (size == 1) {
                mine = hist[round][255 - tid];
            } else {
                uint32_t v[kMaxCluster];       // (all on their way at once)
#pragma unroll
                for (uint32_t r = 0; r < kMaxCluster; ++r)
                    v[r] = r < size ? peer_word(&hist[round][255 - tid], r) : 0u;
#pragma unroll
                for (uint32_t r = 0; r < kMaxCluster; ++r)
                    mine += v[r];
            }
            incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += u;
            }
            if (lane == 31)
                sums[warp] = incl;
        }
        __syncthreads();
        if (tid < 256) {
            for (int w = 0; w < warp; ++w)
                incl += sums[w];
            if (incl >= rest && incl - mine < rest) {
                digit = 255 - tid;
                above = incl - mine;
                inside = mine;
            }
        }
        __syncthreads();
        edge |= digit << shift;
        mask |= 255u << shift;
        rest -= above;
        if (ONE && open != 0) {
            const uint32_t d = digit;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const uint32_t x = (key[e] >> shift) & 255u;
                const uint32_t bit = open & (1u << e);
                won |= x > d ? bit : 0u;
                open ^= x != d ? bit : 0u;
            }
        }
        if (inside == rest)                    // all that share these bits stay
            break;
    }

    // how many tokens of the CTA lie above, and on, the edge
    auto classify = [&](int base, uint32_t& packed, uint32_t& above_bits, uint32_t& equal_bits) {
        above_bits = won, equal_bits = open;
        if constexpr (!ONE) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (competes(base + tid * kPer + e)) {
                    const uint32_t k = key[e] & mask;
                    above_bits |= (k > edge ? 1u : 0u) << e;
                    equal_bits |= (k == edge ? 1u : 0u) << e;
                }
        }
        packed = __popc(above_bits) | (__popc(equal_bits) << 16);      // (a tile: 4,096 at most)
    };
    // exclusive sum over the CTA's threads; `total`: of all
    auto scan = [&](uint32_t v, uint32_t& total) {
        uint32_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        __syncthreads();
        if (lane == 31)
            sums[warp] = incl;
        __syncthreads();
        uint32_t before = incl - v;
        total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t x = sums[w];
            before += w < warp ? x : 0u;
            total += x;
        }
        return before;
    };
    uint32_t n_above = 0, n_equal = 0;         // of the cluster's CTAs before this one
    if (size > 1) {
        uint32_t a = 0, q = 0;
        for (int base = t0; base < t1; base += kTile) {
            if constexpr (!ONE)
                load(base, key);
            uint32_t packed, ab, eb, total;
            classify(base, packed, ab, eb);
            scan(packed, total);
            a += total & 0xffffu;
            q += total >> 16;
        }
        if (tid == 0)
            counts[0] = a, counts[1] = q;
        cluster_sync();
        uint32_t va[kMaxCluster], vq[kMaxCluster];
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            va[r] = r < rank ? peer_word(&counts[0], r) : 0u;
            vq[r] = r < rank ? peer_word(&counts[1], r) : 0u;
        }
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r)
            n_above += va[r], n_equal += vq[r];
        // (nobody leaves while others may read its shared memory: the wait is at the end)
        cluster_arrive();
    }
    for (int base = t0; base < t1; base += kTile) {
        if constexpr (!ONE)
            load(base, key);
        uint32_t packed, ab, eb, total;
        classify(base, packed, ab, eb);
        const uint32_t before = scan(packed, total);
        uint32_t above_so_far = n_above + (before & 0xffffu);
        uint32_t equal_so_far = n_equal + (before >> 16);
        const int i0 = base + tid * kPer;
        if (i0 < t1) {
            float w[kPer];                     // (all on their way at once)
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                w[e] = __ldg(row + min(i0 + e, t1 - 1));
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int i = i0 + e;
                int pos = -1;
                if (i < c0) {
                    pos = i;
                } else if (i >= c1) {
                    pos = b.n - (b.ctx - i);
                } else {
                    const bool is_above = (ab >> e) & 1u, is_equal = (eb >> e) & 1u;
                    if (is_above || (is_equal && equal_so_far < rest))
                        pos = c0 + (int)(above_so_far + min(equal_so_far, rest));
                    above_so_far += is_above;
                    equal_so_far += is_equal;
                }
                if (pos >= 0 && i < t1) {
                    kept[pos] = i;
                    out[pos] = w[e];
                }
            }
        }
        n_above += total & 0xffffu;
        n_equal += total >> 16;
    }
    if (size > 1)
        cluster_wait();
}

// Sixteen E4M3 codes times f.
__device__ __forceinline__ uint4 rescale16(const uint4& v, float f)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(w[i], lo, hi);
        const float2 a = f16x2_to_float2(lo), b = f16x2_to_float2(hi);
        r[i] = pack2(e4m3x2_satfinite(a.x * f, a.y * f), e4m3x2_satfinite(b.x * f, b.y * f));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// RB: bytes of a token's row of one head.
template <int RB, int BS, bool SCALED>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictParams p)
{
    constexpr int LPR = RB / 16;               // lanes to a row
    constexpr int RPA = 32 / LPR;              // rows to a warp's access
    constexpr int NV = BS / RPA;
    const int lane = threadIdx.x & 31;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    const int64_t item = blockIdx.x % items;
    const int blk = (int)(blockIdx.x / items) * kMoveWarps + (threadIdx.x >> 5);
    const int s = (int)(item / p.num_kv_heads);
    const int h = (int)(item - (int64_t)s * p.num_kv_heads);
    pdl_wait_primary();
    pdl_launch_dependents();
    const int rows = min(BS, __ldcg(p.lens_out + s) - blk * BS);
    if (rows <= 0)
        return;
    const int dst = __ldg(p.dst_tables + (int64_t)s * p.max_dst_blocks + blk);
    if (dst < 0 || (int64_t)dst >= p.num_blocks) {
        if (lane == 0)
            flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    // lane r: where row r comes from
    int src = -1, slot = 0;
    float2 old = make_float2(0.f, 0.f);
    if (lane < rows) {
        const int t = __ldcg(p.kept + item * p.most + blk * BS + lane);
        src = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + t / BS);
        slot = t % BS;
        if (src < 0 || (int64_t)src >= p.num_blocks) {
            flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);
            src = -1;
        } else if constexpr (SCALED) {
            old = __ldg(reinterpret_cast<const float2*>(p.scales) + (int64_t)src * p.num_kv_heads + h);
        }
    }
    float2 ratio = make_float2(1.f, 1.f);
    if constexpr (SCALED) {
        // (positive floats order as their bits; a bad block counts as 0)
        const float nk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(old.x)));
        const float nv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(old.y)));
        if (lane == 0 && __float_as_uint(nk) != 0u)
            reinterpret_cast<float2*>(p.scales)[(int64_t)dst * p.num_kv_heads + h] = make_float2(nk, nv);
        ratio = make_float2(old.x == nk ? 1.f : old.x / nk, old.y == nv ? 1.f : old.y / nv);
    }
    const int64_t tile = (int64_t)BS * RB;
    const int64_t to = ((int64_t)dst * p.num_kv_heads + h) * tile;
    const int c = lane % LPR;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const char* cache = reinterpret_cast<const char*>(which ? p.v_cache : p.k_cache);
        uint4 v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int r = i * RPA + lane / LPR;
            const int b = __shfl_sync(0xffffffffu, src, r);
            const int o = __shfl_sync(0xffffffffu, slot, r);
            v[i] = make_uint4(0, 0, 0, 0);
            if (b >= 0)
                v[i] = ld_stream(cache + ((int64_t)b * p.num_kv_heads + h) * tile + o * RB + c * 16);
        }
        char* d = reinterpret_cast<char*>(which ? p.v_cache : p.k_cache) + to;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int r = i * RPA + lane / LPR;
            const bool ok = __shfl_sync(0xffffffffu, src, r) >= 0;
            if constexpr (SCALED) {
                const float f = __shfl_sync(0xffffffffu, which ? ratio.y : ratio.x, r);
                if (f != 1.f)
                    v[i] = rescale16(v[i], f);
            }
            if (ok)
                st_v4(d + r * RB + c * 16, v[i]);
        }
    }
}

template <class K>
cudaError_t launch(K kern, int64_t ctas, int threads, int cluster, cudaStream_t stream,
                   const EvictParams& p)
{
    if (ctas > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int RB, bool SCALED>
cudaError_t move(const EvictParams& p, cudaStream_t stream)
{
    const int64_t blocks = ((int64_t)p.most + p.block_size - 1) / p.block_size;
    const int64_t ctas = (blocks + kMoveWarps - 1) / kMoveWarps * p.num_seqs * p.num_kv_heads;
    switch (p.block_size) {
    case 8: return launch(evict_move_kernel<RB, 8, SCALED>, ctas, kMoveWarps * 32, 1, stream, p);
    case 16: return launch(evict_move_kernel<RB, 16, SCALED>, ctas, kMoveWarps * 32, 1, stream, p);
    case 32: return launch(evict_move_kernel<RB, 32, SCALED>, ctas, kMoveWarps * 32, 1, stream, p);
    default: return cudaErrorNotSupported;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream)
{
    // a row's weights stay in the registers of up to eight CTAs
    int cluster = 1;
    while (cluster < kMaxCluster && (int64_t)cluster * kTile < p.max_context_len)
        cluster *= 2;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    // ONE: no more threads than tokens ask for (512 rows of 2,600 tokens, select and move:
    // 99.7 us with 352 threads a row, which all fit at once, 100.7 with 512)
    const int64_t part = ((int64_t)p.max_context_len + cluster - 1) / cluster;
    const int64_t warps = (part + 32 * kPer - 1) / (32 * kPer);
    int threads = warps < kWarps ? 32 * (int)warps : kThreads;
    if (threads < kFewThreads)
        threads = kFewThreads;
    cudaError_t e = (int64_t)cluster * kTile >= p.max_context_len
                        ? launch(evict_select_kernel<true>, items * cluster, threads, cluster, stream, p)
                        : launch(evict_select_kernel<false>, items * cluster, kThreads, cluster, stream, p);
    if (e != cudaSuccess || p.most == 0)
        return e;
    const bool scaled = p.scales != nullptr;
    switch (p.row_bytes) {
    case 64: return scaled ? move<64, true>(p, stream) : move<64, false>(p, stream);
    case 128: return scaled ? move<128, true>(p, stream) : move<128, false>(p, stream);
    case 256: return scaled ? cudaErrorNotSupported : move<256, false>(p, stream);
    default: return cudaErrorNotSupported;
    }
}

}  // namespace pkv
