// attention_weights.cu -- the attention weights of each sequence's last rows over its
// paged context, summed over rows and the query heads of a KV head, on the
// 5th-generation tensor cores.
//
// Row j of the last m rows of a sequence stands at position p = c - m + j and sees
// tokens t <= p.  With x = scale q_jh . k_t,
//   weights[t] += sum_{j, h} exp(x_jh(t) - max x_jh) / sum_t exp(x_jh(t) - max x_jh).
// A token's sum needs every row's maximum and sum first, so there are two passes
// over K, and one small kernel in front:
//   * tiles: q as operand tiles of 128 (row, head) rows, swizzled as the tensor core
//     reads them, so that the passes fetch a tile panel by panel.  Over an E4M3
//     cache the products are fp16, in which every code is exact; bf16 rows become
//     fp16 times a power of two.  The sign of the scale goes into q, its size and
//     the power into a factor per row.
//   * sums: S = Q K^T, a thread per row of q.  The sum of 2^(x - m) is taken against
//     any score m of the row: fp32 holds sums up to 2^100 as well as those near 1, so
//     only a sum beyond that makes the tile be summed again against its maximum.
//     What is kept is the logarithm, lse = m + log2 sum.
//   * totals: S^T = K Q^T, the operands swapped, a thread per key: 2^(x - lse), added
//     up over the rows in fp32, then to the key's total.  One thread has one key: the
//     same inputs give the same bits.
// A scale per block multiplies scores in fp32, wherever it is.
//
// The key tiles (128 keys) of every (sequence, KV head), laid end to end, go to one
// CTA an SM in equal shares; a share's part of one item is a segment.  Two q tiles
// at a time stay in shared memory while a segment's keys stream through a ring
// (more rows than 256: the keys stream again, from L2).  Warps 0-15: four groups of
// softmax threads, a 128 x 128 block of scores in tensor memory each; warp 16 asks
// for keys and q by bulk and tensor copies; one thread of warp 17 issues the
// products; warps 18-21 (E4M3 caches) turn codes into fp16 operands.  Where a
// segment is not its whole item, its rows' log sums go to scratch, and the CTA that
// finishes the item last merges them.  Every wait is bounded.
//
// Bound by the chain product - softmax - product through tensor memory, of which
// two sets of 128 x 256 scores fit: ~2,600 cycles a key tile for 1,024 of products and
// 1,024 of exponentials (32,768 at 32 a cycle; both pipes are 36-38 % busy).
// Measured: 32 rows of 4 prompts after 16,384..32,768 tokens (64 heads over 8, D
// 128) 165 us; 64 rows of 8 prompts of 512..2,048 (32 heads, bf16 cache) 57 us.  On the
// way: a CTA per run of keys with two groups of softmax warps 267 us, equal shares
// with codes through registers 315, by bulk copies 223, both q tiles' groups side by
// side 190, sums against any score and log sums 175, 256 rows in one product 166.
// Block ids asked for four tiles ahead instead of two: 169 and 55.6.  Few rows (5 of 6
// prompts of 10,594..21,189 tokens, 16 heads each its own) take 160 us at 32 tokens a
// block and 220 at 8: ~1,700 and ~2,400 cycles a tile, one bulk copy for each block of
// it (two teams of converting warps changed nothing).  The merge fetches 8 log sums of a
// row at once: one by one the sums pass over 5 prompts of 8,765..17,530 tokens of one head
// took 31 us instead of 20.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "context_internal.h"
#include "pkv_common.cuh"
#include "tc_common.cuh"

namespace pkv {
namespace {

using namespace tc;

constexpr int kRows = 128;             // rows of an operand tile
constexpr int kGroups = 4;             // of four softmax warps
constexpr int kSoftmax = 128 * kGroups;
constexpr int kFetchWarp = 4 * kGroups;
constexpr int kMmaWarp = kFetchWarp + 1;
constexpr int kConvWarp = kMmaWarp + 1;
constexpr int kConvWarps = 4;

template <bool E8>
constexpr int threads_of()
{
    return 32 * (E8 ? kConvWarp + kConvWarps : kConvWarp);
}
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kScaleRing = 16;
constexpr float kRaise = 8.f;          // log2: how far a score may pass the running maximum
constexpr float kMuch = 1.2676506e30f; // 2^100: sums up to here need no other reference
constexpr float kMost = 3.4028235e38f; // the largest float
constexpr int kInfo = 2 * kRows + 4;   // floats of a q tile: its rows' factors, -log2 of their sums, a flag
constexpr int kAtOnce = 8;             // log sums of a row that are fetched together
constexpr float kTiny = 1e-38f;        // a factor of 0 would turn a masked -inf into NaN

// One sequence's rows.
struct Span {
    int ctx;           // tokens of the context (0: nothing to do)
    int rows;          // (row, head) rows: the last tokens' query heads of a KV head
    int first_pos;     // position of the first of those tokens
    int64_t first_row; // its row of q
};

__device__ __forceinline__ Span span_of(const WeightsParams& p, int s, bool flag)
{
    Span sp{};
    const int cu0 = __ldg(p.cu_seqlens_q + s);
    const int cu1 = __ldg(p.cu_seqlens_q + s + 1);
    const int ctx = __ldg(p.context_lens + s);
    if (cu0 < 0 || cu1 < cu0 || cu1 > p.total_q || ctx < cu1 - cu0 || ctx > p.max_context_len ||
        (ctx + p.block_size - 1) / p.block_size > p.max_blocks_per_seq) {
        if (flag)
            flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
        return sp;
    }
    const int m = min(cu1 - cu0, p.window);
    if (m == 0)
        return sp;
    sp.ctx = ctx;
    sp.rows = m * p.group;
    sp.first_pos = ctx - m;
    sp.first_row = cu1 - m;
    return sp;
}

// ------------------------------------------------------------------ q tiles

constexpr int kTileThreads = 512;
constexpr float kSpread = 4096.f;      // rows of a tile within it share a power of two

// One CTA = one tile of 128 rows; D / 8 lanes to a row.  QT: type of q, CT: of the
// operand.  Where they differ, rows are scaled by a power of two: the one of the tile's
// largest element, if no row's largest is further than kSpread below it, else each
// row's own.  The tile's largest then lies in [2^13, 2^14) and a row's at 2 or above,
// where fp16's step is 2^-24 at least: bf16's 8 bits fit from 2^-18 of the row's largest
// on, smaller elements are off by 2^-26 of it at most.  (Rows with factors of their own:
// 2^-30 and 2^-38.)
template <int QT, int CT, int D>
__global__ void __launch_bounds__(kTileThreads) weights_tiles_kernel(const WeightsParams p)
{
    constexpr int LPR = D / 8;
    constexpr int RPP = kTileThreads / LPR;    // rows at once
    constexpr int N = kRows / RPP;
    __shared__ uint32_t most, least;           // bits of the rows' largest magnitudes (not 0)
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t idx = blockIdx.x;
    const int tile = (int)(idx % p.row_tiles);
    const int64_t item = idx / p.row_tiles;
    const int s = (int)(item / p.num_kv_heads);
    const int g = (int)(item - (int64_t)s * p.num_kv_heads);
    const bool first = tile == 0 && threadIdx.x == 0;
    const Span sp = span_of(p, s, first && g == 0);
    if (first)
        p.finished[item] = 0;
    if (idx == 0 && threadIdx.x == 0)
        *p.failed = 0;
    if (tile * kRows >= sp.rows)
        return;
    const float sign = p.qk_scale_log2 < 0.f ? -1.f : (p.qk_scale_log2 == 0.f ? 0.f : 1.f);
    char* dst = reinterpret_cast<char*>(p.q_tiles) + idx * (kRows * D * 2);
    const int c = threadIdx.x % LPR;
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int rr = tile * kRows + i * RPP + (int)threadIdx.x / LPR;
        const int j = rr / p.group;
        v[i] = make_uint4(0, 0, 0, 0);
        if (rr < sp.rows)
            v[i] = ld_ro(reinterpret_cast<const uint16_t*>(p.q) +
                         ((sp.first_row + j) * p.num_heads + g * p.group + (rr - j * p.group)) * D + c * 8);
    }
    float up[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        up[i] = 1.f;
    bool even = true;
    if constexpr (QT != CT) {
        if (threadIdx.x == 0)
            most = 0u, least = 0xffffffffu;
        __syncthreads();
        float mx[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            mx[i] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<QT>(w[e]);
                mx[i] = fmaxf(mx[i], fmaxf(fabsf(f.x), fabsf(f.y)));
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
            if (c == 0 && mx[i] > 0.f) {
                atomicMax(&most, __float_as_uint(mx[i]));
                atomicMin(&least, __float_as_uint(mx[i]));
            }
        }
        __syncthreads();
        // (an infinity among them: each row for itself)
        const float top = __uint_as_float(most);
        even = top == 0.f || (top < __builtin_huge_valf() && __uint_as_float(least) * kSpread >= top);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float m = even ? top : mx[i];
            // 2^13 / 2^floor(log2 m), kept where it and its inverse are normal
            if (m > 0.f && m < __builtin_huge_valf())
                up[i] = __uint_as_float((uint32_t)min(max(267 - (int)(__float_as_uint(m) >> 23), 7), 247) << 23);
        }
    }
    float* info = p.row_info + idx * kInfo;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = i * RPP + (int)threadIdx.x / LPR;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QT>(w[e]);
            h[e] = pack_rn<CT>(f.x * (up[i] * sign), f.y * (up[i] * sign));
        }
        *reinterpret_cast<uint4*>(dst + panel_off(r, c, kRows)) = make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0)
            info[r] = fabsf(p.qk_scale_log2) * (1.f / up[i]);
    }
    if (threadIdx.x == 0)
        info[2 * kRows] = even ? 1.f : 0.f;    // all rows have the factor of row 0
}

// ------------------------------------------------------------------ the passes

template <int D, bool E8>
struct Layout {
    static constexpr int TB = D * kRows * 2;           // an operand tile
    static constexpr int RB = D * kRows;               // a tile's codes
    static constexpr int ST = E8 ? 3 : 4;              // key tiles of the ring
    static constexpr int RAW = E8 ? 3 : 0;             // tiles of codes
    static constexpr int PB = kRows * 128;             // a panel of an operand tile
    static constexpr int q = 0;                        // two q tiles, panel by panel
    static constexpr int ring = 2 * TB;
    static constexpr int raw = ring + ST * TB;
    static constexpr int bytes = raw + RAW * RB;
    static constexpr int alloc = bytes + 1024;         // room to align the base
};

template <int ST>
struct Bars {
    uint64_t q_full[2];          // the copies of a q tile and its rows' numbers
    uint64_t q_free[2];          // commit, and one arrival per softmax warp
    uint64_t s_full[kGroups];    // commit: scores of the group are in its buffer
    uint64_t s_free[kGroups];    // one arrival per warp of the group: they have been read
    uint64_t full[ST];           // the copies of a key tile, or one arrival per converting warp
    uint64_t empty[ST];          // commit: no longer read
    uint64_t raw_full[3];        // the copies of a tile's codes
    uint64_t raw_free[3];        // one arrival per converting warp: they have been read
    uint64_t drain;              // commit: every product
};

// A share's walk: the segment it is at, then the next.  Every role walks for itself.
struct Walk {
    int64_t left;                // key tiles behind the segment
    int s, h;                    // the segment's item
    int j0, nk, n;               // its key tiles [j0, j0 + nk) of n
    int ctx, rows, pairs;        // tokens; (row, head) rows; pairs of q tiles
    int first_pos;               // position of the first row's token
};

// Tables of the batch's sequences in shared memory: key tiles before a sequence (of
// one KV head), tokens, rows' tokens.
struct Batch {
    const int* first;
    const int* ctx;
    const int* tokens;
    int group, heads;

    __device__ __forceinline__ void enter(Walk& w) const
    {
        w.n = first[w.s + 1] - first[w.s];
        w.nk = (int)min((int64_t)(w.n - w.j0), w.left);
        w.left -= w.nk;
        w.ctx = ctx[w.s];
        w.rows = tokens[w.s] * group;
        w.pairs = (w.rows + 2 * kRows - 1) / (2 * kRows);
        w.first_pos = w.ctx - tokens[w.s];
    }
    // false at the end of the share
    __device__ __forceinline__ bool next(Walk& w) const
    {
        if (w.left <= 0)
            return false;
        w.j0 = 0;
        if (++w.h == heads) {
            w.h = 0;
            do
                ++w.s;
            while (first[w.s + 1] == first[w.s]);
        }
        enter(w);
        return true;
    }
};

// q tiles of pair pr of an item.
__device__ __forceinline__ int q_tiles_of(const Walk& w, int pr)
{
    return min(2, (w.rows + kRows - 1) / kRows - 2 * pr);
}

__device__ __forceinline__ bool aborted(const int* flag)
{
    return *reinterpret_cast<const volatile int*>(flag) != 0;
}

// What every wait of a CTA shares: its flag (some role has given up), the caller's
// error word, and the polls of a wait.  Below kSpin (a test's setting) a poll is one
// look that does not suspend.
struct Waits {
    int* flag;
    int32_t* dev_err;
    uint32_t tries;

    __device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) const
    {
        return tries < kSpin ? test_wait(bar, parity) : try_wait(bar, parity);
    }
    __device__ __forceinline__ void give_up() const
    {
        *reinterpret_cast<volatile int*>(flag) = 1;
        flag_error(dev_err, PKV_DEVERR_TIMEOUT);
    }
};

// Bounded wait by one thread; gives up early once another role has aborted.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, const Waits& w)
{
    WaitClock clock;
    for (uint32_t i = 0; i < w.tries; ++i) {
        if (w.poll(bar, parity))
            return true;
        if (aborted(w.flag))
            return false;
        if (clock.expired(i))
            break;
    }
    w.give_up();
    return false;
}

// The same by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Waits& w)
{
    bool ok = false;
    WaitClock clock;
    for (uint32_t i = 0; i < w.tries; ++i) {
        if (w.poll(bar, parity)) {
            ok = true;
            break;
        }
        if (aborted(w.flag) || clock.expired(i))
            break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok)
        w.give_up();
    return ok;
}

__device__ __forceinline__ void softmax_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory");
}

// The two groups 2 x and 2 x + 1.
__device__ __forceinline__ void pair_sync(int x)
{
    if (x == 0)
        asm volatile("bar.sync 2, 256;" ::: "memory");
    else
        asm volatile("bar.sync 3, 256;" ::: "memory");
}

// Part (reference m, sum l of 2^(x - m)) as log2 of the sum of 2^x.
__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.f ? kNegInf : m + log2f(l);
}

// log2 of a row's sum, as the second pass takes it: weights of a row without any
// score are 2^(x - inf).
__device__ __forceinline__ void put_row(float* info, int row, float lse)
{
    info[(int64_t)(row / kRows) * kInfo + kRows + row % kRows] = lse == kNegInf ? kNegInf : -lse;
}

__device__ __forceinline__ void st_shared16(uint32_t a, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// The wait for a thread's tensor-memory loads, which `r` depends on.
__device__ __forceinline__ void tmem_wait16(float (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]),
                   "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]),
                   "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}

// f(x, c0) for the columns [c0, c0 + 16) of a thread's lane, c0 < end; the next
// columns are on their way meanwhile.
template <class F>
__device__ __forceinline__ void for_columns(uint32_t taddr, int end, F f)
{
    float xa[16], xb[16];
    tmem_ld16(taddr, reinterpret_cast<uint32_t(&)[16]>(xa));
    tmem_wait16(xa);
#pragma unroll 1
    for (int c0 = 0; c0 < end; c0 += 32) {
        tmem_ld16(taddr + c0 + 16, reinterpret_cast<uint32_t(&)[16]>(xb));
        f(xa, c0);
        tmem_wait16(xb);
        if (c0 + 16 >= end)
            break;
        tmem_ld16(taddr + min(c0 + 32, kRows - 16), reinterpret_cast<uint32_t(&)[16]>(xa));
        f(xb, c0 + 16);
        tmem_wait16(xa);
    }
}

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a)
                 : "memory");
    return r;
}

// Arrive on `bar`, whose phase then waits for `bytes` too.
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// CT: operand type; E8: the cache holds E4M3 codes; TOTALS: the second pass.
template <int CT, bool E8, int D, bool TOTALS>
__global__ void __launch_bounds__(threads_of<E8>(), 1)
    weights_pass_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap k_map)
{
    using L = Layout<D, E8>;
    constexpr int kThreads = threads_of<E8>();
    constexpr int ST = L::ST;
    constexpr int NP = D / 64;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) Bars<ST> bars;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag, is_last;
    __shared__ int sm_first[kWindowSeqs + 1], sm_ctx[kWindowSeqs], sm_tokens[kWindowSeqs];
    __shared__ int sm_sums[kThreads / 32];
    __shared__ __align__(16) float row_info[2][kInfo];       // of the two q tiles
    // K's scale of every 8 keys; softmax warps read a tile's up to RAW + ST + 3 tiles
    // after warp 16 has passed it
    __shared__ float ks_ring[kScaleRing][kRows / 8];
    static_assert(kScaleRing > L::RAW + ST + 4, "ring of the scales");
    __shared__ uint32_t raw_good[3];                   // blocks of a tile of codes that are there
    __shared__ float sums[TOTALS ? 2 : 1][2][TOTALS ? kRows : 1];      // of the second q tile
    __shared__ float parts[TOTALS ? 1 : 2][TOTALS ? 1 : kSoftmax];     // a segment's log sums by group

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const Waits waits{&abort_flag, p.dev_err, !TOTALS && p.wait_tries ? p.wait_tries : kSpin};

    // what the kernel before writes is read behind the wait below; the lengths are older
    const uint32_t sb = (s_addr(smem_raw) + 1023u) & ~1023u;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bar_init(s_addr(&bars.q_full[i]), 1);
            bar_init(s_addr(&bars.q_free[i]), 1 + kSoftmax / 32);
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            bar_init(s_addr(&bars.s_full[i]), 1);
            bar_init(s_addr(&bars.s_free[i]), 4);
        }
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            bar_init(s_addr(&bars.full[i]), E8 ? kConvWarps : 1);
            bar_init(s_addr(&bars.empty[i]), 1);
        }
        for (int i = 0; i < 3; ++i) {
            bar_init(s_addr(&bars.raw_full[i]), 1);
            bar_init(s_addr(&bars.raw_free[i]), kConvWarps);
        }
        bar_init(s_addr(&bars.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_flag = 0;
    }
    // key tiles before each sequence
    {
        constexpr int kRun = (kWindowSeqs + kThreads - 1) / kThreads;
        int v[kRun];
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int s = tid * kRun + i;
            v[i] = 0;
            if (s < p.num_seqs) {
                const Span sp = span_of(p, s, false);
                v[i] = (sp.ctx + kRows - 1) / kRows;
                sm_ctx[s] = sp.ctx;
                sm_tokens[s] = sp.rows / p.group;
            }
            sum += v[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        if (lane == 31)
            sm_sums[warp] = incl;
        __syncthreads();
        int at = incl - sum;
        for (int k = 0; k < warp; ++k)
            at += sm_sums[k];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int s = tid * kRun + i;
            if (s <= p.num_seqs)
                sm_first[s] = at;
            at += v[i];
        }
    }
    __syncthreads();
    const Batch batch{sm_first, sm_ctx, sm_tokens, p.group, p.num_kv_heads};
    const int64_t total = (int64_t)sm_first[p.num_seqs] * p.num_kv_heads;
    const int64_t ctas = min((int64_t)gridDim.x, total);
    pdl_wait_primary();
    pdl_launch_dependents();
    if (blockIdx.x >= ctas)
        return;
    // a wait for the sums ran out: totals stay as they are
    const bool failed = TOTALS && __ldcg(p.failed) != 0;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            s_addr(&tmem_holder)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;

    // the share's first segment
    Walk w;
    {
        const int64_t at = blockIdx.x * total / ctas;
        w.left = (blockIdx.x + 1) * total / ctas - at;
        int lo = 0, hi = p.num_seqs;           // the last s with first[s] heads <= at
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)sm_first[mid] * p.num_kv_heads <= at)
                lo = mid;
            else
                hi = mid;
        }
        w.s = lo;
        const int64_t in = at - (int64_t)sm_first[lo] * p.num_kv_heads;
        const int n = sm_first[lo + 1] - sm_first[lo];
        w.h = (int)(in / n);
        w.j0 = (int)(in - (int64_t)w.h * n);
        batch.enter(w);
    }

    if (failed) {
        // ---------------- nothing to do: the CTA gives its tensor memory back ----------------
    } else if (warp < kFetchWarp) {
        // ---------------- softmax: group gi ----------------
        const int gi = warp >> 2;
        const int r = tid & (kRows - 1);               // tensor-memory lane
        const uint32_t t_s = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * gi;
        bool alive = true;
        uint32_t unit = 0;                             // scores this group has seen
        auto next_scores = [&]() {
            alive = alive && wait_warp(s_addr(&bars.s_full[gi]), unit & 1, waits);
            tc_fence_after();
        };
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(s_addr(&bars.s_free[gi]));
            ++unit;
        };
        int tile = 0;                                  // key tiles so far, with repetitions
        uint32_t qn = 0;                               // q tiles so far
        [[maybe_unused]] int turn = 0;                 // which of the parts
        do {
            const int64_t item = (int64_t)w.s * p.num_kv_heads + w.h;
            for (int pr = 0; pr < w.pairs; ++pr, tile += w.nk) {
                const int nq = q_tiles_of(w, pr);
                const int row0 = pr * 2 * kRows;
                for (int qt = 0; qt < nq; ++qt)
                    alive = alive && wait_warp(s_addr(&bars.q_full[(qn + qt) & 1]), ((qn + qt) >> 1) & 1,
                                               waits);
                if constexpr (!TOTALS) {
                    // one row a thread: groups 2 x + y take tile y of two over the key
                    // tiles of parity x; of one tile every fourth key tile each
                    const int qt = nq == 2 ? gi & 1 : 0;
                    const int every = nq == 2 ? 2 : 4;
                    const int row = row0 + qt * kRows + r;
                    const float f = *const_cast<const volatile float*>(&row_info[(qn + qt) & 1][r]);
                    const int pos = w.first_pos + row / p.group;
                    float m_run = kNegInf, l_run = 0.f;
                    // (uniform) from this key on some row of the pair does not see it
                    const int edge_key = w.first_pos + row0 / p.group;
                    for (int j = ((nq == 2 ? gi >> 1 : gi) - tile) & (every - 1); j < w.nk; j += every) {
                        next_scores();
                        if (alive) {
                            const int key0 = (w.j0 + j) * kRows;
                            const bool edge = key0 + kRows - 1 > edge_key;
                            const volatile float* ks = ks_ring[(tile + j) % kScaleRing];
                            // The reference only has to keep the sum from overflowing: any
                            // score of the row will do, the sum's own precision does the rest.
                            float2 ls[2] = {};
                            auto add_up = [&](auto masked) {
                                for_columns(t_s, kRows, [&](float(&x)[16], int c0) {
                                    if constexpr (decltype(masked)::value) {
                                        const int lim = pos - key0 - c0;       // the last key the row sees
#pragma unroll
                                        for (int e = 0; e < 16; ++e)
                                            x[e] = e <= lim ? x[e] : kNegInf;
                                    }
                                    float fb[2];
#pragma unroll
                                    for (int b = 0; b < 2; ++b)
                                        fb[b] = fmaxf(E8 ? f * ks[c0 / 8 + b] : f, kTiny);
                                    // (a row that sees any key of a tile sees its first)
                                    if (m_run == kNegInf)
                                        m_run = x[0] * fb[0];
                                    // without any score yet: hidden keys are 0 against the largest float,
                                    // and a score (the first was -inf) is infinite, which sums the tile again
                                    const float nm = decltype(masked)::value && m_run == kNegInf ? kMost : -m_run;
                                    const float2 nm2 = make_float2(nm, nm);
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const float2 t = ffma2(make_float2(x[e], x[e + 1]),
                                                               make_float2(fb[e / 8], fb[e / 8]), nm2);
                                        ls[(e >> 1) & 1] = fadd2(ls[(e >> 1) & 1],
                                                                 make_float2(fast_exp2(t.x), fast_exp2(t.y)));
                                    }
                                });
                            };
                            if (edge)
                                add_up(std::true_type{});
                            else
                                add_up(std::false_type{});
                            const float u = (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                            if (!__any_sync(0xffffffffu, !(u < kMuch))) {
                                l_run += u;
                            } else {
                                for_columns(t_s, kRows, [&](float(&x)[16], int c0) {
                                    const int lim = pos - key0 - c0;       // the last key the row sees
                                    float mx = kNegInf;
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const float fb = fmaxf(E8 ? f * ks[(c0 + e) / 8] : f, kTiny);
                                        x[e] = e <= lim ? x[e] * fb : kNegInf;
                                        mx = fmaxf(mx, x[e]);
                                    }
                                    if (mx > m_run + kRaise) {     // (the first finite one passes -inf)
                                        l_run *= m_run == kNegInf ? 0.f : fast_exp2(m_run - mx);
                                        m_run = mx;
                                    }
                                    const float nm = m_run == kNegInf ? 0.f : -m_run;
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        l_run += fast_exp2(x[e] + nm);
                                });
                            }
                        }
                        release();
                    }
                    // the groups' parts, of one row in the same place of each part
                    float(&part)[kSoftmax] = parts[turn];
                    turn ^= 1;
                    part[tid] = log_sum(m_run, l_run);
                    softmax_sync();
                    // (nobody writes the same parts again before the barrier behind the next)
                    if (tid < nq * kRows && row0 + tid < w.rows) {
                        const int step = nq * kRows;
                        float M = kNegInf, sum = 0.f;
#pragma unroll
                        for (int k = 0; k < kGroups; ++k)
                            if (k * step < kSoftmax)
                                M = fmaxf(M, part[k * step + tid]);
                        const float ref = M == kNegInf ? 0.f : M;
#pragma unroll
                        for (int k = 0; k < kGroups; ++k)
                            if (k * step < kSoftmax)
                                sum += fast_exp2(part[k * step + tid] - ref);
                        const float lse = log_sum(ref, sum);
                        if (w.nk == w.n) {
                            put_row(p.row_info + item * p.row_tiles * kInfo, row0 + tid, lse);
                        } else {
                            p.partials[(2 * (int64_t)blockIdx.x + (w.j0 == 0 ? 1 : 0)) * p.row_tiles * kRows + row0 +
                                       tid] = lse;
                            __threadfence();
                        }
                    }
                } else {
                    // one key a thread, over the rows of a q tile: groups 2 x + y take tile y
                    // of two for the key tiles of parity x, and the sums of y = 1 go to y = 0;
                    // with one tile every group takes every fourth key tile
                    const int qt = nq == 2 ? gi & 1 : 0;
                    const int every = nq == 2 ? 2 : 4;
                    const float* info = row_info[(qn + qt) & 1];
                    const int end = min(kRows, w.rows - row0 - qt * kRows);
                    const bool even = info[2 * kRows] != 0.f;
                    for (int j = ((nq == 2 ? gi >> 1 : gi) - tile) & (every - 1); j < w.nk; j += every) {
                        const int key = (w.j0 + j) * kRows + r;
                        float* at = p.weights + w.s * p.weights_seq + w.h * p.weights_head + key;
                        float before = 0.f;
                        if (qt == 0 && key < w.ctx)
                            before = *at;
                        float2 acc[2] = {};
                        next_scores();
                        if (alive) {
                            const float k_scale =
                                E8 ? *const_cast<const volatile float*>(&ks_ring[(tile + j) % kScaleRing][r / 8])
                                   : 1.f;
                            // (uniform) some row does not see some key of the tile
                            const bool edge = (w.j0 + j) * kRows + kRows - 1 > w.first_pos;
                            // the first row that sees the key, of the q tile's (keys in front of
                            // the rows may be further off than 32 bits hold times the heads)
                            const int lo = max(key - w.first_pos, 0) * p.group - row0 - qt * kRows;
                            const float f = fmaxf(k_scale * info[0], kTiny);
                            const float2 f2 = make_float2(f, f);
                            if (even && !edge && end == kRows) {
                                for_columns(t_s, kRows, [&](float(&x)[16], int c0) {
                                    const float* at_l = info + kRows + c0;
#pragma unroll
                                    for (int e = 0; e < 16; e += 4) {
                                        const float4 l = *reinterpret_cast<const float4*>(at_l + e);
                                        const float2 a = ffma2(make_float2(x[e], x[e + 1]), f2, make_float2(l.x, l.y));
                                        const float2 b =
                                            ffma2(make_float2(x[e + 2], x[e + 3]), f2, make_float2(l.z, l.w));
                                        acc[0] = fadd2(acc[0], make_float2(fast_exp2(a.x), fast_exp2(a.y)));
                                        acc[1] = fadd2(acc[1], make_float2(fast_exp2(b.x), fast_exp2(b.y)));
                                    }
                                });
                            } else if (even) {
                                for_columns(t_s, end, [&](float(&x)[16], int c0) {
                                    const float* at_l = info + kRows + c0;
#pragma unroll
                                    for (int e = 0; e < 16; e += 4) {
                                        const float4 l = *reinterpret_cast<const float4*>(at_l + e);
                                        const float2 a = ffma2(make_float2(x[e], x[e + 1]), f2, make_float2(l.x, l.y));
                                        const float2 b =
                                            ffma2(make_float2(x[e + 2], x[e + 3]), f2, make_float2(l.z, l.w));
                                        x[e] = fast_exp2(a.x), x[e + 1] = fast_exp2(a.y);
                                        x[e + 2] = fast_exp2(b.x), x[e + 3] = fast_exp2(b.y);
                                    }
                                    // (a row's sum may be NaN, which keys it does not see are not)
                                    if (edge || c0 + 16 > end) {
                                        const int from = min(max(lo - c0, 0), 16), n = min(end - c0, 16);
                                        const uint32_t rows = (0xffffu << from) & (0xffffu >> (16 - n));
#pragma unroll
                                        for (int e = 0; e < 16; ++e)
                                            x[e] = (rows >> e) & 1u ? x[e] : 0.f;
                                    }
#pragma unroll
                                    for (int e = 0; e < 16; e += 2)
                                        acc[(e >> 1) & 1] = fadd2(acc[(e >> 1) & 1], make_float2(x[e], x[e + 1]));
                                });
                            } else {
                                for_columns(t_s, end, [&](float(&x)[16], int c0) {
                                    const float* at_f = info + c0;
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        const float v = fast_exp2(
                                            fmaf(x[e], fmaxf(k_scale * at_f[e], kTiny), at_f[kRows + e]));
                                        acc[e & 1].x += c0 + e >= lo && c0 + e < end ? v : 0.f;
                                    }
                                });
                            }
                        }
                        release();
                        float sum = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                        if (nq == 2) {
                            // (nobody writes the same sums again before the barrier of the next tile)
                            float(&other)[kRows] = sums[gi >> 1][turn];
                            turn ^= 1;
                            if (qt == 1)
                                other[r] = sum;
                            pair_sync(gi >> 1);
                            sum += other[r];
                        }
                        if (qt == 0 && alive && key < w.ctx)
                            *at = before + sum;
                    }
                }
                __syncwarp();
                if (lane == 0)
                    for (int qt = 0; qt < nq; ++qt)
                        bar_arrive(s_addr(&bars.q_free[(qn + qt) & 1]));
                qn += nq;
            }
            if constexpr (!TOTALS) {
                if (w.nk < w.n) {
                    // the CTA that comes last merges the item's segments, in their order
                    const int64_t x = (int64_t)sm_first[w.s] * p.num_kv_heads + (int64_t)w.h * w.n;
                    auto owner = [&](int64_t u) {              // the CTA that holds key tile u
                        int64_t c = u * ctas / total;
                        while (c + 1 < ctas && (c + 1) * total / ctas <= u)
                            ++c;
                        return c;
                    };
                    const int64_t c0 = owner(x), c1 = owner(x + w.n - 1);
                    softmax_sync();
                    if (tid == 0) {
                        __threadfence();
                        is_last = atomicAdd(p.finished + item, 1) == (int)(c1 - c0);
                        __threadfence();
                    }
                    softmax_sync();
                    if (*const_cast<const volatile int*>(&is_last)) {
                        for (int row = tid; row < w.rows; row += kSoftmax) {
                            const float* pt = p.partials + row;
                            const int64_t per = (int64_t)p.row_tiles * kRows;
                            float M = kNegInf, sum = 0.f, ref = 0.f;
                            for (int64_t c = c0; c <= c1; c += kAtOnce) {
                                float v[kAtOnce];
#pragma unroll
                                for (int i = 0; i < kAtOnce; ++i)
                                    v[i] = c + i <= c1 ? __ldcg(pt + (2 * (c + i) + (c + i == c0 ? 1 : 0)) * per)
                                                       : kNegInf;
                                const float was = M;
#pragma unroll
                                for (int i = 0; i < kAtOnce; ++i)
                                    M = fmaxf(M, v[i]);
                                ref = M == kNegInf ? 0.f : M;
                                sum *= fast_exp2(was - ref);
#pragma unroll
                                for (int i = 0; i < kAtOnce; ++i)
                                    sum += fast_exp2(v[i] - ref);
                            }
                            put_row(p.row_info + item * p.row_tiles * kInfo, row, log_sum(ref, sum));
                        }
                    }
                }
            }
        } while (batch.next(w));
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // ---------------- products (one thread) ----------------
            const uint32_t id = instr_desc<CT>(kRows, kRows, 0);
            const uint32_t id2 = instr_desc<CT>(kRows, 2 * kRows, 0);
            constexpr uint32_t hi1k = desc_hi(1024);
            const uint32_t q_lo = desc_lo(sb + L::q, 16);
            const uint32_t k_lo = desc_lo(sb + L::ring, 16);
            uint32_t used = 0, parity = 0;             // by group: had scores; parity of the next wait
            uint32_t tile = 0, qn = 0;
            bool alive = true;
            auto free_group = [&](uint32_t gi) -> bool {
                if ((used >> gi) & 1u) {
                    if (!wait_one(s_addr(&bars.s_free[gi]), (parity >> gi) & 1u, waits))
                        return false;
                    parity ^= 1u << gi;
                }
                used |= 1u << gi;
                return true;
            };
            // scores of group gi; `both`: of gi and gi + 1, the keys against 256 rows of q
            auto product = [&](uint32_t gi, uint32_t q_slot, uint32_t k_off, bool both) -> bool {
                if (!free_group(gi) || (both && !free_group(gi + 1)))
                    return false;
                tc_fence_after();
                const uint32_t q_at = q_lo + (q_slot * L::PB >> 4);
                const uint32_t idesc = both ? id2 : id;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (uint32_t)((k >> 2) * L::PB + (k & 3) * 32) >> 4;
                    const uint32_t off_q = (uint32_t)((k >> 2) * 2 * L::PB + (k & 3) * 32) >> 4;
                    const uint32_t a = TOTALS ? k_lo + k_off + off : q_at + off_q;
                    const uint32_t b = TOTALS ? q_at + off_q : k_lo + k_off + off;
                    umma_h(tmem + 128u * gi, a, hi1k, b, hi1k, idesc, k > 0 ? 1u : 0u);
                }
                umma_commit(s_addr(&bars.s_full[gi]));
                if (both)
                    umma_commit(s_addr(&bars.s_full[gi + 1]));
                return true;
            };
            do {
                for (int pr = 0; alive && pr < w.pairs; ++pr) {
                    const uint32_t nq = q_tiles_of(w, pr);
                    for (uint32_t qt = 0; alive && qt < nq; ++qt)
                        alive = wait_one(s_addr(&bars.q_full[(qn + qt) & 1]), ((qn + qt) >> 1) & 1, waits);
                    for (int j = 0; alive && j < w.nk; ++j, ++tile) {
                        const uint32_t st = tile % ST;
                        alive = wait_one(s_addr(&bars.full[st]), (tile / ST) & 1, waits);
                        if (!alive)
                            break;
                        const uint32_t k_off = st * L::TB >> 4;
                        if (nq == 1)
                            alive = product(tile & 3, qn & 1, k_off, false);
                        else if (TOTALS && (qn & 1) == 0)
                            alive = product(2 * (tile & 1), 0, k_off, true);
                        else
                            alive = product(2 * (tile & 1), qn & 1, k_off, false) &&
                                    product(2 * (tile & 1) + 1, (qn + 1) & 1, k_off, false);
                        umma_commit(s_addr(&bars.empty[st]));
                    }
                    for (uint32_t qt = 0; qt < nq; ++qt)
                        umma_commit(s_addr(&bars.q_free[(qn + qt) & 1]));
                    qn += nq;
                }
            } while (alive && batch.next(w));
            // every product (and every commit's arrival) done before teardown
            umma_commit(s_addr(&bars.drain));
            bar_wait(s_addr(&bars.drain), 0);
        }
    } else if (warp == kFetchWarp) {
        // ---------------- copies of keys and q ----------------
        const int sh = 31 - __clz(p.block_size);       // (a power of two)
        const int bs = 1 << sh;
        const int per_tile = kRows >> sh;              // blocks of a tile, 4..16
        // the q tiles were written by the kernel before, these copies are another proxy's
        asm volatile("fence.proxy.async.global;" ::: "memory");

        // q tiles, in order, by lane 0: a pair's before its first key tile; of one tile,
        // where the pair before has one too, as soon as its slot is free.  (All key
        // tiles in front have been asked for by then, so the wait for a slot ends.)
        uint32_t qn = 0;
        Walk qw = w;                                   // the next pair to ask for
        int q_pr = 0;
        bool q_left = true;
        auto ask_q = [&]() -> bool {
            const int nq = q_tiles_of(qw, q_pr);
            const int64_t at = ((int64_t)qw.s * p.num_kv_heads + qw.h) * p.row_tiles + 2 * q_pr;
            for (int qt = 0; qt < nq; ++qt, ++qn) {
                const uint32_t slot = qn & 1;
                if (qn >= 2 && !wait_one(s_addr(&bars.q_free[slot]), ((qn >> 1) & 1) ^ 1, waits))
                    return false;
                // (a warp that gave up frees slots whose copy may be on its way: no second one)
                if (aborted(&abort_flag))
                    return false;
                const uint32_t bar = s_addr(&bars.q_full[slot]);
                expect_bytes(bar, L::TB + kInfo * 4);
#pragma unroll
                for (int n = 0; n < NP; ++n)
                    bulk_copy(sb + L::q + (2 * n + slot) * L::PB,
                              reinterpret_cast<const char*>(p.q_tiles) + (at + qt) * L::TB + n * L::PB, L::PB, bar);
                bulk_copy(s_addr(row_info[slot]), p.row_info + (at + qt) * kInfo, kInfo * 4, bar);
            }
            if (++q_pr == qw.pairs) {
                q_pr = 0;
                q_left = batch.next(qw);
            }
            return true;
        };

        // the key tiles in order; block ids two tiles ahead of their use, scales one
        struct Tile {
            int id;              // lane i: block i, -1: none
            int h;
            int nq;              // q tiles of its pair, 0: no tile; negative: the pair's first
        };
        int a_pr = 0, a_j = 0;                         // (w: the walk of what is asked for)
        bool a_more = true;
        auto take = [&]() -> Tile {
            Tile t{-1, 0, 0};
            if (!a_more)
                return t;
            t.h = w.h;
            t.nq = q_tiles_of(w, a_pr);
            if (a_j == 0)
                t.nq = -t.nq;
            const int tok = (w.j0 + a_j) * kRows + lane * bs;
            if (lane < per_tile && tok < w.ctx) {
                t.id = __ldg(p.block_tables + (int64_t)w.s * p.max_blocks_per_seq + (tok >> sh));
                if (t.id < 0 || (int64_t)t.id >= p.num_blocks) {
                    flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);
                    t.id = -1;
                }
            }
            if (++a_j == w.nk) {
                a_j = 0;
                if (++a_pr == w.pairs) {
                    a_pr = 0;
                    a_more = batch.next(w);
                }
            }
            return t;
        };
        const float2* scales = reinterpret_cast<const float2*>(p.scales);
        auto scale_of = [&](const Tile& t) -> float {
            if (!E8 || scales == nullptr)
                return 1.f;
            return t.id >= 0 ? __ldg(scales + (int64_t)t.id * p.num_kv_heads + t.h).x : 0.f;
        };
        Tile t0 = take(), t1 = take();
        float sc = scale_of(t0);
        bool alive = true;
        bool asked = false;                            // q of the next pair
        int jj = 0;                                    // key tiles asked for
        constexpr int SLOTS = E8 ? L::RAW : ST;        // that they go to
        for (; t0.nq != 0; ++jj) {
            const Tile t2 = take();
            const float sc1 = scale_of(t1);
            if (t0.nq < 0) {
                bool ok = true;
                if (!asked && lane == 0)
                    ok = ask_q();
                alive = __all_sync(0xffffffffu, ok);
                asked = false;
                if (!alive)
                    break;
            }
            const int slot = jj % SLOTS;
            const uint32_t bar = s_addr(E8 ? &bars.raw_full[E8 ? slot : 0] : &bars.full[E8 ? 0 : slot]);
            alive = wait_warp(s_addr(E8 ? &bars.raw_free[E8 ? slot : 0] : &bars.empty[E8 ? 0 : slot]),
                              ((jj / SLOTS) & 1) ^ 1, waits);
            if (!alive)
                break;
            if constexpr (E8) {
                // (a block's scale, for every 8 of its keys)
                const float v = __shfl_sync(0xffffffffu, sc, min(31, (lane * 8) >> sh));
                if (lane < kRows / 8)
                    *const_cast<volatile float*>(&ks_ring[jj % kScaleRing][lane]) = v;
                __syncwarp();                  // (lane 0's arrival hands on what every lane wrote)
            }
            // A block that the table does not have leaves its rows as they are (no row
            // sees them); a bad one's are zeros: filled by the tensor copy past the
            // cache's end, or by the converting warps.
            if constexpr (E8) {
                const uint32_t good = __ballot_sync(0xffffffffu, t0.id >= 0);
                if (lane == 0) {
                    raw_good[slot] = good;
                    expect_bytes(bar, __popc(good) * bs * D);
                }
                __syncwarp();
                if (t0.id >= 0)
                    bulk_copy(sb + L::raw + slot * L::RB + lane * bs * D,
                              reinterpret_cast<const char*>(p.k_cache) +
                                  ((int64_t)t0.id * p.num_kv_heads + t0.h) * bs * D,
                              bs * D, bar);
            } else {
                if (lane == 0)
                    expect_bytes(bar, L::TB);
                __syncwarp();
                if (lane < per_tile) {
                    const int y = t0.id >= 0 ? (int)(((int64_t)t0.id * p.num_kv_heads + t0.h) * bs)
                                             : (int)(p.num_blocks * p.num_kv_heads * bs);
#pragma unroll
                    for (int n = 0; n < NP; ++n)
                        tma_box(sb + L::ring + slot * L::TB + n * kRows * 128 + lane * bs * 128, &k_map, n * 64, y,
                                bar);
                }
            }
            if (!asked && abs(t0.nq) == 1) {
                bool more = false;
                if (lane == 0 && q_left && q_tiles_of(qw, q_pr) == 1 &&
                    (qn < 2 || test_wait(s_addr(&bars.q_free[qn & 1]), ((qn >> 1) & 1) ^ 1)))
                    more = ask_q();
                asked = __any_sync(0xffffffffu, more);
            }
            t0 = t1;
            t1 = t2;
            sc = sc1;
        }
        // what is on its way lands before the CTA ends, whichever role gave up (bounded)
        if (lane == 0) {
            for (int k = max(0, jj - SLOTS); k < jj; ++k)
                bar_wait(s_addr(E8 ? &bars.raw_full[E8 ? k % SLOTS : 0] : &bars.full[E8 ? 0 : k % SLOTS]),
                         (k / SLOTS) & 1);
            for (uint32_t k = qn < 2 ? 0u : qn - 2; k < qn; ++k)
                bar_wait(s_addr(&bars.q_full[k & 1]), (k >> 1) & 1);
        }
    } else if constexpr (E8) {
        // ---------------- codes into fp16 operands (four warps) ----------------
        // vector i: 32 rows on for every NP, 16 codes; eight lanes read 128 bytes side by
        // side (of two rows where D = 128), and write eight different chunks of the
        // swizzled panels
        const int ct = tid - kConvWarp * 32;
        const int c4 = lane & 3;
        const int rsub = ct >> 2;
        constexpr int NV = NP * 4;
        // tiles of the share, with repetitions
        int tiles = 0;
        do
            tiles += w.nk * w.pairs;
        while (batch.next(w));
        const int sh = 31 - __clz(p.block_size);
        for (int jj = 0; jj < tiles; ++jj) {
            const int rs = jj % L::RAW, st = jj % ST;
            if (!wait_warp(s_addr(&bars.raw_full[rs]), (jj / L::RAW) & 1, waits))
                break;
            const uint32_t src = sb + L::raw + rs * L::RB;
            const uint32_t good = *const_cast<const volatile uint32_t*>(&raw_good[rs]);
            uint4 x[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int row = i / NP * 32 + rsub;
                const int panel = NP == 2 ? ((rsub ^ i) & 1) : 0;
                x[i] = lds16(src + row * D + panel * 64 + c4 * 16);
                if (!((good >> (row >> sh)) & 1u))
                    x[i] = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            if (lane == 0)
                bar_arrive(s_addr(&bars.raw_free[rs]));
            if (!wait_warp(s_addr(&bars.empty[st]), ((jj / ST) & 1) ^ 1, waits))
                break;
            const uint32_t dst = sb + L::ring + st * L::TB;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                uint4 lo, hi;
                e4m3x4_to_f16x2(x[i].x, lo.x, lo.y);
                e4m3x4_to_f16x2(x[i].y, lo.z, lo.w);
                e4m3x4_to_f16x2(x[i].z, hi.x, hi.y);
                e4m3x4_to_f16x2(x[i].w, hi.z, hi.w);
                const int row = i / NP * 32 + rsub;
                const int panel = NP == 2 ? ((rsub ^ i) & 1) : 0;
                const uint32_t at = dst + panel * kRows * 128 + row * 128;
                st_shared16(at + (((2 * c4) ^ (row & 7)) << 4), lo);
                st_shared16(at + (((2 * c4 + 1) ^ (row & 7)) << 4), hi);
            }
            async_proxy_fence();
            __syncwarp();
            if (lane == 0)
                bar_arrive(s_addr(&bars.full[st]));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (!TOTALS && tid == 0 && aborted(&abort_flag))
        *p.failed = 1;
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <class... Args>
cudaError_t launch_early(void (*kern)(Args...), int64_t ctas, int threads, int smem, cudaStream_t stream,
                         Args... args)
{
    if (ctas > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int QT, int CT, bool E8, int D>
cudaError_t run(const WeightsParams& p, cudaStream_t stream)
{
    using L = Layout<D, E8>;
    static std::atomic<bool> configured[64];      // (threads may call at once)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        for (auto kern : {weights_pass_kernel<CT, E8, D, false>, weights_pass_kernel<CT, E8, D, true>}) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::alloc);
            if (e != cudaSuccess)
                return e;
        }
        configured[dev] = true;
    }
    CUtensorMap map = {};
    if (!E8 && !cache_map(&map, p.k_cache, p.num_blocks * p.num_kv_heads * p.block_size, D, p.block_size))
        return cudaErrorNotSupported;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    e = launch_early(weights_tiles_kernel<QT, CT, D>, items * p.row_tiles, kTileThreads, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    e = launch_early(weights_pass_kernel<CT, E8, D, false>, p.ctas, threads_of<E8>(), L::alloc, stream, p, map);
    if (e != cudaSuccess)
        return e;
    return launch_early(weights_pass_kernel<CT, E8, D, true>, p.ctas, threads_of<E8>(), L::alloc, stream, p, map);
}

template <int QT, int CT, bool E8>
cudaError_t by_dim(const WeightsParams& p, cudaStream_t stream)
{
    return p.head_dim == 128 ? run<QT, CT, E8, 128>(p, stream) : run<QT, CT, E8, 64>(p, stream);
}

}  // namespace

cudaError_t launch_attention_weights(const WeightsParams& p, cudaStream_t stream)
{
    if (p.num_seqs > kWindowSeqs)
        return cudaErrorNotSupported;
    if (p.cache_dtype == kE4M3)
        return p.q_dtype == kF16 ? by_dim<kF16, kF16, true>(p, stream)
                                 : by_dim<kBF16, kF16, true>(p, stream);
    return p.q_dtype == kF16 ? by_dim<kF16, kF16, false>(p, stream)
                             : by_dim<kBF16, kBF16, false>(p, stream);
}

}  // namespace pkv
