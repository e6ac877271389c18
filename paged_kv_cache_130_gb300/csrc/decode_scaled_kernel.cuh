// decode_scaled_kernel.cuh -- decode attention over an E4M3 cache with a scale per
// block and KV head: the kernels of decode_scaled.cu (plain), decode_weights.cu and
// decode_scaled_prefix.cu.
//
// With code c and the block's scales ks, vs:
//   x_t = (scale ks) (q . ck_t),   out = sum_t exp(x_t - m) vs cv_t / sum_t exp(x_t - m).
// A scale belongs to a whole block of one head, so it never touches the
// elements: ks multiplies the token's score, vs its softmax weight.  The codes
// go to the tensor cores as fp16, in which every E4M3 value is exact.
//
// One CTA takes a run of tokens of one sequence and KV head with up to 16 query
// heads; its warps stride over the run in steps of 16 tokens.  Lane
// (g, t) = (lane / 4, lane % 4).
//   * S^T = K Q^T (mma m16n8k16, fp16 in, fp32 out): rows = the 16 tokens,
//     columns = 8 query heads.  The order of head_dim inside the dot product
//     is free, so lane (g, t) takes 16-byte vectors of the rows of tokens g and
//     g + 8 as they lie in memory, and q is laid out to match.
//   * q is scaled per head by a power of two to at most 2^14 in size, which
//     makes bf16 values fp16 without loss down to 2^-28 of the head's largest.
//   * Softmax: fp32, base 2.  The running maximum moves only when some score
//     passes it by more than 2^8 (weights stay below 2^8); one vote per step
//     decides, the sums over lanes wait for the end.
//   * O^T = V^T P^T: rows = head_dim, k = the tokens.  Lane (g, t) takes V of
//     tokens 2t, 2t + 1, 2t + 8, 2t + 9 for its 1/8 of head_dim; a byte permute
//     pairs two tokens' codes, and the conversion to fp16 yields the operand.
//     P^T comes from the scores through movmatrix.  The weights are rounded to
//     fp16 after the multiplication by vs / vref 2^6, vref = at most twice the
//     largest vs so far: each is off by at most 2^-11 of itself, or, where that
//     product is subnormal (a weight times vs below 2^-19 or so of the largest of
//     both), by 2^-30 of the largest weight times the largest vs.
// The running maximum, sums and the output accumulators are fp32.
//
// Bound by HBM where contexts are long: 16 of 8,192..32,768 tokens, 32 heads, D
// 128, block 32: 2,480 MB in 371 us, 6.68 TB/s (the partitions of 2,048 tokens
// that this replaced: 410 us). 64 contexts of 1,024..4,096 tokens, 64 heads over
// 8: 337 MB in 64 us; there the 4 us to the first codes, the changes of item and
// the reduce (3 us) show. Measured beside it: two or eight warps a CTA 68 and 88
// us, four CTAs of 128 registers 383 us on the long contexts.
#pragma once

#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "pkv_common.cuh"
#include "scaled_internal.h"

namespace pkv {
namespace dsk {

using dec::ceil_div_i;
using dec::kNegInf;
using dec::PartitionWork;

constexpr int kWarps = 4;
constexpr int kMaxGroup = 16;          // query heads per KV head
constexpr int kOnePass = 1024;         // tokens: contexts up to here are one CTA's work
constexpr float kRaise = 8.f;          // log2: how far a score may pass the maximum
constexpr float kWeightScale = 64.f;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements, lane 4i + j holding row i,
// columns 2j and 2j + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^floor(log2 x) of a positive finite x, at least 2^-126.
__device__ __forceinline__ float floor_pow2(float x)
{
    return __uint_as_float(max(__float_as_uint(x) & 0x7f800000u, 0x00800000u));
}

// The vectors of one lane's part of a row: D / 4 bytes of K, D / 8 of V.
template <int D>
struct Step {
    uint32_t k[2][D / 16];      // rows g, g + 8
    uint32_t v[4][D / 32];      // tokens 2t, 2t + 1, 2t + 8, 2t + 9
};

__device__ __forceinline__ uint2 ld_stream8(const void* p)
{
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// Equal shares: tokens of every (sequence, KV head) in units of kUnit, laid end
// to end (sequence, then head, then position), kItemUnits units without tokens in
// front of each item for what starting it costs; CTA c of C takes units
// [floor(c T / C), floor((c + 1) T / C)) of the T there are, whatever items they
// belong to.  An item whose tokens one CTA holds whole is written out; a CTA has
// at most two others, which it files as partials 2 c + 1 (starts at the item's
// first token) and 2 c (starts inside the item), and the reduce kernel finds an
// item's partials from the same arithmetic.
constexpr int kUnit = 16 * kWarps;         // tokens: one step for each warp
constexpr int kItemUnits = 3;              // merge, q and first codes: ~4 us beside ~1.1 us a unit
constexpr int kMinUnits = 8;               // smallest share
// (a share has at least kMinUnits / 2 units: 9 in two are 4 and 5)
static_assert(kMinUnits / 2 > kItemUnits, "at most one CTA of an item has none of its tokens");
constexpr int kMaxBalanced = 1024;         // sequences

// What the kernels do beside the plain decode.
//   kWeights: every score goes to `scores`, from which each token's softmax weight,
//     summed over the query heads of its KV head, is added to `weights`: here where
//     a CTA holds whole contexts, else by the kernel of decode_weights.cu.
//   kShared: sequences [grp_begin[i], grp_begin[i + 1]) share their leading blocks.
//     A group's prefix is read once for each `rows` rows (members x query heads of
//     a KV head), each sequence's own tokens for its query heads; the reduce
//     kernel merges what belongs to a row.
constexpr int kPlain = 0, kWeights = 1, kShared = 2;
constexpr int kMaxEntries = kSharedEntries;        // kShared: groups and sequences

template <int MODE>
constexpr int max_entries()
{
    return MODE == kShared ? kMaxEntries : kMaxBalanced;
}

struct Shares {
    int64_t total;                         // units
    uint32_t ctas;                         // CTAs that have any
    int64_t each;                          // total / ctas
    uint32_t rest;                         // total % ctas
    __device__ __forceinline__ int64_t begin(uint32_t c) const
    {
        return c * each + c * rest / ctas;       // (ctas < 2^16: 32 bits hold c rest)
    }
    // the CTA that holds unit x
    __device__ __forceinline__ uint32_t owner(int64_t x) const
    {
        uint32_t c = min(ctas - 1, (uint32_t)((float)x * (float)ctas / (float)total));
        while (c > 0 && begin(c) > x)
            --c;
        while (c + 1 < ctas && begin(c + 1) <= x)
            ++c;
        return c;
    }
};

// Units of sequence s: 0 for an empty context and for one that cannot be used.
__device__ __forceinline__ int units_of(const DecodeParams& p, int s, bool flag)
{
    const int ctx = __ldg(p.context_lens + s);
    if (ctx < 0 || ctx > p.max_context_len || ctx > p.max_blocks_per_seq * p.block_size) {
        if (flag)
            flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
        return 0;
    }
    return ctx > 0 ? ceil_div_i(ctx, kUnit) + kItemUnits : 0;
}

// Group i: its first member, its members and the tokens of its prefix; no tokens
// when its entry cannot be used.
struct Group {
    int begin, members, prefix;
};

__device__ __forceinline__ Group group_at(const DecodeParams& p, int i, bool flag)
{
    Group g;
    g.begin = __ldg(p.grp_begin + i);
    const int end = __ldg(p.grp_begin + i + 1);
    const int blocks = __ldg(p.grp_prefix_blocks + i);
    g.members = min(end - g.begin, p.max_group_size);
    g.prefix = blocks * p.block_size;
    if (g.begin < 0 || end < g.begin || end > p.num_seqs || blocks < 0 || blocks > p.max_prefix_blocks) {
        if (flag)
            flag_error(p.dev_err, PKV_DEVERR_PREFIX);
        g.members = g.prefix = 0;
    }
    return g;
}

// Row tiles of a group's prefix: `rt` rows (member, query head) each.
__device__ __forceinline__ int tiles_of(const DecodeParams& p, const Group& g, int rt)
{
    return ceil_div_i(g.members * p.group, rt);
}

// The group of sequence s (the last that starts at or before it).
__device__ __forceinline__ int group_of(const DecodeParams& p, int s)
{
    int i = 0, hi = p.num_groups;
    while (hi - i > 1) {
        const int mid = (i + hi) >> 1;
        if (__ldg(p.grp_begin + mid) <= s)
            i = mid;
        else
            hi = mid;
    }
    return i;
}

// Prefix tokens of sequence s, of group g, and whether its output is zero: a
// length that cannot be used, or a group entry or member number that cannot.
__device__ __forceinline__ int own_begin(const DecodeParams& p, int s, int ctx, int i, const Group& g,
                                         bool& bad)
{
    bad = ctx < 0 || ctx > p.max_context_len || ctx > p.max_blocks_per_seq * p.block_size;
    if (__ldg(p.grp_prefix_blocks + i) == 0)
        return 0;
    bad = bad || g.prefix <= 0 || s < g.begin || s - g.begin >= g.members || ctx < g.prefix;
    return g.prefix;
}

// An entry of a shared batch: the groups' prefixes, then the sequences' own tokens.
// The item of a KV head begins at token `from` (of sequence `from`: a prefix) and ends
// before token `end`.
struct Entry {
    int from, end;
    int rows;                  // members x query heads of a KV head; 0: no item
};

__device__ __forceinline__ Entry entry_at(const DecodeParams& p, int e, const int* begins, bool flag)
{
    Entry en{0, 0, 0};
    if (e < p.num_groups) {
        const Group g = group_at(p, e, flag);
        if (g.prefix > 0 && p.prefix_partition == 0)
            en = Entry{g.begin, g.prefix, g.members * p.group};
        return en;
    }
    const int s = e - p.num_groups;
    const int ctx = __ldg(p.context_lens + s);
    int i = 0, hi = p.num_groups;              // the group: the last that starts at or before s
    while (hi - i > 1) {
        const int mid = (i + hi) >> 1;
        if (begins[mid] <= s)
            i = mid;
        else
            hi = mid;
    }
    bool bad;
    const int pre = own_begin(p, s, ctx, i, group_at(p, i, false), bad);
    if (bad && flag)
        flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
    if (!bad && ctx > pre)
        en = Entry{pre, ctx, p.group};
    return en;
}

// Its units (of one KV head), with all the row tiles of a prefix.
__device__ __forceinline__ int entry_units(const DecodeParams& p, int e, const Entry& en, int rt)
{
    if (en.rows == 0)
        return 0;
    return e < p.num_groups ? (ceil_div_i(en.end, kUnit) + kItemUnits) * ceil_div_i(en.rows, rt)
                            : ceil_div_i(en.end - en.from, kUnit) + kItemUnits;
}

// Shared memory of a shared batch beside the kernel's own: its entries, and the
// groups' first members.
inline size_t shared_entries_bytes(int num_groups, int num_seqs)
{
    return ((size_t)num_groups + num_seqs) * sizeof(Entry) + ((size_t)num_groups + 1) * sizeof(int);
}

// first[e] = units before entry e (of one KV head), first[entries] = all; an
// entry is a sequence, or (kShared) as above.  Called by a whole CTA of kWarps
// warps.  Every thread takes a run of up to max_entries / (32 kWarps) entries, so
// that the lengths cost one round trip.
template <int MODE>
__device__ __forceinline__ void scan_units(const DecodeParams& p, int* first, int rt, bool flag,
                                           Entry* table = nullptr)
{
    constexpr int kRun = max_entries<MODE>() / (32 * kWarps);
    const int entries = MODE == kShared ? p.num_groups + p.num_seqs : p.num_seqs;
    __shared__ int sums[kWarps];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int per = ceil_div_i(entries, 32 * kWarps);          // <= kRun
    const int s0 = threadIdx.x * per;
    int v[kRun];
    int sum = 0;
    int* begins = reinterpret_cast<int*>(table + entries);
    if constexpr (MODE == kShared) {
        for (int i = threadIdx.x; i <= p.num_groups; i += 32 * kWarps)
            begins[i] = __ldg(p.grp_begin + i);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        v[i] = 0;
        if (i < per && s0 + i < entries) {
            if constexpr (MODE == kShared) {
                const Entry en = entry_at(p, s0 + i, begins, flag);
                table[s0 + i] = en;
                v[i] = entry_units(p, s0 + i, en, rt);
            } else {
                v[i] = units_of(p, s0 + i, flag);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i)
        sum += v[i];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += u;
    }
    if (lane == 31)
        sums[warp] = incl;
    __syncthreads();
    int at = incl - sum;
#pragma unroll
    for (int k = 0; k < kWarps; ++k)
        at += k < warp ? sums[k] : 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        if (i < per && s0 + i < entries)
            first[s0 + i] = at;
        at += v[i];
    }
    if (threadIdx.x == 32 * kWarps - 1)
        first[entries] = at;
    __syncthreads();
}

__device__ __forceinline__ Shares shares_of(const DecodeParams& p, int units, uint32_t ctas)
{
    Shares sh;
    sh.total = (int64_t)units * p.num_kv_heads;
    sh.ctas = min((int64_t)ctas, (sh.total + kMinUnits - 1) / kMinUnits);
    if (sh.ctas == 0) {
        sh.each = sh.rest = 0;
    } else if (sh.total <= 0xffffffffll) {
        sh.each = (uint32_t)sh.total / sh.ctas;          // (64-bit divisions are long)
        sh.rest = (uint32_t)sh.total % sh.ctas;
    } else {
        sh.each = sh.total / sh.ctas;
        sh.rest = (uint32_t)(sh.total % sh.ctas);
    }
    return sh;
}

// sum over the query heads of 2^(x - maximum) / sum; a masked score is -inf, and
// the sum of a row without any score 0.
__device__ __forceinline__ float token_weight(const float* sc, int G, int pitch, const float2* fin)
{
    float w = 0.f;
    auto add = [&](float x, int r) {
        if (r < G && x != kNegInf)
            w = fmaf(exp2_fast(x - fin[r].x), fin[r].y, w);
    };
    if (pitch >= 4) {
        for (int r = 0; r < G; r += 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(sc + r));
            add(v.x, r), add(v.y, r + 1), add(v.z, r + 2), add(v.w, r + 3);
        }
    } else {
        for (int r = 0; r < G; ++r)
            add(__ldcg(sc + r), r);
    }
    return w;
}

// BAL: equal shares; otherwise one CTA per (partition, sequence, KV head).
template <int QT, int D, int BS, int NNT, bool BAL, int MODE>
__global__ void __launch_bounds__(kWarps * 32, NNT == 1 ? 3 : 2)
    decode_scaled_kernel(const DecodeParams p, const float2* __restrict__ scales, const DecodeExtra x_)
{
    static_assert(BAL || MODE != kShared, "a shared batch is cut into equal shares");
    constexpr int NKS = D / 16;                // k-steps of the scores
    constexpr int NM = D / 16;                 // m-tiles of the output
    constexpr int NKV = D / 64;                // 16-byte vectors of a K row per lane
    constexpr int BPS = BS == 8 ? 2 : 1;       // blocks per step
    constexpr int SPB = BS == 32 ? 2 : 1;      // steps per block
    constexpr int RT = 8 * NNT;                // rows
    constexpr int PITCH = D + 2;               // (two-way conflicts at most)

    __shared__ float sm_m[kWarps][RT];
    __shared__ float sm_l[kWarps][RT];
    __shared__ float sm_q[RT];                 // 1 / the heads' q scales
    __shared__ __align__(8) float sm_acc[kWarps * RT * PITCH];
    __shared__ uint2 sm_qf[NNT * NKS * 32];    // q fragments by lane
    __shared__ float2 sm_final[MODE == kWeights && !BAL ? RT : 1];   // maximum, 1 / sum
    __shared__ int sm_first[BAL ? max_entries<MODE>() + 1 : 1];

    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int g = lane >> 2;
    const int t = lane & 3;
    const int G = p.group;

    // what comes before in the stream may still write q, the cache and the tables;
    // the kernel of the prefixes only writes their partials: it is waited for at the end
    const bool beside = MODE == kShared && p.prefix_partition > 0;
    if (!beside)
        pdl_wait_primary();
    pdl_launch_dependents();

    // BAL: units left of the CTA's share, and where it stands: unit u0 of KV
    // head bal_h of sequence bal_s (kShared: item bal_h, head by head, of entry
    // bal_s, whose heads have `tiles` items of n units each)
    int64_t left = 1;
    int bal_s = 0, bal_h = 0, u0 = 0;
    [[maybe_unused]] int tiles = 1, bal_n = 0;
    extern __shared__ int sm_dyn[];
    [[maybe_unused]] Entry* table_e = reinterpret_cast<Entry*>(sm_dyn);    // kShared
    [[maybe_unused]] auto enter = [&](int e) {
        tiles = e < p.num_groups ? ceil_div_i(table_e[e].rows, RT) : 1;
        bal_n = (sm_first[e + 1] - sm_first[e]) / tiles;
    };
    if constexpr (BAL) {
        const int entries = MODE == kShared ? p.num_groups + p.num_seqs : p.num_seqs;
        scan_units<MODE>(p, sm_first, RT, blockIdx.x == 0, table_e);
        if (MODE == kShared && blockIdx.x == 0)        // for the kernel behind
            for (int i = threadIdx.x; i <= entries; i += kWarps * 32)
                x_.first[i] = sm_first[i];
        const Shares sh = shares_of(p, sm_first[entries], gridDim.x);
        if (blockIdx.x >= sh.ctas) {
            if (beside)
                pdl_wait_primary();
            return;
        }
        const int64_t at = sh.begin(blockIdx.x);
        left = sh.begin(blockIdx.x + 1) - at;
        int hi = entries;                      // the last s with first[s] Hkv <= at
        while (hi - bal_s > 1) {
            const int mid = (bal_s + hi) >> 1;
            if ((int64_t)sm_first[mid] * p.num_kv_heads <= at)
                bal_s = mid;
            else
                hi = mid;
        }
        int n = sm_first[bal_s + 1] - sm_first[bal_s];
        if constexpr (MODE == kShared) {
            enter(bal_s);
            n = bal_n;
        }
        const int64_t in = at - (int64_t)sm_first[bal_s] * p.num_kv_heads;
        bal_h = in <= 0xffffffffll ? (int)((uint32_t)in / (uint32_t)n) : (int)(in / n);
        u0 = (int)(in - (int64_t)bal_h * n);
    }
    while (left > 0) {
    int s, head, t_begin, t_end;
    bool direct;
    int64_t prow;                              // first row of the partial
    int nrows = G;
    // kShared: row r is query head head G + (rr0 + r) % G of sequence s + (rr0 + r) / G
    [[maybe_unused]] int rr0 = 0;
    [[maybe_unused]] bool whole = false;       // filed by sequence and head
    if constexpr (MODE == kShared) {
        const int e = bal_s;
        const int n = bal_n;
        const int u1 = (int)min((int64_t)n, u0 + left);
        const int b = max(u0 - kItemUnits, 0) * kUnit;
        head = bal_h / tiles;
        const Entry en = table_e[e];
        const int end = en.end;
        bool prefix = e < p.num_groups;
        if (prefix) {
            rr0 = (bal_h - head * tiles) * RT;
            s = en.from;
            nrows = min(RT, en.rows - rr0);
            t_begin = b;
        } else {
            s = e - p.num_groups;
            t_begin = en.from + b;
            prefix = en.from > 0;
        }
        t_end = min(end, t_begin - b + (u1 - kItemUnits) * kUnit);
        whole = u0 <= kItemUnits && u1 == n;
        direct = whole && !prefix;
        // pieces lie behind one another, two a CTA; behind them the rows of whole
        // items: the own tokens' as in q, then the prefixes'
        prow = whole ? 2 * (int64_t)gridDim.x * RT +
                           (e < p.num_groups ? (int64_t)p.num_seqs * p.num_heads : 0)
                     : (2 * (int64_t)blockIdx.x + (u0 <= kItemUnits ? 1 : 0)) * RT;
        left -= u1 - u0;
        u0 = 0;
        if (++bal_h == p.num_kv_heads * tiles && left > 0) {
            bal_h = 0;
            do
                ++bal_s;
            while (sm_first[bal_s + 1] == sm_first[bal_s]);
            enter(bal_s);
        }
        if (u1 <= kItemUnits)
            break;                             // the share ends before the item's tokens
    } else if constexpr (BAL) {
        s = bal_s;
        head = bal_h;
        const int n = sm_first[s + 1] - sm_first[s];
        const int u1 = (int)min((int64_t)n, u0 + left);
        t_begin = max(u0 - kItemUnits, 0) * kUnit;
        t_end = min(__ldg(p.context_lens + s), (u1 - kItemUnits) * kUnit);
        direct = u0 <= kItemUnits && u1 == n;
        prow = (2 * (int64_t)blockIdx.x + (u0 <= kItemUnits ? 1 : 0)) * RT;
        left -= u1 - u0;
        // the next item: the next head, or head 0 of the next sequence with tokens
        u0 = 0;
        if (++bal_h == p.num_kv_heads && left > 0) {
            bal_h = 0;
            do
                ++bal_s;
            while (sm_first[bal_s + 1] == sm_first[bal_s]);
        }
        if (u1 <= kItemUnits)
            break;                             // the share ends before the item's tokens
    } else {
        int64_t idx = blockIdx.x;
        head = (int)(idx % p.num_kv_heads);
        idx /= p.num_kv_heads;
        s = (int)(idx % p.num_seqs);
        const int part = (int)(idx / p.num_seqs);
        const PartitionWork w = dec::locate(p, s, part, threadIdx.x == 0);
        if (w.idle || w.zero_out || w.zero_partial) {
            if (!w.idle)
                dec::write_trivial<QT>(p, w, head * G, G, threadIdx.x, blockDim.x);
            return;
        }
        t_begin = w.t_begin;
        t_end = w.t_end;
        direct = w.direct;
        prow = dec::partial_row(p, s, head * G, w.slot);
        left = 0;
    }

    // row r of the item as a row of q and out
    auto row_of = [&](int r) -> int64_t {
        if constexpr (MODE == kShared) {
            const int m = (rr0 + r) / G;
            return (int64_t)(s + m) * p.num_heads + head * G + (rr0 + r - m * G);
        } else {
            return (int64_t)s * p.num_heads + head * G + r;
        }
    };

    // q: each warp scales rows warp, warp + 4, ... by a power of two that
    // brings the largest element into [2^13, 2^14), and files the fragments
    for (int r = warp; r < 8 * NNT; r += kWarps) {
        constexpr int EPL = D / 32;            // elements per lane
        float x[EPL];
        float mx = 0.f;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + row_of(r) * D;
#pragma unroll
        for (int e = 0; e < EPL; e += 2) {
            const uint32_t u =
                r < nrows ? __ldg(reinterpret_cast<const uint32_t*>(src) + (lane * EPL + e) / 2) : 0u;
            const float2 f = unpack2<QT>(u);
            x[e] = f.x, x[e + 1] = f.y;
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // up = 2^13 / 2^floor(log2 mx), kept where it and its inverse are normal
        float up = 1.f;
        if (mx > 0.f && mx < __builtin_huge_valf())
            up = exp2f(fminf(fmaxf(13.f - (float)((int)(__float_as_uint(mx) >> 23) - 127), -120.f), 120.f));
        if (lane == 0)
            sm_q[r] = 1.f / up;
        // dims d = 64 v + 16 t' + 4 w + e of k-step 4 v + w belong to lane (r, t')
#pragma unroll
        for (int e = 0; e < EPL; e += 2) {
            const int d = lane * EPL + e;
            const int ks = 4 * (d / 64) + (d % 16) / 4;
            const int ln = 4 * (r & 7) + (d % 64) / 16;
            reinterpret_cast<uint32_t*>(sm_qf)[(((r >> 3) * NKS + ks) * 32 + ln) * 2 + (d % 4) / 2] =
                pack_f16(x[e] * up, x[e + 1] * up);
        }
    }
    __syncthreads();
    float qk[NNT][2];
#pragma unroll
    for (int n = 0; n < NNT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            qk[n][h] = p.qk_scale_log2 * sm_q[8 * n + 2 * t + h];

    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks_per_seq + t_begin / BS;
    const int nblk = ceil_div_i(t_end - t_begin, BS);
    const int nstep = ceil_div_i(t_end - t_begin, 16);
    const int64_t tile = (int64_t)BS * D;
    const char* kbase = reinterpret_cast<const char*>(p.k_cache) + head * tile;
    const char* vbase = reinterpret_cast<const char*>(p.v_cache) + head * tile;
    const int64_t stride = (int64_t)p.num_kv_heads * tile;

    float acc[NNT][NM][4];
    float m_h[NNT][2], l_h[NNT][2];
    float vref = 0.f;
#pragma unroll
    for (int n = 0; n < NNT; ++n) {
        m_h[n][0] = m_h[n][1] = kNegInf;
        l_h[n][0] = l_h[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < NM; ++j)
            acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.f;
    }

    // The warp's steps are warp, warp + kWarps, ...; lane i keeps the block
    // entries and scales of step (chunk * (32 / BPS) + i / BPS).
    const int my_steps = nstep > warp ? ceil_div_i(nstep - warp, kWarps) : 0;
    constexpr int SPC = 32 / BPS;              // steps whose entries the lanes hold
    int ent = -1;
    float2 ent_s = make_float2(0.f, 0.f);
    auto refill = [&](int it) {
        const int step = warp + (it + lane / BPS) * kWarps;
        const int bi = BPS == 2 ? step * 2 + (lane & 1) : step / SPB;
        ent = -1;
        ent_s = make_float2(0.f, 0.f);
        if (bi < nblk) {
            ent = __ldg(table + bi);
            if (ent < 0 || (int64_t)ent >= p.num_blocks) {
                flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);
                ent = -1;
            } else {
                ent_s = __ldg(scales + (int64_t)ent * p.num_kv_heads + head);
            }
        }
    };
    struct Meta {
        float ks[BPS], vs[BPS];
        bool ok[BPS];
    };
    auto load = [&](int it, Step<D>& st, Meta& me) {
        const int i = it % SPC;
        if (i == 0)
            refill(it);
        const int step = warp + it * kWarps;
        const char* kp[BPS];
        const char* vp[BPS];
#pragma unroll
        for (int b = 0; b < BPS; ++b) {
            const int e = __shfl_sync(0xffffffffu, ent, i * BPS + b);
            me.ks[b] = __shfl_sync(0xffffffffu, ent_s.x, i * BPS + b);
            me.vs[b] = __shfl_sync(0xffffffffu, ent_s.y, i * BPS + b);
            me.ok[b] = e >= 0;
            const int64_t off = (int64_t)max(e, 0) * stride + (SPB == 2 ? (step & 1) * 16 * D : 0);
            kp[b] = kbase + off;
            vp[b] = vbase + off;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int b = BPS == 2 ? hf : 0;
            const int row = BPS == 2 ? g : hf * 8 + g;
#pragma unroll
            for (int v = 0; v < NKV; ++v) {
                const uint4 u = me.ok[b] ? ld_stream(kp[b] + row * D + v * 64 + t * 16)
                                         : make_uint4(0, 0, 0, 0);
                st.k[hf][4 * v] = u.x, st.k[hf][4 * v + 1] = u.y;
                st.k[hf][4 * v + 2] = u.z, st.k[hf][4 * v + 3] = u.w;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = BPS == 2 ? j >> 1 : 0;
            const int row = 2 * t + (j & 1) + (BPS == 2 ? 0 : 8 * (j >> 1));
            if constexpr (D == 128) {
                const uint4 u = me.ok[b] ? ld_stream(vp[b] + row * D + g * 16)
                                         : make_uint4(0, 0, 0, 0);
                st.v[j][0] = u.x, st.v[j][1] = u.y, st.v[j][2] = u.z, st.v[j][3] = u.w;
            } else {
                const uint2 u = me.ok[b] ? ld_stream8(vp[b] + row * D + g * 8) : make_uint2(0, 0);
                st.v[j][0] = u.x, st.v[j][1] = u.y;
            }
        }
    };

    auto compute = [&](int it, Step<D>& st, const Meta& me) {
        const int tb = t_begin + (warp + it * kWarps) * 16;    // first token of the step
        // scores
        float sc[NNT][2][4];
#pragma unroll
        for (int n = 0; n < NNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sc[n][0][e] = sc[n][1][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(st.k[0][ks], a0, a2);
            e4m3x4_to_f16x2(st.k[1][ks], a1, a3);
#pragma unroll
            for (int n = 0; n < NNT; ++n) {
                const uint2 q = sm_qf[(n * NKS + ks) * 32 + lane];
                mma_f16(sc[n][ks & 1], a0, a1, a2, a3, q.x, q.y);
            }
        }
        // x[n][e]: token tb + g + 8 (e >> 1), head 8 n + 2 t + (e & 1)
        const bool tail = tb + 16 > t_end;
        float x[NNT][4];
        bool raise = false;
#pragma unroll
        for (int n = 0; n < NNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int b = BPS == 2 ? e >> 1 : 0;
                x[n][e] = (sc[n][0][e] + sc[n][1][e]) * (qk[n][e & 1] * me.ks[b]);
                if (!me.ok[b] || (tail && tb + g + 8 * (e >> 1) >= t_end))
                    x[n][e] = kNegInf;
                raise |= x[n][e] > m_h[n][e & 1] + kRaise;
            }
        if constexpr (MODE == kWeights) {
            // by token and (padded) query head: the warp's 16 tokens lie together
            float* at = x_.scores + ((int64_t)(s * (int64_t)p.num_kv_heads + head) * x_.score_tokens + tb + g) *
                                        x_.pitch + 2 * t;
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                for (int n = 0; n < NNT; ++n) {
                    float* a = at + h2 * 8 * x_.pitch + 8 * n;
                    if (tb + g + 8 * h2 < t_end) {
                        if (8 * n + 2 * t + 1 < x_.pitch)
                            *reinterpret_cast<float2*>(a) = make_float2(x[n][2 * h2], x[n][2 * h2 + 1]);
                        else if (8 * n + 2 * t < x_.pitch)
                            *a = x[n][2 * h2];
                    }
                }
        }
        const float vmax = BPS == 2 ? fmaxf(me.vs[0], me.vs[BPS - 1]) : me.vs[0];
        if (__any_sync(0xffffffffu, raise) || vmax > vref) {
            // a power of two, so that vs / vref and the rescale are exact
            float fv = 1.f;
            if (vmax > vref) {
                const float nv = fminf(floor_pow2(vmax) * 2.f, 1.7014118e38f);
                fv = vref / nv;
                vref = nv;
            }
#pragma unroll
            for (int n = 0; n < NNT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mx = fmaxf(x[n][h], x[n][h + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float mn = fmaxf(m_h[n][h], mx);
                    const float al = m_h[n][h] == kNegInf ? 0.f : exp2_fast(m_h[n][h] - mn);
                    m_h[n][h] = mn;
                    l_h[n][h] *= al;
#pragma unroll
                    for (int j = 0; j < NM; ++j) {
                        acc[n][j][h] *= al * fv;
                        acc[n][j][h + 2] *= al * fv;
                    }
                }
        }
        const float wf0 = vref > 0.f ? me.vs[0] / vref * kWeightScale : 0.f;
        const float wf1 = BPS == 2 ? (vref > 0.f ? me.vs[BPS - 1] / vref * kWeightScale : 0.f) : wf0;
        uint32_t pb[NNT][2];
#pragma unroll
        for (int n = 0; n < NNT; ++n) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pr[e] = x[n][e] == kNegInf ? 0.f : exp2_fast(x[n][e] - m_h[n][e & 1]);
                l_h[n][e & 1] += pr[e];
            }
            pb[n][0] = transpose8x8(pack_f16(pr[0] * wf0, pr[1] * wf0));
            pb[n][1] = transpose8x8(pack_f16(pr[2] * wf1, pr[3] * wf1));
        }
        if (tail) {
            // whatever sits behind the context must not become 0 x NaN
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (tb + 2 * t + (j & 1) + 8 * (j >> 1) >= t_end)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        st.v[j][i] = 0u;
        }
        // output: m-tile 2 i + u of word i has rows (dims) D/8 g + 4 i + 2 u + {0, 1}
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t sel = u ? 0x7362u : 0x5140u;
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2(__byte_perm(st.v[0][i], st.v[1][i], sel), a0, a1);
                e4m3x4_to_f16x2(__byte_perm(st.v[2][i], st.v[3][i], sel), a2, a3);
#pragma unroll
                for (int n = 0; n < NNT; ++n)
                    mma_f16(acc[n][2 * i + u], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
        }
    };

    Step<D> sa, sb;
    Meta ma, mb;
    if (my_steps > 0)
        load(0, sa, ma);
    for (int it = 0; it < my_steps; it += 2) {
        if (it + 1 < my_steps)
            load(it + 1, sb, mb);
        compute(it, sa, ma);
        if (it + 1 < my_steps) {
            if (it + 2 < my_steps)
                load(it + 2, sa, ma);
            compute(it + 1, sb, mb);
        }
    }

    // this warp's state: sums over the lanes that share a head, O in V's units
    const float ov = vref * (1.f / kWeightScale);
#pragma unroll
    for (int n = 0; n < NNT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = l_h[n][h];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int r = 8 * n + 2 * t + h;
            if (r < nrows) {
                if (g == 0) {
                    sm_m[warp][r] = m_h[n][h];
                    sm_l[warp][r] = l;
                }
                float* o = sm_acc + (warp * RT + r) * PITCH + g * (D / 8);
#pragma unroll
                for (int j = 0; j < NM; ++j)
                    *reinterpret_cast<float2*>(o + 2 * j) =
                        make_float2(acc[n][j][h] * ov, acc[n][j][h + 2] * ov);
            }
        }
    __syncthreads();
    // merge of the warps, two dims a thread; warp i's weight is 2^(m_i - M)
    for (int i = threadIdx.x; i < nrows * (D / 2); i += kWarps * 32) {
        const int r = i / (D / 2);
        const int d = (i - r * (D / 2)) * 2;
        float M = sm_m[0][r];
#pragma unroll
        for (int k = 1; k < kWarps; ++k)
            M = fmaxf(M, sm_m[k][r]);
        float L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float mk = sm_m[k][r];
            const float f = mk == kNegInf ? 0.f : exp2_fast(mk - M);
            const float2 o = *reinterpret_cast<const float2*>(sm_acc + (k * RT + r) * PITCH + d);
            L += sm_l[k][r] * f;
            o0 += o.x * f;
            o1 += o.y * f;
        }
        if (direct) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + row_of(r) * D + d) =
                pack2(round_to<QT>(o0 * inv), round_to<QT>(o1 * inv));
            if constexpr (MODE == kWeights) {
                if (d == 0) {
                    if constexpr (BAL)
                        x_.whole[row_of(r)] = make_float2(M, inv);
                    else
                        sm_final[r] = make_float2(M, inv);
                }
            }
        } else {
            // BAL: rows of one partial lie together; else heads are apart
            int64_t row = BAL ? prow + r : prow + (int64_t)r * p.max_partitions;
            if constexpr (MODE == kShared)
                if (whole)
                    row = prow + row_of(r);
            if (d == 0) {
                p.ws_m[row] = M;
                p.ws_l[row] = L;
            }
            *reinterpret_cast<float2*>(p.ws_o + row * D + d) = make_float2(o0, o1);
        }
    }
    if constexpr (MODE == kWeights && !BAL) {
        // the scores come back from L2, where this CTA put them
        __syncthreads();
        const float* sc = x_.scores + (int64_t)(s * (int64_t)p.num_kv_heads + head) * x_.score_tokens * x_.pitch;
        float* w = x_.weights + s * x_.weights_seq + head * x_.weights_head;
        for (int tok = threadIdx.x; tok < t_end; tok += kWarps * 32)
            w[tok] += token_weight(sc + (int64_t)tok * x_.pitch, G, x_.pitch, sm_final);
    }
    // (the next item's q is filed once every warp is past the barrier above, its
    // states once every warp is past the one behind q)
    }
    if (beside)
        pdl_wait_primary();
}

// The partials of one item of n units from unit x on: which CTAs filed them.
struct Pieces {
    uint32_t c0, c1;           // the same CTA: it held the item whole
    __device__ __forceinline__ int64_t row(uint32_t c, int rt, int r) const
    {
        return (2 * (int64_t)c + (c == c0 ? 1 : 0)) * rt + r;
    }
};

__device__ __forceinline__ Pieces pieces_of(const Shares& sh, int64_t x, int n)
{
    Pieces pc;
    pc.c0 = sh.owner(x);
    pc.c1 = sh.owner(x + n - 1);
    if (pc.c0 < pc.c1 && sh.begin(pc.c0 + 1) - x <= kItemUnits)
        ++pc.c0;                               // (its share ended before the item's tokens)
    return pc;
}

// Merge of the partials of the equal shares: one warp per (sequence, query
// head).  Items that one CTA held whole are left alone (kShared: unless the row
// has a prefix); sequences without tokens (or with an unusable length) get zeros.
// kWeights: a row's maximum and 1 / sum are filed too.
constexpr int kReduceRows = kWarps;          // (scan_units wants kWarps warps)

template <int QT, int D, int MODE>
__global__ void __launch_bounds__(kReduceRows * 32)
    reduce_shares_kernel(const DecodeParams p, int64_t grid, int rows_per_partial, const DecodeExtra x_)
{
    constexpr int DPL = D / 32;
    __shared__ int sm_first[MODE == kShared ? 1 : kMaxBalanced + 1];
    const int* first = sm_first;               // units before each entry
    if constexpr (MODE == kShared)
        first = x_.first;                      // (filed by the kernel before)
    else
        scan_units<MODE>(p, sm_first, rows_per_partial, false);
    const int entries = MODE == kShared ? p.num_groups + p.num_seqs : p.num_seqs;
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)p.num_seqs * p.num_heads;
    const int64_t row = (int64_t)blockIdx.x * kReduceRows + (threadIdx.x >> 5);
    if (row >= rows)
        return;
    const int s = (int)(row / p.num_heads);
    const int hq = (int)(row - (int64_t)s * p.num_heads);
    const int head = hq / p.group;
    int r = hq - head * p.group;
    const int e = MODE == kShared ? p.num_groups + s : s;
    // kShared: the prefix's item (item number ipre of group gpre), if the row has one
    [[maybe_unused]] int npre = 0, rpre = 0, gpre = 0;
    [[maybe_unused]] int64_t ipre = 0;
    bool zero = false;
    if constexpr (MODE == kShared) {
        const int ctx = __ldg(p.context_lens + s);
        const int i = group_of(p, s);
        const Group g = group_at(p, i, false);
        bool bad;
        const int pre = own_begin(p, s, ctx, i, g, bad);
        zero = bad || ctx == 0;
        if (!bad && pre > 0) {
            const int tiles = tiles_of(p, g, rows_per_partial);
            const int rr = (s - g.begin) * p.group + r;
            npre = p.prefix_partition > 0 ? ceil_div_i(pre, p.prefix_partition)
                                          : ceil_div_i(pre, kUnit) + kItemUnits;
            rpre = rr % rows_per_partial;
            gpre = i;
            ipre = (int64_t)head * tiles + rr / rows_per_partial;
            // a table that differs inside the prefix: the first member's is used
            if (hq == 0 && p.dev_err != nullptr) {
                const int32_t* a = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
                const int32_t* b = p.block_tables + (int64_t)g.begin * p.max_blocks_per_seq;
                for (int k = lane; k < pre / p.block_size; k += 32)
                    if (__ldg(a + k) != __ldg(b + k))
                        flag_error(p.dev_err, PKV_DEVERR_PREFIX);
            }
        }
    }
    float acc[DPL];
#pragma unroll
    for (int d = 0; d < DPL; ++d)
        acc[d] = 0.f;
    float L = 0.f;
    int n = 0;
    Shares sh;
    if constexpr (MODE != kShared) {
        n = first[e + 1] - first[e];
        sh = shares_of(p, first[entries], grid);
        zero = n == 0;
    }
    pdl_wait_primary();
    pdl_launch_dependents();
    if constexpr (MODE == kShared) {
        n = first[e + 1] - first[e];
        sh = shares_of(p, first[entries], grid);
    }
    auto add = [&](int64_t pr, float M) {
        const float m = p.ws_m[pr];
        const float f = m == kNegInf ? 0.f : exp2_fast(m - M);
        L += f * p.ws_l[pr];
        const float* o = p.ws_o + pr * D + lane * DPL;
        if constexpr (DPL == 4) {
            const float4 v = *reinterpret_cast<const float4*>(o);
            acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(o);
            acc[0] += f * v.x, acc[1] += f * v.y;
        }
    };
    if (!zero) {
        Pieces own{0, 0}, pre{0, 0};
        const bool has_own = n > 0;
        if (has_own)
            own = pieces_of(sh, (int64_t)first[e] * p.num_kv_heads + (int64_t)head * n, n);
        // (prefixes with a kernel of their own: npre runs, each with its rows)
        const bool runs = MODE == kShared && p.prefix_partition > 0;
        if (npre > 0 && !runs)
            pre = pieces_of(sh, (int64_t)first[gpre] * p.num_kv_heads + ipre * npre, npre);
        if (npre == 0 && own.c0 == own.c1)
            return;
        // rows of whole items: behind the pieces
        const int64_t wown = 2 * grid * rows_per_partial + row;
        const int64_t wpre = wown + rows;
        float M = kNegInf;
        auto most = [&](const Pieces& pc, int rr, int64_t whole) {
            if (pc.c0 == pc.c1) {
                M = fmaxf(M, p.ws_m[whole]);
                return;
            }
            for (uint32_t c = pc.c0 + lane; c <= pc.c1; c += 32)
                M = fmaxf(M, p.ws_m[pc.row(c, rows_per_partial, rr)]);
        };
        auto sum = [&](const Pieces& pc, int rr, int64_t whole) {
            if (pc.c0 == pc.c1) {
                add(whole, M);
                return;
            }
#pragma unroll 4
            for (uint32_t c = pc.c0; c <= pc.c1; ++c)
                add(pc.row(c, rows_per_partial, rr), M);
        };
        if (runs)
            for (int i = lane; i < npre; i += 32)
                M = fmaxf(M, p.ws_m[wpre + i * rows]);
        else if (npre > 0)
            most(pre, rpre, wpre);
        if (has_own)
            most(own, r, wown);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (runs) {
#pragma unroll 4
            for (int i = 0; i < npre; ++i)
                add(wpre + i * rows, M);
        } else if (npre > 0) {
            sum(pre, rpre, wpre);
        }
        if (has_own)
            sum(own, r, wown);
        if constexpr (MODE == kWeights)
            if (lane == 0)
                x_.whole[row] = make_float2(M, L == 0.f ? 0.f : 1.f / L);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + row * D + lane * DPL;
#pragma unroll
    for (int d = 0; d < DPL; d += 2)
        *reinterpret_cast<uint32_t*>(out + d) =
            pack2(round_to<QT>(acc[d] * inv), round_to<QT>(acc[d + 1] * inv));
}

// The kernels here start while what precedes them in the stream ends, and wait
// for it before they read anything it may write.
template <class... Args>
cudaError_t launch_early_smem(void (*kern)(Args...), int64_t ctas, int threads, size_t smem,
                              cudaStream_t stream, Args... args)
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

template <class... Args>
cudaError_t launch_early(void (*kern)(Args...), int64_t ctas, int threads, cudaStream_t stream,
                         Args... args)
{
    return launch_early_smem(kern, ctas, threads, 0, stream, args...);
}

}  // namespace dsk
}  // namespace pkv
