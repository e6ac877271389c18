// prefill_scaled_kernel.cuh -- causal attention of prompts and chunks over an E4M3
// cache with a scale per block and KV head, on the 5th-generation tensor cores: the
// kernel of prefill_scaled.cu, and (PREFIX) of decode_scaled_prefix.cu, where the
// rows are the query heads of a group's members, which all see a run of the keys
// that the group shares.
//
// Row j of sequence s, at position p = context_lens[s] - n_s + j, attends to
// tokens t <= p of values code * scale.
//
// One CTA = two query tiles (a, b) of 128 (token, head) rows of one (sequence,
// KV head), as in prefill_ws.cu, whose schedule this kernel keeps; new is how
// operands come about.  Four warpgroups share the registers by setmaxnreg:
//   * warps 12-15 (load and convert): walk the block table, copy codes one slot
//     ahead, turn them into fp16 and store them into the 128-byte-swizzled
//     operand tiles of a ring, slot j = K(j) and V(j - 1).  Codes cross HBM and
//     L2 at half a 16-bit cache's traffic.
//     The scale's power of two goes into the conversion: a block's K becomes
//     code * 2^(e - eref + 7) with 2^eref the power of two of the CTA's largest
//     ks (V alike), which fp16 holds exactly down to 2^-22 of the largest; what
//     a block further down loses is at most 2^-31 of the largest scale.  So one
//     factor serves all scores, one all outputs, and while the scales are powers
//     of two, as the append makes them, the softmax does not know about blocks.
//     Otherwise the rest of each scale, in [1, 2), multiplies its block's scores
//     and weights there, in fp32 (rounding it into the fp16 factor moved all
//     scores of a block by up to 2^-11); chunks then take 281 us instead of 226,
//     prompts 198 instead of 174.
//   * warps 8 and 10 (one issuing thread each): O_w += P_w(j-1) V(j-1), then
//     S_w(j) = Q_w K(j)^T, taking turns by slot.
//   * warps 0-3 and 4-7: softmax, one thread per row.  q is fp16 per row times
//     a power of two (bf16 values fit without loss); the weights are fp16, so
//     P V is one product for both types: each is off by at most 2^-11 of itself,
//     or by 2^-31 where it is a subnormal.  For that they are stored times 2^6
//     (at most 2^14 with the maximum's lag of 2^8), which the sums carry too and
//     O / l leaves out; at 2^0 a flat tail 2^-25 below one large weight, however
//     long, became nothing.
// NaN codes of V: a weight of 0 times NaN would reach rows that may not see the
// token, so the converter stores 0 and notes the first position of a NaN per
// output column; rows at or past it get NaN there.
// Every wait is bounded, as in prefill_ws.cu.
//
// Bound by the chain of a slot (scores, softmax, product: ~3,500 cycles for 32
// products of 128 x 128 x 16, of which the tensor core is busy ~2,700), and by
// ~8,000 cycles to a CTA's first product. Measured: 4 chunks of 512 tokens after
// 1,024..4,096 (64 heads over 8, D 128, block 16) 226 us, 1,010 TFLOP/s; 8 prompts
// of 512..2,048 tokens (32 heads) 174 us, 568 TFLOP/s. (Scales of any value cost
// 1.3 % of that: 223 and 172 us without.) Beside it, on the way, the chunks:
// codes waited for as they are read 391 us, kept in registers 263-313, conversion
// two vectors at a time 255, weights handed over whole 259, on the half 246.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pkv_common.cuh"
#include "scaled_internal.h"
#include "tc_common.cuh"

namespace pkv {
namespace pfs {

using namespace tc;

constexpr int kRows = 128;             // rows per query tile = tensor-memory lanes
constexpr int kKeys = 128;             // keys per K/V tile
constexpr int kMmaWarp = 8;            // issues query tile a's products; warp 10 b's
constexpr int kConvWarp = 12;          // first of the four converting warps
constexpr int kConvWarps = 4;
constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128;
constexpr int kSoftmaxRegs = 184;
constexpr int kMmaRegs = 48;
constexpr int kConvRegs = 96;
static_assert(2 * kSoftmaxRegs + kMmaRegs + kConvRegs <= 4 * kLaunchRegs, "register split");
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kBatch = 4;             // vectors a converting lane has in hand
constexpr float kUnit = 128.f;         // fp16 value of a code at the reference scale
constexpr float kRaise = 8.f;          // log2: how far a score may pass the running maximum
constexpr float kWeightExp = 6.f;      // log2 of the weight at the running maximum

template <int D>
struct Layout {
    static constexpr int NP = D / 64;                  // 64-dim panels
    static constexpr int ST = D == 128 ? 2 : 4;        // slots of the ring
    static constexpr int QB = NP * kRows * 128;        // one query tile
    static constexpr int KVB = NP * kKeys * 128;       // one K or V tile
    static constexpr int q = 0;
    static constexpr int slot = q + 2 * QB;            // [ST][K, V]
    static constexpr int SLOT = 2 * KVB;
    static constexpr int raw = slot + ST * SLOT;       // codes of one slot: K, V
    static constexpr int bytes = raw + 2 * kKeys * D;
    static constexpr int alloc = bytes + 1024;         // room to align the base
    static constexpr uint32_t cols = 512;
};

template <int ST>
struct Bars {
    uint64_t q_full[2];      // 128 arrivals: the group's Q rows are in shared memory
    uint64_t s_full[2];      // commit: S_w(kt) (and every earlier product of w) done
    uint64_t p_most[2];      // 128 arrivals: three quarters of P_w(kt) written
    uint64_t p_full[2];      // 128 arrivals: all of it
    uint64_t o_full[2];      // commit: the last O_w += P_w V done
    uint64_t full[ST];       // one arrival per converting warp: slot j is stored
    uint64_t empty[ST];      // one arrival per issuing warp: slot j no longer read
    uint64_t issued[2];      // issuing thread w has queued its products of slot j
    uint64_t drain[2];       // commit: every product issued by warp w done
};

__device__ __forceinline__ bool aborted(const int* flag)
{
    return *reinterpret_cast<const volatile int*>(flag) != 0;
}

__device__ __forceinline__ void set_abort(int* flag, int32_t* dev_err)
{
    *reinterpret_cast<volatile int*>(flag) = 1;
    flag_error(dev_err, PKV_DEVERR_TIMEOUT);
}

// Bounded wait by one thread; gives up early once another role has aborted.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, int* flag,
                                         int32_t* dev_err)
{
    WaitClock clock;
    for (uint32_t i = 0; i < kSpin; ++i) {
        if (try_wait(bar, parity))
            return true;
        if (aborted(flag))
            return false;
        if (clock.expired(i))
            break;
    }
    set_abort(flag, dev_err);
    return false;
}

// The same by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int* flag,
                                          int32_t* dev_err)
{
    bool ok = false;
    WaitClock clock;
    for (uint32_t i = 0; i < kSpin; ++i) {
        if (try_wait(bar, parity)) {
            ok = true;
            break;
        }
        if (aborted(flag) || clock.expired(i))
            break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok)
        set_abort(flag, dev_err);
    return ok;
}

// A normal scale = power_of(scale) * rest_of(scale), a power of two and a number
// in [1, 2).
__device__ __forceinline__ float power_of(float scale)
{
    return __uint_as_float(__float_as_uint(scale) & 0x7f800000u);
}
__device__ __forceinline__ float rest_of(float scale)
{
    return __uint_as_float((__float_as_uint(scale) & 0x007fffffu) | 0x3f800000u);
}

// The power of two of the scale whose bits these are, a normal number.
__device__ __forceinline__ float reference_of(const uint32_t* bits)
{
    const uint32_t e = *reinterpret_cast<const volatile uint32_t*>(bits) & 0x7f800000u;
    return __uint_as_float(min(max(e, 0x00800000u), 0x7f000000u));
}

// code * f for 16 codes, as 16 fp16 values (f: the factor in both halves).
__device__ __forceinline__ void convert16(const uint4& c, uint32_t f, uint4& lo, uint4& hi)
{
    auto mul = [f](uint32_t h) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(f));
        return r;
    };
    uint32_t a, b;
    e4m3x4_to_f16x2(c.x, a, b);
    lo.x = mul(a), lo.y = mul(b);
    e4m3x4_to_f16x2(c.y, a, b);
    lo.z = mul(a), lo.w = mul(b);
    e4m3x4_to_f16x2(c.z, a, b);
    hi.x = mul(a), hi.y = mul(b);
    e4m3x4_to_f16x2(c.w, a, b);
    hi.z = mul(a), hi.w = mul(b);
}

// Larger magnitudes of two words of bf16 values (NaN gives way to a number).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
    return r;
}

// Non-zero where a byte of w is a NaN code (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// w with its NaN codes cleared; each one's column gets the smallest position.
static __device__ __noinline__ uint32_t note_nans(uint32_t w, int* nan_pos, int* any_nan, int position)
{
    const uint32_t nc = nan_codes(w);
    for (int b = 0; b < 4; ++b)
        if (nc & (0x80u << (8 * b))) {
            atomicMin(nan_pos + b, position);
            *reinterpret_cast<volatile int*>(any_nan) = 1;
            w &= ~(0xffu << (8 * b));
        }
    return w;
}

// Zero `rows` tokens' outputs of one KV head.
static __device__ __noinline__ void zero_rows(uint16_t* out, int64_t token_stride, int rows, int row_elems)
{
    for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5)
        for (int i = (threadIdx.x & 31) * 2; i < row_elems; i += 64)
            *reinterpret_cast<uint32_t*>(out + r * token_stride + i) = 0u;
}

__device__ __forceinline__ void st_shared16(uint32_t a, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a));
    return r;
}

// A group's rows: sequences [begin, begin + members), whose tables' first `prefix`
// tokens are one.
struct PrefixRows {
    int begin, members, prefix;
};

__device__ __forceinline__ PrefixRows prefix_rows(const PrefixParams& x, int i, int num_seqs, int block_size)
{
    PrefixRows g;
    g.begin = __ldg(x.grp_begin + i);
    const int end = __ldg(x.grp_begin + i + 1);
    const int blocks = __ldg(x.grp_prefix_blocks + i);
    g.members = min(end - g.begin, x.max_group_size);
    g.prefix = blocks * block_size;
    if (g.begin < 0 || end < g.begin || end > num_seqs || blocks < 0 || blocks > x.max_prefix_blocks)
        g.members = g.prefix = 0;              // (flagged by the kernel for the own tokens)
    return g;
}

template <int QT_, int D, int BS, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_scaled_kernel(const __grid_constant__ ScaledPrefillParams sp, const __grid_constant__ PrefixParams px)
{
    using L = Layout<D>;
    constexpr int CT = QT_;                    // type of q and out
    constexpr int ST = L::ST;
    constexpr int NB = kKeys / BS;             // blocks per K/V tile
    // tiles whose scales' rests are kept: the converting warps write tile j's once
    // slot j - ST is free, so tile j - ST may still be in the softmax
    constexpr int NR = ST < 4 ? 4 : 8;
    static_assert(NR > ST && (NR & (NR - 1)) == 0, "ring of the rests");
    const PrefillParams& p = sp.p;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) Bars<ST> bars;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    __shared__ uint32_t ref_bits[2];           // largest ks, vs of the CTA's blocks
    __shared__ int any_rest;                   // some scale is no power of two (PREFIX: or a block is bad)
    __shared__ float rests[NR][2][NB];         // then: the rests of ks, vs by tile (PREFIX: bad blocks' ks 0)
    __shared__ int nan_pos[D];                 // first key whose V is NaN in this column
    __shared__ int any_nan;
    __shared__ int64_t first_rows[2];          // where the query tiles' outputs start

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int G = p.group;
    if constexpr (PREFIX)
        pdl_launch_dependents();               // (the shares of the own tokens, beside this)
    const int QT = kRows / G;                  // new tokens per query tile
    const int span = 2 * QT;                   // new tokens per CTA
    const int ntiles = ((PREFIX ? px.max_group_size : p.max_q_len) + span - 1) / span;
    const int64_t units = (int64_t)(PREFIX ? px.num_groups : p.num_seqs) * p.num_kv_heads;
    int64_t idx = blockIdx.x;
    [[maybe_unused]] int split = 0;            // PREFIX: which run of the keys
    if constexpr (PREFIX) {
        split = (int)(idx / (units * ntiles));
        idx -= split * units * ntiles;
    }
    const int tile = ntiles - 1 - (int)(idx / units);      // heaviest tiles first
    int s = (int)((idx % units) / p.num_kv_heads);
    const int g = (int)(idx % p.num_kv_heads);
    const int j0 = tile * span;
    uint16_t* out = reinterpret_cast<uint16_t*>(p.out);
    int cu0, n, ctx, skip = 0;
    if constexpr (PREFIX) {
        const PrefixRows gr = prefix_rows(px, s, p.num_seqs, BS);
        s = cu0 = gr.begin;
        n = gr.members;
        skip = split * px.run;
        ctx = min(gr.prefix - skip, px.run);   // keys of this CTA
        if (j0 >= n || ctx <= 0)
            return;
    } else {
        cu0 = __ldg(p.cu_seqlens_q + s);
        const int cu1 = __ldg(p.cu_seqlens_q + s + 1);
        n = cu1 - cu0;
        if (cu0 < 0 || cu1 < cu0 || cu1 > p.total_q) {
            if (tid == 0 && tile == 0 && g == 0)
                flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
            return;
        }
        if (j0 >= n)
            return;
        ctx = __ldg(p.context_lens + s);
    }
    auto row_off = [&](int j, int h) -> int64_t {     // element offset of (token j, head h)
        return ((int64_t)(cu0 + j) * p.num_heads + g * G + h) * D;
    };
    if (!PREFIX && (ctx < n || ctx > p.max_context_len || n > p.max_q_len ||
                    (ctx + BS - 1) / BS > p.max_blocks_per_seq)) {
        if (tid == 0 && j0 == 0 && g == 0)
            flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
        // zero rows; the last tile's CTA takes the rows no tile covers
        const int last = tile == ntiles - 1 ? n : min(n, j0 + span);
        zero_rows(out + row_off(j0, 0), (int64_t)p.num_heads * D, last - j0, G * D);
        return;
    }
    // the two query tiles: tokens [j0 + w QT, j0 + w QT + ntok_w)
    const int ntok0 = min(QT, n - j0);
    const int ntok1 = max(0, min(QT, n - j0 - QT));
    // position of tile a's first token (PREFIX: of every row's last key)
    const int pos00 = PREFIX ? ctx - 1 : ctx - n + j0;
    const int pos01 = PREFIX ? ctx - 1 : pos00 + QT;
    const int nkv0 = ((PREFIX ? ctx : pos00 + ntok0) + kKeys - 1) / kKeys;
    const int nkv1 = ntok1 > 0 ? ((PREFIX ? ctx : pos01 + ntok1) + kKeys - 1) / kKeys : 0;
    const int nk = max(nkv0, nkv1);            // K/V tiles the CTA loads
    const int kv_end = PREFIX ? ctx : (ntok1 > 0 ? pos01 + ntok1 : pos00 + ntok0);
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks_per_seq + skip / BS;
    const float2* scales = reinterpret_cast<const float2*>(sp.scales);

    const uint32_t raw = s_addr(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    // the scan of the scales below: its first ids (of up to 512 blocks) are asked
    // for here, the scales when the ids have come
    const int nblocks = (kv_end + BS - 1) / BS;
    const int id_first = tid < nblocks ? __ldg(table + tid) : 0;

    if (tid == 0) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            bar_init(s_addr(&bars.q_full[w]), kRows);
            bar_init(s_addr(&bars.s_full[w]), 1);
            bar_init(s_addr(&bars.p_most[w]), kRows);
            bar_init(s_addr(&bars.p_full[w]), kRows);
            bar_init(s_addr(&bars.o_full[w]), 1);
        }
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            bar_init(s_addr(&bars.full[i]), kConvWarps);
            bar_init(s_addr(&bars.empty[i]), ntok1 > 0 ? 2 : 1);
        }
        bar_init(s_addr(&bars.issued[0]), 1);
        bar_init(s_addr(&bars.issued[1]), 1);
        bar_init(s_addr(&bars.drain[0]), 1);
        bar_init(s_addr(&bars.drain[1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_flag = 0;
        any_nan = 0;
        any_rest = 0;
        first_rows[0] = row_off(j0, 0);
        first_rows[1] = row_off(j0 + QT, 0);
        ref_bits[0] = ref_bits[1] = 0u;
    }
    if (tid < D)
        nan_pos[tid] = 0x7fffffff;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         s_addr(&tmem_holder)),
                     "r"(L::cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;
    auto block_ok = [&](int phys) { return phys >= 0 && (int64_t)phys < p.num_blocks; };
    // (PREFIX: the keys of such a block are masked by the form with rests)
    auto bad_block = [&]() {
        flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);
        if constexpr (PREFIX)
            *reinterpret_cast<volatile int*>(&any_rest) = 1;
    };
    float2 sc_first = make_float2(0.f, 0.f);
    if (tid < nblocks) {
        if (block_ok(id_first))
            sc_first = __ldg(scales + (int64_t)id_first * p.num_kv_heads + g);
        else
            bad_block();
    }
    // ---------------- what can start before the scales are known ----------------
    // Softmax warps: q, in its own type.  A warp copies its 32 rows side by side
    // into their places; rows past the tile's are zero.
    constexpr int LPR = D / 8;                 // lanes to a row
    constexpr int RPA = 32 / LPR;              // rows to an access
    constexpr int NA = 32 / RPA;               // accesses
    const int qw = (warp >> 2) & 1;            // the warp's query tile
    const int nrows = (qw ? ntok1 : ntok0) * G;
    const int row0 = (warp & 3) * 32;
    const uint32_t qs = sb + L::q + qw * L::QB;
    // offset of row rr of the tile from its first: rr / G tokens on, by a
    // multiplication (exact: 128 rows, G <= 128)
    const uint32_t by_g = ((1u << 24) + G - 1) / G;
    const int64_t first_row = row_off(j0 + qw * QT, 0);
    auto row_at = [&](int rr) -> int64_t {
        return (int64_t)((rr * by_g) >> 24) * ((p.num_heads - G) * D) + rr * D;
    };
    if (warp < 8 && nrows > 0) {
        const int c = lane % LPR;
#pragma unroll 4
        for (int i = 0; i < NA; ++i) {
            const int rr = row0 + i * RPA + lane / LPR;
            const bool ok = rr < nrows;
            cp16z(qs + panel_off(rr, c, kRows),
                  reinterpret_cast<const uint16_t*>(p.q) + (ok ? first_row + row_at(rr) + c * 8 : 0), ok);
        }
        cp_async_commit();
    }
    // Converting warps: the first tile's codes.
    // A lane's vector i (16 codes) of a tile: row group i / NP (32 rows: 8 to a
    // warp), 64-dim panel i % NP, row `rsub` and quarter `c4` of the panel's
    // row.  Eight lanes write two rows' chunks of one parity, which the
    // swizzle sends to eight different banks.
    constexpr int NP = L::NP;
    constexpr int NV = NP * 4;
    static_assert(NV % kBatch == 0, "whole batches");
    const int cw = warp - kConvWarp;
    const int c4 = lane & 3;
    const int rsub = cw * 8 + (lane >> 2);
    const int64_t tile_bytes = (int64_t)BS * D;
    const unsigned char* kbase = reinterpret_cast<const unsigned char*>(p.k_cache) + g * tile_bytes;
    const unsigned char* vbase = reinterpret_cast<const unsigned char*>(p.v_cache) + g * tile_bytes;
    const int64_t stride = p.num_kv_heads * tile_bytes;
    // lane i < NB: block i of a K/V tile: its id (-1: none), its factors.  The
    // id is asked for three tiles ahead, the scales two, so that neither
    // load is waited for.
    auto id_of = [&](int kt) -> int {
        const int tok = kt * kKeys + lane * BS;
        return kt < nk && lane < NB && tok < kv_end ? __ldg(table + tok / BS) : -1;
    };
    // Codes travel through a staging area in which every thread has places of
    // its own (vector i at i * 128 + thread): copied asynchronously one slot
    // ahead, read back and converted by the thread that asked for them, so
    // no barrier stands between.
    const uint32_t raw_k = sb + L::raw + (tid - kConvWarp * 32) * 16;
    const uint32_t raw_v = raw_k + kKeys * D;
    constexpr int PITCH = 32 * kConvWarps * 16;
    // start the copies of vectors i0 ... of a tile whose first key is `first`
    auto fetch = [&](uint32_t dst, const unsigned char* base, int id, int i0, int first, int end) {
#pragma unroll
        for (int u = 0; u < kBatch; u += NP) {
            const int row = (i0 + u) / NP * 32 + rsub;
            const int phys = __shfl_sync(0xffffffffu, id, row / BS);
            const bool ok = block_ok(phys) && first + row < end;
            const unsigned char* src = base + (ok ? phys * stride + (row % BS) * D + c4 * 16 : 0);
#pragma unroll
            for (int q = 0; q < NP; ++q)
                cp16z(dst + (i0 + u + q) * PITCH, src + q * 64, ok);
        }
    };
    int id0 = -1, id1 = -1, id2 = -1;          // tiles j, j + 1, j + 2
    if (warp >= kConvWarp) {
        id0 = id_of(0);
        id1 = id_of(1);
        id2 = id_of(2);
#pragma unroll
        for (int i0 = 0; i0 < NV; i0 += kBatch)
            fetch(raw_k, kbase, id0, i0, 0, kv_end);
        cp_async_commit();
    }
    // the largest scales of the CTA's blocks (positive floats order as their
    // bits; anything else counts as 0)
    {
        uint32_t mk = sc_first.x > 0.f ? __float_as_uint(sc_first.x) : 0u;
        uint32_t mv = sc_first.y > 0.f ? __float_as_uint(sc_first.y) : 0u;
        uint32_t rest = mk | mv;
        for (int b = tid + kThreads; b < nblocks; b += kThreads) {
            const int phys = __ldg(table + b);
            if (!block_ok(phys)) {
                bad_block();
                continue;
            }
            const float2 sc = __ldg(scales + (int64_t)phys * p.num_kv_heads + g);
            const uint32_t ks = sc.x > 0.f ? __float_as_uint(sc.x) : 0u;
            const uint32_t vs = sc.y > 0.f ? __float_as_uint(sc.y) : 0u;
            mk = max(mk, ks);
            mv = max(mv, vs);
            rest |= ks | vs;
        }
        mk = __reduce_max_sync(0xffffffffu, mk);
        mv = __reduce_max_sync(0xffffffffu, mv);
        if (lane == 0) {
            atomicMax(&ref_bits[0], mk);
            atomicMax(&ref_bits[1], mv);
        }
        if (rest & 0x007fffffu)
            *reinterpret_cast<volatile int*>(&any_rest) = 1;
    }
    // The converting warps wait for everybody's part; the others read the maxima
    // when the first slot, which those warps fill, has come to them.
    // (They give their registers up before that: the softmax warps' q waits for
    // the registers.)
    if (warp >= kConvWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    } else {
        asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
    }

    if (warp < 8) {
        // ---------------- softmax of query tile w ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int w = qw;
        const int r = tid & (kRows - 1);
        if (nrows > 0) {
            const int pos0 = w ? pos01 : pos00;
            const int nkv = w ? nkv1 : nkv0;
            // fp16 q takes part as it is; bf16 q is scaled per row to at most 2^14
            // in size, every thread turning its own row into fp16 in place.
            // (Loops kept short: code that runs once is fetched at a few bytes a
            // cycle; all of this unrolled took 11,000 cycles.)
            float qk;                                  // this row's factor of the scores
            {
                cp_async_wait<0>();
                __syncwarp();
                float mx = 0.f;
                if constexpr (CT == kBF16) {
                    uint32_t m2 = 0u;
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = lds16(qs + panel_off(r, c, kRows));
                        m2 = max_abs2(max_abs2(m2, v.x), v.y);
                        m2 = max_abs2(max_abs2(m2, v.z), v.w);
                    }
                    const float2 mm = unpack2<CT>(m2);
                    mx = fmaxf(mm.x, mm.y);
                }
                // 2^13 / 2^floor(log2 mx), kept where it and its inverse are normal
                float up = 1.f;
                if (mx > 0.f && mx < __builtin_huge_valf())
                    up = __uint_as_float(
                        (uint32_t)min(max(267 - (int)(__float_as_uint(mx) >> 23), 7), 247) << 23);
                // the factor of the scores stays positive: the scale's sign (or a
                // scale of 0) goes into q
                const float sign = p.qk_scale_log2 < 0.f ? -1.f : (p.qk_scale_log2 == 0.f ? 0.f : 1.f);
                qk = sign == 0.f ? 0.f : fabsf(p.qk_scale_log2) * (1.f / up) * (1.f / kUnit);
                up *= sign;
                if (up != 1.f || CT == kBF16)
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint32_t at = qs + panel_off(r, c, kRows);
                    const uint4 v = lds16(at);
                    const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = unpack2<CT>(w4[e]);
                        h[e] = pack_rn<kF16>(x.x * up, x.y * up);
                    }
                    st_shared16(at, make_uint4(h[0], h[1], h[2], h[3]));
                }
                async_proxy_fence();
                bar_arrive(s_addr(&bars.q_full[w]));
            }
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t t_s = tmem + lanes + 128u * w;
            const uint32_t t_o = tmem + lanes + 256u + (uint32_t)D * w;
            const int pos = PREFIX ? pos0 : pos0 + r / G;      // this row's position
            float m_run = kNegInf;                     // running max of the scaled logits
            float l_run = 0.f;
            // The tiles' loop has two forms that differ in the rests of the scales
            // only: with a branch for them inside one loop the chunks took 239-264
            // us instead of 227.  (Its body keeps the loop's own indentation.)
            bool alive = wait_warp(s_addr(&bars.s_full[w]), 0, &abort_flag, p.dev_err);
            // K's reference and the kind of the scales come with the first keys.
            // (The factor is at least 1e-30, where the scores of such small keys
            // vanish all the same: 0 times a masked key's -inf would be NaN.)
            qk = fmaxf(qk * reference_of(&ref_bits[0]), 1e-30f);
            auto tiles = [&](auto with_rests) {
            constexpr bool kRests = decltype(with_rests)::value;
            for (int kt = 0; kt < nkv; ++kt) {
                if (kt > 0 && !wait_warp(s_addr(&bars.s_full[w]), kt & 1, &abort_flag, p.dev_err)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                float x[kKeys];
#pragma unroll
                for (int c0 = 0; c0 < kKeys; c0 += 16)
                    tmem_ld16(t_s + c0, *reinterpret_cast<uint32_t(*)[16]>(x + c0));
                tmem_wait_ld();
                // causal mask only where some key passes some row's position
                if (kt * kKeys + kKeys - 1 > pos0) {
                    const int lim = pos - kt * kKeys;      // the last key the row sees
#pragma unroll
                    for (int j0 = 0; j0 < kKeys; j0 += 32) {
                        const int n = lim - j0 + 1;
                        const uint32_t bits = n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            x[j0 + j] = (bits >> j) & 1u ? x[j0 + j] : kNegInf;
                    }
                }
                [[maybe_unused]] const volatile float* rest = &rests[kt & (NR - 1)][0][0];
                if constexpr (kRests) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float f = rest[b];
#pragma unroll
                        for (int j = 0; j < BS; ++j)
                            if constexpr (PREFIX)
                                x[b * BS + j] = f == 0.f ? kNegInf : x[b * BS + j] * f;
                            else
                                x[b * BS + j] *= f;
                    }
                }
                // row max: eight independent chains of three-input maxima
                float mc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mc[i] = fmaxf(x[2 * i], x[2 * i + 1]);
#pragma unroll
                for (int j = 16; j < kKeys; j += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mc[i] = fmax3(mc[i], x[j + 2 * i], x[j + 2 * i + 1]);
                const float mx = fmax3(fmax3(mc[0], mc[1], mc[2]), fmax3(mc[3], mc[4], mc[5]),
                                       fmaxf(mc[6], mc[7]));
                const float m_cand = fmaxf(m_run, mx * qk);
                const bool raise = m_cand > m_run + kRaise;
                const float m_new = raise ? m_cand : m_run;
                const float alpha = raise ? fast_exp2(m_run - m_new) : 1.f;   // 0 on the first tile
                if (kt > 0 && __any_sync(0xffffffffu, raise)) {
                    // O_w += P_w(kt-1) V(kt-1) has completed: the commit behind
                    // S_w(kt) covers every earlier product
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t r16[16];              // (x stays live: few registers)
                        tmem_ld16(t_o + c0, r16);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            r16[j] = __float_as_uint(__uint_as_float(r16[j]) * alpha);
                        tmem_st16(t_o + c0, r16);
                    }
                }
                m_run = m_new;
                const float2 qk2 = make_float2(qk, qk);
                // (PREFIX: no key of the tiles so far is there: -inf + 0 is no weight)
                const float nm = PREFIX && kRests && m_new == kNegInf ? 0.f : kWeightExp - m_new;
                const float2 nm2 = make_float2(nm, nm);
                float2 ls[4] = {};                     // four pairs of partial sums
                // P over S: 16 keys as 8 columns of fp16 pairs at the start of
                // those keys' own 16 columns
#pragma unroll
                for (int c0 = 0; c0 < kKeys; c0 += 16) {
                    uint32_t hi[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // 2^6 exp2(s qk - m); a masked key (-inf) gives 0
                        const float2 t = ffma2(make_float2(x[c0 + 2 * e], x[c0 + 2 * e + 1]), qk2, nm2);
                        float2 pp = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                        ls[e & 3] = fadd2(ls[e & 3], pp);
                        if constexpr (kRests) {
                            const float f = rest[NB + (c0 + 2 * e) / BS];
                            pp.x *= f, pp.y *= f;
                        }
                        hi[e] = pack_rn<kF16>(pp.x, pp.y);
                    }
                    tmem_st8(t_s + c0, hi);
                    if (c0 + 16 == kKeys / 4 * 3) {
                        // the product may start on the first three quarters
                        tmem_wait_st();
                        tc_fence_before();
                        bar_arrive(s_addr(&bars.p_most[w]));
                    }
                }
                const float lsum = ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) +
                                   ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
                tmem_wait_st();
                l_run = l_run * alpha + lsum;
                tc_fence_before();
                bar_arrive(s_addr(&bars.p_full[w]));
            }
            };
            if (alive) {
                if (__builtin_expect(*reinterpret_cast<volatile int*>(&any_rest) == 0, 1))
                    tiles(std::false_type{});
                else
                    tiles(std::true_type{});
            }
            if (alive)
                alive = wait_warp(s_addr(&bars.o_full[w]), 0, &abort_flag, p.dev_err);
            if (alive) {
                if constexpr (PREFIX) {
                    // the row's partial: weights and sum without the 2^6
                    tc_fence_after();
                    const float unit = reference_of(&ref_bits[1]) * (1.f / kUnit) * exp2f(-kWeightExp);
                    const bool nans = *reinterpret_cast<volatile int*>(&any_nan) != 0;
                    // (fetched here: what stays in registers around the loop is spilled)
                    const int64_t row = px.first_row + split * (int64_t)p.num_seqs * p.num_heads +
                                        *reinterpret_cast<volatile int64_t*>(&first_rows[w]) / D +
                                        (int64_t)((r * by_g) >> 24) * (p.num_heads - G) + r;
                    if (r < nrows) {
                        px.ws_m[row] = m_run;
                        px.ws_l[row] = l_run * exp2f(-kWeightExp);
                    }
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t o16[16];
                        tmem_ld16(t_o + c0, o16);
                        tmem_wait_ld();
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[e] = __uint_as_float(o16[e]) * unit;
                        if (nans)
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (*reinterpret_cast<volatile int*>(&nan_pos[c0 + e]) <= pos)
                                    v[e] = __uint_as_float(0x7fc00000u);
                        if (r < nrows)
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<float4*>(px.ws_o + row * D + c0 + e) =
                                    make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                } else {
                // epilogue: O / l for this thread's row
                tc_fence_after();
                const float inv = l_run > 0.f ? (1.f / l_run) * (reference_of(&ref_bits[1]) * (1.f / kUnit))
                                              : (l_run == 0.f ? 0.f : l_run);
                const bool nans = *reinterpret_cast<volatile int*>(&any_nan) != 0;
                // through shared memory (this tile's q, which every product has
                // read), so that the warp writes its rows side by side
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o32[32];
                    tmem_ld16(t_o + c0, *reinterpret_cast<uint32_t(*)[16]>(o32));
                    tmem_ld16(t_o + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(o32 + 16));
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o4[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o4[e] = pack_rn<CT>(__uint_as_float(o32[8 * c + 2 * e]) * inv,
                                                __uint_as_float(o32[8 * c + 2 * e + 1]) * inv);
                        st_shared16(qs + panel_off(r, c0 / 8 + c, kRows),
                                    make_uint4(o4[0], o4[1], o4[2], o4[3]));
                    }
                }
                if (nans) {
                    // columns in which a key that the row sees has NaN
#pragma unroll 1
                    for (int d = 0; d < D; ++d)
                        if (*reinterpret_cast<volatile int*>(&nan_pos[d]) <= pos)
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(qs + panel_off(r, d >> 3, kRows) +
                                                                         (d & 7) * 2),
                                         "h"((uint16_t)0x7fff)
                                         : "memory");
                }
                __syncwarp();
                // (kept in shared memory meanwhile: a register spilled around the
                // loop above comes back from L2, which cost the prompts 5 %)
                const int64_t first_row = *reinterpret_cast<volatile int64_t*>(&first_rows[w]);
                const int c = lane % LPR;
#pragma unroll 4
                for (int i = 0; i < NA; ++i) {
                    const int rr = row0 + i * RPA + lane / LPR;
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(qs + panel_off(rr, c, kRows))
                                 : "memory");
                    if (rr < nrows)
                        st_v4(out + first_row + row_at(rr) + c * 8, v);
                }
                }
            }
        }
    } else if (warp < kConvWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        if ((warp == kMmaWarp || warp == kMmaWarp + 2) && lane == 0 &&
            (warp == kMmaWarp || ntok1 > 0)) {
            // ---------------- tensor-core issue for query tile w (one thread) ----------------
            // The two threads take turns by slot (a's P V of slot j, b's, a's of
            // slot j + 1, ...; each thread's S follows its P V), so that one
            // tile's softmax runs while the tensor core runs the other's products.
            const int w = warp == kMmaWarp ? 0 : 1;
            const int nkv = w ? nkv1 : nkv0;
            const uint32_t id_s = instr_desc<kF16>(kRows, kKeys, 0);
            const uint32_t id_o = instr_desc<kF16>(kRows, D, 1);
            // descriptor halves: every K step only adds (bytes >> 4) to a low half
            constexpr uint32_t hi1k = desc_hi(1024);
            const uint32_t q_lo = desc_lo(sb + L::q + w * L::QB, 16);
            const uint32_t k_lo = desc_lo(sb + L::slot, 16);
            const uint32_t v_lo = desc_lo(sb + L::slot + L::KVB, kKeys * 128);
            const uint32_t s_col = tmem + 128u * w;
            const uint32_t o_col = tmem + 256u + (uint32_t)D * w;
            bool alive = wait_one(s_addr(&bars.q_full[w]), 0, &abort_flag, p.dev_err);
            for (int j = 0; alive && j <= nk; ++j) {
                const uint32_t sl = (uint32_t)((j % ST) * L::SLOT >> 4);
                if (!wait_one(s_addr(&bars.full[j % ST]), (j / ST) & 1, &abort_flag, p.dev_err))
                    break;
                const bool pv = j > 0 && j <= nkv;
                // (the weights last: they are the ones that come late, and every
                // wait that has to be looked at costs a few hundred cycles)
                if (w == 1 ? !wait_one(s_addr(&bars.issued[0]), j & 1, &abort_flag, p.dev_err)
                           : (ntok1 > 0 && j > 0 &&
                              !wait_one(s_addr(&bars.issued[1]), (j - 1) & 1, &abort_flag, p.dev_err)))
                    break;
                if (pv && !wait_one(s_addr(&bars.p_most[w]), (j - 1) & 1, &abort_flag, p.dev_err))
                    break;
                bool used = false;
                if (pv) {
                    tc_fence_after();
                    const uint32_t acc0 = j > 1 ? 1u : 0u;
#pragma unroll
                    for (int ks = 0; ks < kKeys / 64 * 3; ++ks)
                        umma_ts_h(o_col, s_col + ks * 16, v_lo + sl + (uint32_t)(ks * 16 * 128 >> 4),
                                  hi1k, id_o, ks > 0 ? 1u : acc0);
                    if (!wait_one(s_addr(&bars.p_full[w]), (j - 1) & 1, &abort_flag, p.dev_err))
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = kKeys / 64 * 3; ks < kKeys / 16; ++ks)
                        umma_ts_h(o_col, s_col + ks * 16, v_lo + sl + (uint32_t)(ks * 16 * 128 >> 4),
                                  hi1k, id_o, 1u);
                    if (j == nkv)
                        umma_commit(s_addr(&bars.o_full[w]));
                    used = true;
                }
                // the other thread may queue its P V while this one queues S
                bar_arrive(s_addr(&bars.issued[w]));
                if (j < nkv) {
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (uint32_t)(((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4);
                        const uint32_t offk = (uint32_t)(((ks >> 2) * kKeys * 128 + (ks & 3) * 32) >> 4);
                        umma_h(s_col, q_lo + off, hi1k, k_lo + sl + offk, hi1k, id_s, ks > 0 ? 1u : 0u);
                    }
                    umma_commit(s_addr(&bars.s_full[w]));
                    used = true;
                }
                // this thread no longer reads slot j once its products are done
                if (used)
                    umma_commit(s_addr(&bars.empty[j % ST]));
                else
                    bar_arrive(s_addr(&bars.empty[j % ST]));
            }
            // every product (and every commit's arrival) done before teardown
            umma_commit(s_addr(&bars.drain[w]));
            bar_wait(s_addr(&bars.drain[w]), 0);
        }
    } else {
        // ---------------- load and convert (four warps) ----------------
        auto scales_of = [&](int phys) -> float2 {
            return block_ok(phys) ? __ldg(scales + (int64_t)phys * p.num_kv_heads + g) : make_float2(0.f, 0.f);
        };
        // (the references are powers of two: their inverses are exact)
        const float kinv = 1.f / reference_of(&ref_bits[0]), vinv = 1.f / reference_of(&ref_bits[1]);
        auto factor = [&](float sc, float inv) -> uint32_t {
            const float f = power_of(sc) * inv * kUnit;
            return pack_rn<kF16>(f, f);
        };
        // convert vectors i0 ..., with their blocks' factors, into their places of
        // an operand tile; a batch's reads, conversions and writes stand
        // together, since one warp per scheduler has nothing but its own
        // independent instructions to hide their latency
        const uint32_t place = panel_off(rsub, 2 * c4, kKeys);
        const uint32_t place1 = panel_off(rsub, 2 * c4 + 1, kKeys);
        auto store = [&](uint32_t dst, uint32_t f, int i0, const uint4(&x)[kBatch]) {
            uint4 lo[kBatch], hi[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; u += NP) {
                const uint32_t fi = __shfl_sync(0xffffffffu, f, ((i0 + u) / NP * 32 + rsub) / BS);
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    convert16(x[u + q], fi, lo[u + q], hi[u + q]);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t at = (i0 + u) / NP * 32 * 128 + (i0 + u) % NP * kKeys * 128;
                st_shared16(dst + place + at, lo[u]);
                st_shared16(dst + place1 + at, hi[u]);
            }
        };
        const bool uneven = *reinterpret_cast<volatile int*>(&any_rest) != 0;
        float2 sc0 = scales_of(id0), sc1 = scales_of(id1);
        uint32_t fv = 0u;                                          // V's factor of tile j - 1
        for (int j = 0; j <= nk; ++j) {
            const int st = j % ST;
            const int id3 = id_of(j + 3);
            const float2 sc2 = scales_of(id2);
            const uint32_t fk = factor(sc0.x, kinv);
            cp_async_wait<0>();
            if (!wait_warp(s_addr(&bars.empty[st]), ((j / ST) & 1) ^ 1, &abort_flag, p.dev_err))
                break;
            const uint32_t dst = sb + L::slot + st * L::SLOT;
            if (uneven && j < nk && cw == 0 && lane < NB) {
                rests[j & (NR - 1)][0][lane] = PREFIX && !block_ok(id0) ? 0.f : rest_of(sc0.x);
                rests[j & (NR - 1)][1][lane] = rest_of(sc0.y);
            }
            // each place is refilled for the next slot once its codes are used
            if (j < nk) {
#pragma unroll
                for (int i0 = 0; i0 < NV; i0 += kBatch) {
                    uint4 x[kBatch];
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        x[u] = lds16(raw_k + (i0 + u) * PITCH);
                    store(dst, fk, i0, x);
                    if (j + 1 < nk)
                        fetch(raw_k, kbase, id1, i0, (j + 1) * kKeys, kv_end);
                }
            }
#pragma unroll
            for (int i0 = 0; i0 < NV; i0 += kBatch) {
                if (j > 0) {
                    uint4 x[kBatch];
                    uint32_t bad = 0;
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        x[u] = lds16(raw_v + (i0 + u) * PITCH);
                        bad |= nan_codes(x[u].x) | nan_codes(x[u].y) | nan_codes(x[u].z) |
                               nan_codes(x[u].w);
                    }
                    if (bad != 0) {
                        // NaN codes: 0 in the tile, the position noted
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) {
                            const int row = (i0 + u) / NP * 32 + rsub;
                            int* col = nan_pos + (i0 + u) % NP * 64 + c4 * 16;
                            uint32_t w4[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                            for (int q4 = 0; q4 < 4; ++q4)
                                w4[q4] = note_nans(w4[q4], col + q4 * 4, &any_nan, (j - 1) * kKeys + row);
                            x[u] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                    }
                    __syncwarp();
                    store(dst + L::KVB, fv, i0, x);
                }
                if (j < nk)
                    fetch(raw_v, vbase, id0, i0, j * kKeys, kv_end);
            }
            cp_async_commit();
            async_proxy_fence();
            __syncwarp();
            if (lane == 0)
                bar_arrive(s_addr(&bars.full[st]));
            fv = factor(sc0.y, vinv);
            id0 = id1;
            id1 = id2;
            id2 = id3;
            sc0 = sc1;
            sc1 = sc2;
        }
        cp_async_wait<0>();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(L::cols));
    }
}

}  // namespace pfs
}  // namespace pkv
