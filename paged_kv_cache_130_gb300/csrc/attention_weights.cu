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
//     reads them, so that the passes fetch a tile in one copy.  Over an E4M3 cache
//     the products are fp16, in which every code is exact; bf16 rows become fp16
//     times a power of two, without loss down to 2^-28 of the row's largest.  The
//     sign of the scale goes into q, its size and the power into a factor per row.
//   * sums: S = Q K^T, a thread per row of q: running maximum and sum over the CTA's
//     keys, in fp32.
//   * totals: S^T = K Q^T, the operands swapped, a thread per key: the rows' maxima
//     and sums (merged over the CTAs of the first pass) make weights, which the
//     thread adds up in fp32 and adds to the key's total.  One thread has one key:
//     the same inputs give the same bits.
// A scale per block multiplies scores in fp32, wherever it is.
//
// One CTA = a run of 128-key tiles of one (sequence, KV head); two q tiles at a
// time stay in shared memory while the keys stream through a ring (more rows than
// 256: the keys stream again, from L2).  Warps 0-3 and 4-7: two groups of softmax
// threads; warp 8: one thread issues the products; warps 9-12 bring K.  Every wait
// is bounded.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "context_internal.h"
#include "pkv_common.cuh"
#include "tc_common.cuh"

namespace pkv {
namespace {

using namespace tc;

constexpr int kRows = 128;             // rows of an operand tile
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr int kLoadWarps = 4;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kScaleRing = 16;
constexpr float kRaise = 8.f;          // log2: how far a score may pass the running maximum

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

// One CTA = one tile of 128 rows; D / 8 lanes to a row.  QT: type of q, CT: of the
// operand.
template <int QT, int CT, int D>
__global__ void __launch_bounds__(256) weights_tiles_kernel(const WeightsParams p)
{
    constexpr int LPR = D / 8;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t idx = blockIdx.x;
    const int tile = (int)(idx % p.row_tiles);
    const int64_t item = idx / p.row_tiles;
    const int s = (int)(item / p.num_kv_heads);
    const int g = (int)(item - (int64_t)s * p.num_kv_heads);
    const Span sp = span_of(p, s, tile == 0 && g == 0 && threadIdx.x == 0);
    if (tile * kRows >= sp.rows)
        return;
    const float sign = p.qk_scale_log2 < 0.f ? -1.f : (p.qk_scale_log2 == 0.f ? 0.f : 1.f);
    char* dst = reinterpret_cast<char*>(p.q_tiles) + idx * (kRows * D * 2);
    const int c = threadIdx.x % LPR;
    for (int r = threadIdx.x / LPR; r < kRows; r += 256 / LPR) {
        const int rr = tile * kRows + r;
        const bool ok = rr < sp.rows;
        const int j = rr / p.group;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (ok)
            v = ld_ro(reinterpret_cast<const uint16_t*>(p.q) +
                      ((sp.first_row + j) * p.num_heads + g * p.group + (rr - j * p.group)) * D + c * 8);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float x[8];
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<QT>(w[e]);
            x[2 * e] = f.x, x[2 * e + 1] = f.y;
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        float up = 1.f;
        if constexpr (QT != CT) {
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // 2^13 / 2^floor(log2 mx), kept where it and its inverse are normal
            if (mx > 0.f && mx < __builtin_huge_valf())
                up = __uint_as_float(
                    (uint32_t)min(max(267 - (int)(__float_as_uint(mx) >> 23), 7), 247) << 23);
        }
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = pack_rn<CT>(x[2 * e] * (up * sign), x[2 * e + 1] * (up * sign));
        *reinterpret_cast<uint4*>(dst + panel_off(r, c, kRows)) = make_uint4(h[0], h[1], h[2], h[3]);
        if (c == 0)
            p.factors[idx * kRows + r] = fabsf(p.qk_scale_log2) * (1.f / up);
    }
}

// ------------------------------------------------------------------ the passes

template <int D, bool E8>
struct Layout {
    static constexpr int TB = D * kRows * 2;           // an operand tile
    static constexpr int ST = 4;                       // key tiles of the ring
    static constexpr int q = 0;                        // two q tiles
    static constexpr int ring = 2 * TB;
    static constexpr int bytes = ring + ST * TB;
    static constexpr int alloc = bytes + 1024;         // room to align the base
};

template <int ST>
struct Bars {
    uint64_t q_full;             // the copies of the q tiles
    uint64_t s_full[2][2];       // commit: scores of group w in buffer b
    uint64_t s_free[2][2];       // one arrival per warp of the group: they have been read
    uint64_t full[ST];           // one arrival per loading warp: key tile is stored
    uint64_t empty[ST];          // commit: no longer read
    uint64_t drain;              // commit: every product so far
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
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, int* flag, int32_t* dev_err)
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
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int* flag, int32_t* dev_err)
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

__device__ __forceinline__ void softmax_sync()
{
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ float2 fmul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
        " mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ void st_shared16(uint32_t a, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// CT: operand type; E8: the cache holds E4M3 codes; TOTALS: the second pass.
template <int CT, bool E8, int D, bool TOTALS>
__global__ void __launch_bounds__(kThreads, 1) weights_pass_kernel(const WeightsParams p)
{
    using L = Layout<D, E8>;
    constexpr int ST = L::ST;
    constexpr int NP = D / 64;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) Bars<ST> bars;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_flag;
    // K's scale of every 8 keys; softmax warps read a tile's up to ST + 3 tiles after
    // the loading warps have passed it
    __shared__ float ks_ring[kScaleRing][kRows / 8];
    static_assert(kScaleRing > ST + 4, "ring of the scales");
    // TOTALS: factor, -maximum and 1 / sum of the q tiles' rows, pairs of rows apart
    __shared__ __align__(16) float2 row_f[TOTALS ? kRows : 1], row_m[TOTALS ? kRows : 1],
        row_l[TOTALS ? kRows : 1];

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;

    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t idx = blockIdx.x;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    const int chunk = (int)(idx / items);
    const int64_t item = idx - (int64_t)chunk * items;
    const int s = (int)(item / p.num_kv_heads);
    const int g = (int)(item - (int64_t)s * p.num_kv_heads);
    const Span sp = span_of(p, s, false);
    const int tile0 = chunk * p.chunk_tiles;           // key tiles [tile0, tile0 + nk)
    const int nk = min((sp.ctx + kRows - 1) / kRows - tile0, p.chunk_tiles);
    if (sp.rows == 0 || nk <= 0)
        return;
    const int row_tiles = (sp.rows + kRows - 1) / kRows;
    const int pairs = (row_tiles + 1) / 2;

    const uint32_t sb = (s_addr(smem_raw) + 1023u) & ~1023u;
    if (tid == 0) {
        bar_init(s_addr(&bars.q_full), 1);
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                bar_init(s_addr(&bars.s_full[w][b]), 1);
                bar_init(s_addr(&bars.s_free[w][b]), 4);
            }
#pragma unroll
        for (int i = 0; i < ST; ++i) {
            bar_init(s_addr(&bars.full[i]), kLoadWarps);
            bar_init(s_addr(&bars.empty[i]), 1);
        }
        bar_init(s_addr(&bars.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_flag = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            s_addr(&tmem_holder)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;

    if (warp < 8) {
        // ---------------- softmax: group w ----------------
        const int w = warp >> 2;
        const int r = tid & (kRows - 1);               // tensor-memory lane
        const uint32_t t_s = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u * w;
        bool alive = true;
        int unit = 0;                                  // scores this group has seen
        auto next_scores = [&]() {
            alive = alive && wait_warp(s_addr(&bars.s_full[w][unit & 1]), (unit >> 1) & 1, &abort_flag,
                                       p.dev_err);
            tc_fence_after();
        };
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(s_addr(&bars.s_free[w][unit & 1]));
            ++unit;
        };
        for (int pr = 0; pr < pairs; ++pr) {
            const int nq = min(2, row_tiles - 2 * pr);
            const int row0 = pr * 2 * kRows;
            if constexpr (!TOTALS) {
                // one row a thread: of tile w over every key tile, or (one tile) over
                // the key tiles of the group's parity
                const int row = row0 + (nq == 2 ? w * kRows : 0) + r;
                const float f = row < sp.rows ? p.factors[(item * p.row_tiles * kRows) + row] : 0.f;
                const int pos = sp.first_pos + row / p.group;
                float m_run = kNegInf, l_run = 0.f;
                // tile by tile, 32 keys at a time
                for (int j = nq == 2 ? 0 : w; j < nk; j += nq == 2 ? 1 : 2) {
                    next_scores();
                    if (alive) {
                        const int key0 = (tile0 + j) * kRows;
                        // (uniform) some key passes some row's position
                        const bool edge = key0 + kRows - 1 > sp.first_pos + row0 / p.group;
                        const volatile float* ks = ks_ring[(pr * nk + j) % kScaleRing];
#pragma unroll 1
                        for (int c0 = 0; c0 < kRows; c0 += 32) {
                            float x[32];
                            tmem_ld16(t_s + 128u * (unit & 1) + c0, *reinterpret_cast<uint32_t(*)[16]>(x));
                            tmem_ld16(t_s + 128u * (unit & 1) + c0 + 16,
                                      *reinterpret_cast<uint32_t(*)[16]>(x + 16));
                            tmem_wait_ld();
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const float fb = E8 ? f * ks[c0 / 8 + b] : f;
#pragma unroll
                                for (int e = 0; e < 8; e += 2) {
                                    const float2 t = fmul2(make_float2(x[8 * b + e], x[8 * b + e + 1]),
                                                           make_float2(fb, fb));
                                    x[8 * b + e] = t.x, x[8 * b + e + 1] = t.y;
                                }
                            }
                            if (edge) {
                                const int lim = pos - key0 - c0;       // the last key the row sees
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    x[e] = e <= lim ? x[e] : kNegInf;
                            }
                            float mc[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mc[i] = fmaxf(x[2 * i], x[2 * i + 1]);
#pragma unroll
                            for (int e = 8; e < 32; e += 8)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mc[i] = fmax3(mc[i], x[e + 2 * i], x[e + 2 * i + 1]);
                            const float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
                            if (mx > m_run + kRaise || (mx > m_run && m_run == kNegInf)) {
                                l_run *= m_run == kNegInf ? 0.f : fast_exp2(m_run - mx);
                                m_run = mx;
                            }
                            const float nm = m_run == kNegInf ? 0.f : -m_run;
                            const float2 nm2 = make_float2(nm, nm);
                            float2 ls[2] = {};
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float2 t = fadd2(make_float2(x[e], x[e + 1]), nm2);
                                ls[(e >> 1) & 1] =
                                    fadd2(ls[(e >> 1) & 1], make_float2(fast_exp2(t.x), fast_exp2(t.y)));
                            }
                            l_run += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                        }
                    }
                    release();
                }
                if (row < sp.rows)
                    p.partials[((item * p.chunks + chunk) * 2 + (nq == 2 ? 0 : w)) * p.row_tiles * kRows + row] =
                        make_float2(m_run, l_run);
            } else {
                // the rows' maxima and sums: thread i has row i of the two tiles
                softmax_sync();                        // (the rows before have been used)
                {
                    const int row = row0 + tid;
                    float M = kNegInf, sum = 0.f, f = 0.f;
                    if (row < sp.rows) {
                        const int n = ((sp.ctx + kRows - 1) / kRows + p.chunk_tiles - 1) / p.chunk_tiles;
                        const float2* pt = p.partials + item * p.chunks * 2 * p.row_tiles * kRows + row;
                        const int64_t step = (int64_t)(nq == 2 ? 2 : 1) * p.row_tiles * kRows;
                        const int parts = nq == 2 ? n : 2 * n;
                        for (int i = 0; i < parts; ++i)
                            M = fmaxf(M, __ldcg(pt + i * step).x);
                        for (int i = 0; i < parts; ++i) {
                            const float2 v = __ldcg(pt + i * step);
                            sum += v.x == kNegInf ? 0.f : fast_exp2(v.x - M) * v.y;
                        }
                        f = p.factors[item * p.row_tiles * kRows + row];
                    }
                    const bool any = M != kNegInf;
                    reinterpret_cast<float*>(row_f)[tid] = f;
                    reinterpret_cast<float*>(row_m)[tid] = any ? -M : 0.f;
                    reinterpret_cast<float*>(row_l)[tid] = sum == 0.f ? 0.f : 1.f / sum;
                }
                softmax_sync();
                for (int j = w; j < nk; j += 2) {
                    const int key = (tile0 + j) * kRows + r;
                    // the first row that sees the key, and the end, of the pair's rows
                    const int lo = max(0, (key - sp.first_pos) * p.group - row0);
                    const int hi = sp.rows - row0;
                    float2 acc[2] = {};
                    float k_scale = 1.f;
                    for (int qt = 0; qt < nq; ++qt) {
                        next_scores();
                        if (alive) {
                            if (E8 && qt == 0)
                                k_scale = *const_cast<const volatile float*>(
                                    &ks_ring[(pr * nk + j) % kScaleRing][r / 8]);
                            const float2 ks2 = make_float2(k_scale, k_scale);
                            const int end = min(kRows, hi - qt * kRows);
                            // (uniform) some row does not see some key of the tile
                            const bool edge = (tile0 + j) * kRows + kRows - 1 > sp.first_pos;
#pragma unroll 1
                            for (int c0 = 0; c0 < end; c0 += 32) {
                                float x[32];
                                tmem_ld16(t_s + 128u * (unit & 1) + c0,
                                          *reinterpret_cast<uint32_t(*)[16]>(x));
                                tmem_ld16(t_s + 128u * (unit & 1) + c0 + 16,
                                          *reinterpret_cast<uint32_t(*)[16]>(x + 16));
                                tmem_wait_ld();
                                const int at = (qt * kRows + c0) / 2;
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    float2 t = make_float2(x[e], x[e + 1]);
                                    if constexpr (E8)
                                        t = fmul2(t, ks2);
                                    t = ffma2(t, row_f[at + e / 2], row_m[at + e / 2]);
                                    x[e] = fast_exp2(t.x), x[e + 1] = fast_exp2(t.y);
                                }
                                if (edge || c0 + 32 > end) {
                                    const int a = lo - qt * kRows - c0, b = end - c0;
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        x[e] = e >= a && e < b ? x[e] : 0.f;
                                    // (a row's 1 / sum may be NaN, and is not for keys it does not see)
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (e >= a && e < b)
                                            acc[0].x = fmaf(x[e], reinterpret_cast<const float*>(row_l)[2 * at + e],
                                                            acc[0].x);
                                } else {
#pragma unroll
                                    for (int e = 0; e < 32; e += 2)
                                        acc[(e >> 1) & 1] = ffma2(make_float2(x[e], x[e + 1]), row_l[at + e / 2],
                                                                  acc[(e >> 1) & 1]);
                                }
                            }
                        }
                        release();
                    }
                    if (alive && key < sp.ctx) {
                        float* at = p.weights + s * p.weights_seq + g * p.weights_head + key;
                        *at += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    }
                }
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // ---------------- copies of q, products (one thread) ----------------
            const uint32_t id = instr_desc<CT>(kRows, kRows, 0);
            constexpr uint32_t hi1k = desc_hi(1024);
            const uint32_t q_lo = desc_lo(sb + L::q, 16);
            const uint32_t k_lo = desc_lo(sb + L::ring, 16);
            const char* q_src = reinterpret_cast<const char*>(p.q_tiles) + item * p.row_tiles * (int64_t)L::TB;
            int units[2] = {0, 0};
            int jj = 0;                                // key tiles so far, all pairs
            bool alive = true;
            int drains = 0;
            // (the tiles were written by the kernel before, these copies are another proxy's)
            asm volatile("fence.proxy.async.global;" ::: "memory");
            auto product = [&](int w, uint32_t q_off, uint32_t k_off) {
                const int u = units[w]++;
                if (u >= 2 && !wait_one(s_addr(&bars.s_free[w][u & 1]), ((u >> 1) & 1) ^ 1, &abort_flag,
                                        p.dev_err))
                    return false;
                tc_fence_after();
                const uint32_t d = tmem + 256u * w + 128u * (u & 1);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (uint32_t)(((k >> 2) * kRows * 128 + (k & 3) * 32) >> 4);
                    const uint32_t a = (TOTALS ? k_lo + k_off : q_lo + q_off) + off;
                    const uint32_t b = (TOTALS ? q_lo + q_off : k_lo + k_off) + off;
                    umma_h(d, a, hi1k, b, hi1k, id, k > 0 ? 1u : 0u);
                }
                umma_commit(s_addr(&bars.s_full[w][u & 1]));
                return true;
            };
            for (int pr = 0; alive && pr < pairs; ++pr) {
                const int nq = min(2, row_tiles - 2 * pr);
                if (pr > 0) {
                    // the products that read the tiles before
                    umma_commit(s_addr(&bars.drain));
                    alive = wait_one(s_addr(&bars.drain), drains & 1, &abort_flag, p.dev_err);
                    ++drains;
                    if (!alive)
                        break;
                }
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s_addr(&bars.q_full)),
                             "r"(nq * L::TB)
                             : "memory");
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                        sb + L::q),
                    "l"(q_src + (int64_t)pr * 2 * L::TB), "r"(nq * L::TB), "r"(s_addr(&bars.q_full))
                    : "memory");
                alive = wait_one(s_addr(&bars.q_full), pr & 1, &abort_flag, p.dev_err);
                for (int j = 0; alive && j < nk; ++j, ++jj) {
                    const int st = jj % ST;
                    if (!wait_one(s_addr(&bars.full[st]), (jj / ST) & 1, &abort_flag, p.dev_err)) {
                        alive = false;
                        break;
                    }
                    const uint32_t k_off = (uint32_t)(st * L::TB >> 4);
                    if constexpr (TOTALS) {
                        for (int qt = 0; alive && qt < nq; ++qt)
                            alive = product(j & 1, (uint32_t)(qt * L::TB >> 4), k_off);
                    } else if (nq == 2) {
                        alive = product(0, 0u, k_off) && product(1, (uint32_t)(L::TB >> 4), k_off);
                    } else {
                        alive = product(j & 1, 0u, k_off);
                    }
                    umma_commit(s_addr(&bars.empty[st]));
                }
            }
            // every product (and every commit's arrival) done before teardown
            umma_commit(s_addr(&bars.drain));
            bar_wait(s_addr(&bars.drain), drains & 1);
        }
    } else {
        // ---------------- keys into the ring (four warps) ----------------
        const int cw = warp - kLoadWarp;
        const int lt = tid - kLoadWarp * 32;
        const int sh = 31 - __clz(p.block_size);       // (a power of two)
        const int bs = 1 << sh;
        const int per_tile = kRows >> sh;              // blocks of a tile, 4..16
        const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
        const int64_t tile_bytes = (int64_t)bs * D * (E8 ? 1 : 2);
        const char* base = reinterpret_cast<const char*>(p.k_cache) + g * tile_bytes;
        const int64_t stride = p.num_kv_heads * tile_bytes;
        const int total = pairs * nk;
        // lane i: block i of key tile jj (counted over the pairs); -1: none
        auto id_of = [&](int jj) -> int {
            const int tok = (tile0 + jj % nk) * kRows + lane * bs;
            if (jj >= total || lane >= per_tile || tok >= sp.ctx)
                return -1;
            const int id = __ldg(table + (tok >> sh));
            if (id >= 0 && (int64_t)id < p.num_blocks)
                return id;
            flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);
            return -1;
        };
        if constexpr (E8) {
            const int c4 = lane & 3;
            const int rsub = cw * 8 + (lane >> 2);
            constexpr int NV = NP * 4;                 // vectors of a lane: see below
            const float2* scales = reinterpret_cast<const float2*>(p.scales);
            auto scale_of = [&](int id) -> float {
                return scales == nullptr ? 1.f
                                         : (id >= 0 ? __ldg(scales + (int64_t)id * p.num_kv_heads + g).x : 0.f);
            };
            // vector i: row 32 (i / NP) + rsub, panel i % NP, 16 codes c4 of its 64
            auto fetch = [&](int jj, int id, uint4(&x)[NV]) {
                const int key0 = (tile0 + jj % nk) * kRows;
#pragma unroll
                for (int i = 0; i < NV; i += NP) {
                    const int row = i / NP * 32 + rsub;
                    const int phys = __shfl_sync(0xffffffffu, id, row >> sh);
                    const bool ok = phys >= 0 && key0 + row < sp.ctx;
                    const char* src = base + (ok ? phys * stride + (row & (bs - 1)) * D + c4 * 16 : 0);
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        x[i + q] = ok ? ld_stream(src + q * 64) : make_uint4(0, 0, 0, 0);
                }
            };
            const uint32_t place = panel_off(rsub, 2 * c4, kRows);
            const uint32_t place1 = panel_off(rsub, 2 * c4 + 1, kRows);
            auto store = [&](int jj, float sc, const uint4(&x)[NV]) -> bool {
                const int st = jj % ST;
                if (!wait_warp(s_addr(&bars.empty[st]), ((jj / ST) & 1) ^ 1, &abort_flag, p.dev_err))
                    return false;
                const uint32_t dst = sb + L::ring + st * L::TB;
                if (cw == 0) {
                    // (a block's scale, for every 8 of its keys)
                    const float v = __shfl_sync(0xffffffffu, sc, min(31, (lane * 8) >> sh));
                    if (lane < kRows / 8)
                        *const_cast<volatile float*>(&ks_ring[jj % kScaleRing][lane]) = v;
                }
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    uint4 lo, hi;
                    e4m3x4_to_f16x2(x[i].x, lo.x, lo.y);
                    e4m3x4_to_f16x2(x[i].y, lo.z, lo.w);
                    e4m3x4_to_f16x2(x[i].z, hi.x, hi.y);
                    e4m3x4_to_f16x2(x[i].w, hi.z, hi.w);
                    const uint32_t at = i / NP * 32 * 128 + i % NP * kRows * 128;
                    st_shared16(dst + place + at, lo);
                    st_shared16(dst + place1 + at, hi);
                }
                async_proxy_fence();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(s_addr(&bars.full[st]));
                return true;
            };
            // ids three tiles ahead, codes and scales two
            uint4 xa[NV], xb[NV];
            int id0 = id_of(0), id1 = id_of(1), id2 = id_of(2);
            float sa = scale_of(id0), sc1 = scale_of(id1);
            fetch(0, id0, xa);
            fetch(1, id1, xb);
            for (int jj = 0; jj < total; jj += 2) {
                int id3 = id_of(jj + 3);
                if (!store(jj, sa, xa))
                    break;
                fetch(jj + 2, id2, xa);
                sa = scale_of(id2);
                id2 = id_of(jj + 4);
                if (jj + 1 < total && !store(jj + 1, sc1, xb))
                    break;
                fetch(jj + 3, id3, xb);
                sc1 = scale_of(id3);
            }
        } else {
            constexpr int LPR = D / 8;                 // lanes to a row
            constexpr int RPA = 32 / LPR;              // rows to a warp's access
            constexpr int NA = kRows / (RPA * kLoadWarps);
            constexpr int kAhead = ST - 2;             // tiles on their way
            const int c = lt % LPR;
            int id0 = id_of(0), id1 = id_of(1);
            auto landed = [&](int jj) {
                async_proxy_fence();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(s_addr(&bars.full[jj % ST]));
            };
            int jj = 0;
            for (; jj < total; ++jj) {
                const int st = jj % ST;
                const int id2 = id_of(jj + 2);
                if (!wait_warp(s_addr(&bars.empty[st]), ((jj / ST) & 1) ^ 1, &abort_flag, p.dev_err))
                    break;
                const int key0 = (tile0 + jj % nk) * kRows;
                const uint32_t dst = sb + L::ring + st * L::TB;
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    const int row = (i * kLoadWarps + cw) * RPA + lane / LPR;
                    const int phys = __shfl_sync(0xffffffffu, id0, row >> sh);
                    const bool ok = phys >= 0 && key0 + row < sp.ctx;
                    cp16z(dst + panel_off(row, c, kRows),
                          base + (ok ? phys * stride + (row & (bs - 1)) * (D * 2) + c * 16 : 0), ok);
                }
                cp_async_commit();
                if (jj >= kAhead) {
                    cp_async_wait<kAhead>();
                    landed(jj - kAhead);
                }
                id0 = id1;
                id1 = id2;
            }
            cp_async_wait<0>();
            if (jj == total)
                for (int k = max(0, total - kAhead); k < total; ++k)
                    landed(k);
        }
    }

    tc_fence_before();
    __syncthreads();
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
    static bool configured[64] = {};
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
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    e = launch_early(weights_tiles_kernel<QT, CT, D>, items * p.row_tiles, 256, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    e = launch_early(weights_pass_kernel<CT, E8, D, false>, items * p.chunks, kThreads, L::alloc, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_early(weights_pass_kernel<CT, E8, D, true>, items * p.chunks, kThreads, L::alloc, stream, p);
}

template <int QT, int CT, bool E8>
cudaError_t by_dim(const WeightsParams& p, cudaStream_t stream)
{
    return p.head_dim == 128 ? run<QT, CT, E8, 128>(p, stream) : run<QT, CT, E8, 64>(p, stream);
}

}  // namespace

// Runs of key tiles: about four CTAs an SM, at least four tiles each.
WeightsPlan plan_weights(int32_t num_seqs, int32_t num_kv_heads, int32_t group, int32_t window,
                         int32_t max_context_len, int sms)
{
    WeightsPlan pl{};
    const int64_t tiles = ((int64_t)max_context_len + kRows - 1) / kRows;
    const int64_t items = (int64_t)num_seqs * num_kv_heads;
    const int64_t want = (items * tiles + 4 * sms - 1) / (4 * sms);
    pl.chunk_tiles = (int32_t)(want < 4 ? 4 : want);
    pl.chunks = (int32_t)((tiles + pl.chunk_tiles - 1) / pl.chunk_tiles);
    pl.row_tiles = (int32_t)(((int64_t)window * group + kRows - 1) / kRows);
    return pl;
}

cudaError_t launch_attention_weights(const WeightsParams& p, cudaStream_t stream)
{
    if (p.cache_dtype == kE4M3)
        return p.q_dtype == kF16 ? by_dim<kF16, kF16, true>(p, stream)
                                 : by_dim<kBF16, kF16, true>(p, stream);
    return p.q_dtype == kF16 ? by_dim<kF16, kF16, false>(p, stream)
                             : by_dim<kBF16, kBF16, false>(p, stream);
}

}  // namespace pkv
