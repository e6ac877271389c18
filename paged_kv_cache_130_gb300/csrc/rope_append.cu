// rope_append.cu -- rotary positions on the new tokens' q and K, and the write
// of K and V into the paged cache, in one pass.
//
// A token at position p turns pair i of each head by p * inv_freq[i]:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin).
// Angles: inv_freq / 2 pi becomes a 64-bit binary fraction of a turn, so that
// p * that fraction, taken modulo 2^64 by integer wrap-around, is the turn's
// fraction to 2^-53 p whatever the position; an fp32 product would be off by
// 2^-24 p radians.  sincospif sees the fraction rounded to 24 bits.
//
// One CTA holds one block of one sequence (the at most block_size new tokens
// that fall into it): it computes the cosines and sines of its tokens once
// into shared memory, and its warps share out the rows.
//   * K and V: one warp per (KV head, K or V) holds all the block's new rows of
//     that head in registers.  For a cache with a scale per block and head it
//     first takes the largest magnitude of the rows as they came in (times a
//     bound on what the rotation can add: it keeps a^2 + b^2, so sqrt(2) m),
//     which fixes the scale before anything is rotated, then rotates and
//     rounds once, from fp32, to E4M3.  The scale is a power of two: E4M3 is a
//     floating format, so a power of two costs no precision, and when a later
//     token raises the scale of a part-filled block, shifting the older codes
//     is exact but for the subnormal ones.
//   * q: one warp per (token, 16 heads), its cosines and sines in registers.
// The warp that owns (block, head, K or V) is the only reader and writer of
// that scale and of those codes.
// Bound by the bytes moved on prompts: Llama-2-7B shape, 9,329 tokens, 382 MB in
// 69 us (5.5 TB/s); a 16-bit chunk of 2,048 tokens x (64 + 8 + 8) heads, 84 MB
// in 12.3 us (6.8 TB/s).  Measured beside it: 8 heads a task 75 us, 256 threads
// 71-75, three and four of those resident 73-79, codes from cosines read with
// bank conflicts and one rounding per value 101.
#include <cuda_runtime.h>

#include <type_traits>

#include "pkv_common.cuh"
#include "scaled_internal.h"
#include "tc_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kSame = 0;               // cache of the input type
constexpr int kTensor = 1;             // E4M3, one scale per cache
constexpr int kScaled = 2;             // E4M3, a scale per block and head
constexpr int kHeadsPerTask = 16;

// The smallest power of two s >= 2^-126 with bound <= 448 s; 448 = 1.75 x 2^8.
__device__ __forceinline__ float power_of_two(float bound)
{
    const uint32_t u = __float_as_uint(fminf(bound, 3.4028235e38f));
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // biased
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// inv_freq (radians) as a 64-bit binary fraction of a turn: the 53-bit
// significand times 2^65 / pi = 2^66 / (2 pi) (`per_radian`), shifted into place.
// All in integers: this GPU's fp64 units would take longer over a block's angles
// than its rows.
__device__ __forceinline__ uint64_t turns_of(double inv_freq, uint64_t per_radian)
{
    const uint64_t b = (uint64_t)__double_as_longlong(inv_freq);
    const int e = (int)(b >> 52) & 0x7ff;
    if (e == 0 || e > 1023 + 52)                       // zero and what is no frequency
        return 0;
    const uint64_t m = (b & 0xfffffffffffffull) | (1ull << 52);
    const uint64_t lo = m * per_radian;
    const uint64_t hi = __umul64hi(m, per_radian);
    const int sh = 1077 - e;                           // >= 2
    const uint64_t t = sh >= 128 ? 0ull
                                 : (sh >= 64 ? hi >> (sh - 64) : (hi << (64 - sh)) | (lo >> sh));
    return (b >> 63) ? 0ull - t : t;
}

// fp32 fraction of a half turn in [-1, 1) of position pos: turns = the turn
// per position as a 64-bit binary fraction.
__device__ __forceinline__ float half_turns(uint64_t turns, int pos)
{
    const uint64_t t = turns * (uint64_t)(int64_t)pos;
    return (float)(int32_t)(t >> 32) * 4.656612873077393e-10f;    // 2^-31
}

// a b in two fp32 lanes per instruction.
__device__ __forceinline__ float2 fmul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
        " mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// Two 16-bit values (of one word) as an fp32 pair, and back, to nearest even.
template <int IT>
__device__ __forceinline__ uint32_t pack_pair(float2 x)
{
    uint32_t r;
    if constexpr (IT == kBF16)
        asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(x.x), "f"(x.y));
    else
        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(x.x), "f"(x.y));
    return r;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i)
{
    return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Eight values -> eight E4M3 codes of value * inv, saturating.
__device__ __forceinline__ uint2 codes8(const float2 (&x)[4], float inv)
{
    const float2 f = make_float2(inv, inv);
    uint16_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = fmul2(x[i], f);
        c[i] = e4m3x2_satfinite(y.x, y.y);
    }
    return make_uint2(pack2(c[0], c[1]), pack2(c[2], c[3]));
}

// Larger magnitudes of two words of 16-bit values (NaN gives way to a number).
template <int IT>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (IT == kBF16)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
    else
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b & 0x7fff7fffu));
    return r;
}

// A lane's 8-element vector `c` of a row, and how the rotation reaches it.
struct Place {
    bool rotated;
    bool inter;        // pairs inside the vector
    int partner;       // lane that holds the other halves of this lane's pairs
    uint32_t flip;     // sign bits that the other halves take (first halves: -)
    int set;           // which set of frequencies: 8 (4 if inter) a set
};

__device__ __forceinline__ Place place_of(int c, int lane, int rot, bool interleaved)
{
    Place pl;
    const int h = rot / 16;                      // vectors in half of the rotated part
    pl.rotated = c < 2 * h;
    pl.inter = interleaved;
    const bool first = c < h;
    pl.partner = (pl.rotated && !interleaved) ? (first ? lane + h : lane - h) : lane;
    pl.flip = first ? 0x80008000u : 0u;
    pl.set = !pl.rotated ? 0 : (interleaved || first ? c : c - h);
    return pl;
}

// Cosines and sines (times m) of a vector's frequencies: in shared memory, per
// token, rh cosines then rh sines; four frequencies of a set are 16 bytes, and
// the sets' first (and second) fours lie side by side, so that a row's lanes
// read without conflicts.
struct Turn {
    float4 c[2], s[2];
};

__device__ __forceinline__ float4 lds4(uint32_t a)
{
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "r"(a));
    return r;
}

__device__ __forceinline__ Turn turn_of(uint32_t table, int t, int rh, const Place& pl)
{
    Turn z;
    const uint32_t a = table + (uint32_t)(t * 2 * rh + pl.set * 4) * 4u;
    z.c[0] = lds4(a);
    z.s[0] = lds4(a + rh * 4);
    z.c[1] = z.c[0];
    z.s[1] = z.s[0];
    if (!pl.inter) {
        z.c[1] = lds4(a + rh * 2);
        z.s[1] = lds4(a + rh * 6);
    }
    return z;
}

// Rotate a lane's vector: y = x c + (other half) s, pair by pair.  Called by
// whole warps (the other halves come by shuffle).  What is not rotated has to be
// taken from w itself.
template <int IT>
__device__ __forceinline__ void rotate8(const uint4& w, const Place& pl, const Turn& z,
                                        float2 (&y)[4])
{
    if (pl.inter) {
        const float c[4] = {z.c[0].x, z.c[0].y, z.c[0].z, z.c[0].w};
        const float s[4] = {z.s[0].x, z.s[0].y, z.s[0].z, z.s[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<IT>(word(w, i));
            y[i] = make_float2(x.x * c[i] - x.y * s[i], x.y * c[i] + x.x * s[i]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t o = __shfl_sync(0xffffffffu, word(w, i), pl.partner) ^ pl.flip;
        const float4 c4 = z.c[i >> 1], s4 = z.s[i >> 1];
        const float2 c = i & 1 ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
        const float2 s = i & 1 ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
        y[i] = tc::ffma2(unpack2<IT>(o), s, fmul2(unpack2<IT>(word(w, i)), c));
    }
}

template <int MODE, int IT, int D, int BS>
__global__ void __launch_bounds__(kThreads, 4)
    rope_append_kernel(const RopeParams p)
{
    constexpr int VPR = D / 8;                    // vectors per row
    constexpr int RPI = 32 / VPR;                 // rows per warp access
    constexpr int NV = BS / RPI;                  // vectors a lane holds of a block
    constexpr int C = MODE == kSame ? 2 : 1;      // cache bytes per element
    __shared__ __align__(16) float sh_cs[BS * D];

    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int s = blockIdx.z * 65535 + blockIdx.y;
    if (s >= p.num_seqs)
        return;
    pdl_launch_dependents();
    const int cu0 = __ldg(p.cu_seqlens_q + s);
    const int cu1 = __ldg(p.cu_seqlens_q + s + 1);
    const int ctx = __ldg(p.context_lens + s);
    const int n = cu1 - cu0;
    const int ntouch = (p.max_q_len + BS - 2) / BS + 1;
    const int split = gridDim.x / ntouch;         // CTAs that share a block's rows
    const int bi = blockIdx.x / split;
    const int part = blockIdx.x % split;
    if (cu0 < 0 || cu1 < cu0 || cu1 > p.total_q || n > p.max_q_len || ctx < n ||
        ctx > p.max_context_len || (ctx + BS - 1) / BS > p.max_blocks_per_seq) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            flag_error(p.dev_err, PKV_DEVERR_CONTEXT);
        return;
    }
    const int first = ctx - n;                    // position of the first new token
    const int blk = first / BS + bi;              // the block, in logical order
    const int lo = max(first, blk * BS);
    const int hi = min(ctx, blk * BS + BS);
    if (lo >= hi)
        return;
    const int T = hi - lo;                        // new tokens in the block
    const int off = lo - blk * BS;                // offset of the first of them
    const int64_t row0 = (int64_t)cu0 + (lo - first);

    const int rh = p.rot_dim / 2;
    const bool inter = p.interleaved != 0;
    const uint32_t table = static_cast<uint32_t>(__cvta_generic_to_shared(sh_cs));
    const int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + blk);
    const bool good = phys >= 0 && (int64_t)phys < p.num_blocks;
    if (!good && threadIdx.x == 0 && part == 0)
        flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);

    const int c = lane % VPR;
    const int rsub = lane / VPR;
    const Place pl = place_of(c, lane, p.rot_dim, inter);
    const int kv_tasks = 2 * p.num_kv_heads;
    const int hchunks = p.q != nullptr ? (p.num_heads + kHeadsPerTask - 1) / kHeadsPerTask : 0;
    const int tasks = kv_tasks + T * hchunks;

    const int shift = p.position_offsets != nullptr ? __ldg(p.position_offsets + s) : 0;
    // cosines and sines of the block's tokens
    for (int f = lane; f < rh; f += 32) {
        const uint64_t turns = turns_of(__ldg(p.inv_freq + f), p.per_radian);
        // (set, frequency) = (f / 4, f % 4), or (f / 8, f % 8) in two fours
        float* at = sh_cs + (inter ? f : ((f >> 2) & 1) * (rh >> 1) + (f >> 3) * 4 + (f & 3));
        for (int t = warp; t < T; t += kWarps) {
            float sn, cn;
            sincospif(half_turns(turns, lo + t + shift), &sn, &cn);
            at[t * 2 * rh] = cn * p.mscale;
            at[t * 2 * rh + rh] = sn * p.mscale;
        }
    }
    __syncthreads();

    // K or V of one head.  FULL: the call writes the whole block, the usual case
    // of a prompt, without a test per row.
    auto kv_task = [&](auto full, int task) {
        constexpr bool FULL = decltype(full)::value;
        const int g = task >> 1;
        const bool is_v = task & 1;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(is_v ? p.v : p.k) +
                              (row0 + rsub) * stride + (int64_t)g * D + c * 8;
        char* tile = reinterpret_cast<char*>(is_v ? p.v_cache : p.k_cache) +
                     ((int64_t)phys * p.num_kv_heads + g) * (BS * D) * C;
        uint4 w[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (FULL || i * RPI + rsub < T)
                w[i] = ld_ro(src + i * RPI * stride);
        }
        [[maybe_unused]] float inv = is_v ? p.v_inv_scale : p.k_inv_scale;
        if constexpr (MODE == kScaled) {
            float* sp = p.scales + ((int64_t)phys * p.num_kv_heads + g) * 2 + (is_v ? 1 : 0);
            const float old = off > 0 ? *sp : 0.f;
            uint32_t m2 = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    m2 = max_abs2<IT>(m2, word(w[i], j));
            float2 mm = unpack2<IT>(m2);
            float mx = fmaxf(mm.x, mm.y);
            if (!(mx < __int_as_float(0x7f800000))) {
                // an infinity among them: the largest finite one
                mx = 0.f;
#pragma unroll 1
                for (int t = rsub; t < T; t += RPI) {
                    const uint4 u = ld_ro(src + (t - rsub) * stride);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mm = unpack2<IT>(word(u, j) & 0x7fff7fffu);
                        mx = mm.x < __int_as_float(0x7f800000) ? fmaxf(mx, mm.x) : mx;
                        mx = mm.y < __int_as_float(0x7f800000) ? fmaxf(mx, mm.y) : mx;
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float need = power_of_two(is_v ? mx : mx * p.k_bound);
            const float sc = off > 0 ? fmaxf(old, need) : need;
            inv = 1.f / sc;
            if (off > 0 && sc != old) {
                // the codes of the block's other slots follow the scale
                const float f = old / sc;
                for (int i = lane; i < (BS - T) * (D / 8); i += 32) {
                    const int j = i < off * (D / 8) ? i : i + T * (D / 8);
                    uint2* cp = reinterpret_cast<uint2*>(tile) + j;
                    const uint2 u = *cp;
                    float2 x[4];
                    const uint32_t ww[2] = {u.x, u.y};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t h0, h1;
                        e4m3x4_to_f16x2(ww[j], h0, h1);
                        x[2 * j] = f16x2_to_float2(h0);
                        x[2 * j + 1] = f16x2_to_float2(h1);
                    }
                    *cp = codes8(x, f);
                }
            }
            if (lane == 0)
                *sp = sc;
        }
        char* dst = tile + ((off + rsub) * D + c * 8) * C;
        const bool turn = !is_v && p.rot_dim > 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int t = i * RPI + rsub;
            if (!FULL && i * RPI >= T)                // warp-uniform
                break;
            float2 y[4];
            if (turn)
                rotate8<IT>(w[i], pl, turn_of(table, FULL ? t : min(t, T - 1), rh, pl), y);
            const bool plain = !turn || !pl.rotated;
            if constexpr (MODE == kSame) {
                if (FULL || t < T)
                    st_v4(dst + i * RPI * D * C,
                          plain ? w[i]
                                : make_uint4(pack_pair<IT>(y[0]), pack_pair<IT>(y[1]),
                                             pack_pair<IT>(y[2]), pack_pair<IT>(y[3])));
            } else {
                if (plain) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[j] = unpack2<IT>(word(w[i], j));
                }
                const uint2 codes = codes8(y, inv);
                if (FULL || t < T)
                    *reinterpret_cast<uint2*>(dst + i * RPI * D * C) = codes;
            }
        }
    };
    // kHeadsPerTask heads (FULL), or the last few, of one token's q
    auto q_task = [&](auto full, int t, int h0) {
        constexpr bool FULL = decltype(full)::value;
        constexpr int NQ = kHeadsPerTask / RPI;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + (row0 + t) * p.q_stride +
                              (h0 + rsub) * D + c * 8;
        uint16_t* dst = reinterpret_cast<uint16_t*>(p.q_out) +
                        ((row0 + t) * p.num_heads + h0 + rsub) * D + c * 8;
        const int left = p.num_heads - h0 - rsub;
        uint4 w[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {        // (plain loads: q_out may be q)
            w[i] = make_uint4(0, 0, 0, 0);
            if (FULL || i * RPI < left)
                w[i] = *reinterpret_cast<const uint4*>(src + i * RPI * D);
        }
        Turn z{};
        if (p.rot_dim > 0)
            z = turn_of(table, t, rh, pl);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            float2 y[4];
            rotate8<IT>(w[i], pl, z, y);
            if (pl.rotated)
                w[i] = make_uint4(pack_pair<IT>(y[0]), pack_pair<IT>(y[1]), pack_pair<IT>(y[2]),
                                  pack_pair<IT>(y[3]));
            if (FULL || i * RPI < left)
                st_v4(dst + i * RPI * D, w[i]);
        }
    };
    for (int task = part * kWarps + warp; task < tasks; task += split * kWarps) {
        if (task < kv_tasks) {
            if (!good)
                continue;
            if (T == BS)
                kv_task(std::true_type{}, task);
            else
                kv_task(std::false_type{}, task);
        } else {
            const int t = (task - kv_tasks) / hchunks;
            const int h0 = (task - kv_tasks - t * hchunks) * kHeadsPerTask;
            if (h0 + kHeadsPerTask <= p.num_heads)
                q_task(std::true_type{}, t, h0);
            else
                q_task(std::false_type{}, t, h0);
        }
    }
}

template <int MODE, int IT, int D, int BS>
cudaError_t run(const RopeParams& p, int sms, cudaStream_t stream)
{
    const int64_t ntouch = (p.max_q_len + BS - 2) / BS + 1;
    // few blocks (a decode step): several CTAs share the rows of each block,
    // down to one warp task each, up to twice the CTAs that fit at once (four
    // times as many cost the 2,048-token chunk 14.6 us instead of 12.3: each
    // starts with the latency of its lengths, frequencies and sines)
    const int T = p.max_q_len < BS ? p.max_q_len : BS;
    const int64_t hchunks = p.q ? (p.num_heads + kHeadsPerTask - 1) / kHeadsPerTask : 0;
    const int64_t tasks = 2 * p.num_kv_heads + T * hchunks;
    int64_t split = (8 * (int64_t)sms) / (ntouch * p.num_seqs);
    const int64_t most = (tasks + kWarps - 1) / kWarps;
    split = split < 1 ? 1 : (split > most ? most : split);
    if (ntouch * split > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    const unsigned gy = p.num_seqs < 65535 ? (unsigned)p.num_seqs : 65535u;
    const unsigned gz = (unsigned)((p.num_seqs + 65534) / 65535);
    rope_append_kernel<MODE, IT, D, BS>
        <<<dim3((unsigned)(ntouch * split), gy, gz), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int MODE, int IT, int D>
cudaError_t by_block(const RopeParams& p, int sms, cudaStream_t st)
{
    switch (p.block_size) {
    case 8: return run<MODE, IT, D, 8>(p, sms, st);
    case 16: return run<MODE, IT, D, 16>(p, sms, st);
    case 32: return run<MODE, IT, D, 32>(p, sms, st);
    default: return cudaErrorNotSupported;
    }
}

template <int MODE, int IT>
cudaError_t by_dim(const RopeParams& p, int sms, cudaStream_t st)
{
    return p.head_dim == 128 ? by_block<MODE, IT, 128>(p, sms, st)
                             : by_block<MODE, IT, 64>(p, sms, st);
}

template <int MODE>
cudaError_t by_type(const RopeParams& p, int sms, cudaStream_t st)
{
    return p.in_dtype == kF16 ? by_dim<MODE, kF16>(p, sms, st) : by_dim<MODE, kBF16>(p, sms, st);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t stream)
{
    if (p.num_seqs <= 0 || p.max_q_len <= 0 || p.total_q <= 0)
        return cudaSuccess;
    if (p.scales != nullptr)
        return by_type<kScaled>(p, sms, stream);
    return p.cache_dtype == kE4M3 ? by_type<kTensor>(p, sms, stream)
                                  : by_type<kSame>(p, sms, stream);
}

}  // namespace pkv
