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
//   * q: one warp per (token, 8 heads), its cosines and sines in registers.
// The warp that owns (block, head, K or V) is the only reader and writer of
// that scale and of those codes.
#include <cuda_runtime.h>

#include "pkv_common.cuh"
#include "scaled_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSame = 0;               // cache of the input type
constexpr int kTensor = 1;             // E4M3, one scale per cache
constexpr int kScaled = 2;             // E4M3, a scale per block and head
constexpr int kHeadsPerTask = 8;

// The smallest power of two s >= 2^-126 with bound <= 448 s; 448 = 1.75 x 2^8.
__device__ __forceinline__ float power_of_two(float bound)
{
    const uint32_t u = __float_as_uint(fminf(bound, 3.4028235e38f));
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // biased
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// inv_freq (radians) as a 64-bit binary fraction of a turn: the 53-bit
// significand times 2^65 / pi, shifted into place.  All in integers: this
// GPU's fp64 units would take longer over a block's angles than its rows.
__device__ __forceinline__ uint64_t turns_of(double inv_freq)
{
    constexpr uint64_t kTurn = 0xa2f9836e4e441529ull;               // floor(2^65 / pi) = 2^66 / (2 pi)
    const uint64_t b = (uint64_t)__double_as_longlong(inv_freq);
    const int e = (int)(b >> 52) & 0x7ff;
    if (e == 0 || e > 1023 + 52)                       // zero and what is no frequency
        return 0;
    const uint64_t m = (b & 0xfffffffffffffull) | (1ull << 52);
    const uint64_t lo = m * kTurn;
    const uint64_t hi = __umul64hi(m, kTurn);
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

template <int IT>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8])
{
    unpack_vec<IT>(w, x);
}

template <int IT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack2(round_to<IT>(x[0]), round_to<IT>(x[1])),
                      pack2(round_to<IT>(x[2]), round_to<IT>(x[3])),
                      pack2(round_to<IT>(x[4]), round_to<IT>(x[5])),
                      pack2(round_to<IT>(x[6]), round_to<IT>(x[7])));
}

// Eight values -> eight E4M3 codes of value * inv, saturating.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv)
{
    return make_uint2(pack2(e4m3x2_satfinite(x[0] * inv, x[1] * inv),
                            e4m3x2_satfinite(x[2] * inv, x[3] * inv)),
                      pack2(e4m3x2_satfinite(x[4] * inv, x[5] * inv),
                            e4m3x2_satfinite(x[6] * inv, x[7] * inv)));
}

// A lane's 8-element vector `c` of a row, and how the rotation reaches it.
struct Place {
    bool rotated;
    bool inter;        // pairs inside the vector
    int partner;       // lane that holds the other halves of this lane's pairs
    float sign;        // -1 for the first halves, +1 for the second
    int freq;          // first frequency
};

__device__ __forceinline__ Place place_of(int c, int lane, int rot, bool interleaved)
{
    Place pl;
    const int h = rot / 16;                      // vectors in half of the rotated part
    pl.rotated = c < 2 * h;
    pl.inter = interleaved;
    const bool first = c < h;
    pl.partner = (pl.rotated && !interleaved) ? (first ? lane + h : lane - h) : lane;
    pl.sign = first ? -1.f : 1.f;
    pl.freq = !pl.rotated ? 0 : (interleaved ? 4 * c : 8 * (first ? c : c - h));
    return pl;
}

// Rotate a lane's vector; cs: cosine and sine (already times m) of the
// vector's frequencies: 4 of them for pairs inside the vector, 8 otherwise.
// Called by whole warps (the other halves come by shuffle).
template <int IT>
__device__ __forceinline__ void rotate8(const uint4& w, const Place& pl, const float2* cs,
                                        float (&y)[8])
{
    float x[8];
    unpack8<IT>(w, x);
    if (pl.inter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = cs[i];
            y[2 * i] = pl.rotated ? x[2 * i] * z.x - x[2 * i + 1] * z.y : x[2 * i];
            y[2 * i + 1] = pl.rotated ? x[2 * i + 1] * z.x + x[2 * i] * z.y : x[2 * i + 1];
        }
        return;
    }
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, w.x, pl.partner);
    o.y = __shfl_sync(0xffffffffu, w.y, pl.partner);
    o.z = __shfl_sync(0xffffffffu, w.z, pl.partner);
    o.w = __shfl_sync(0xffffffffu, w.w, pl.partner);
    float b[8];
    unpack8<IT>(o, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 z = cs[i];
        y[i] = pl.rotated ? x[i] * z.x + pl.sign * (b[i] * z.y) : x[i];
    }
}

template <int MODE, int IT, int D, int BS>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p)
{
    constexpr int VPR = D / 8;                    // vectors per row
    constexpr int RPI = 32 / VPR;                 // rows per warp access
    constexpr int NV = BS / RPI;                  // vectors a lane holds of a block
    constexpr int C = MODE == kSame ? 2 : 1;      // cache bytes per element
    __shared__ float2 sh_cs[BS * (D / 2)];

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

    // cosines and sines of the block's tokens
    const int rh = p.rot_dim / 2;
    for (int i = threadIdx.x; i < T * rh; i += kThreads) {
        const int t = i / rh;
        const int f = i - t * rh;
        float sn, cn;
        sincospif(half_turns(turns_of(__ldg(p.inv_freq + f)), lo + t), &sn, &cn);
        sh_cs[t * rh + f] = make_float2(cn * p.mscale, sn * p.mscale);
    }
    __syncthreads();

    const int phys = __ldg(p.block_tables + (int64_t)s * p.max_blocks_per_seq + blk);
    const bool good = phys >= 0 && (int64_t)phys < p.num_blocks;
    if (!good && threadIdx.x == 0 && part == 0)
        flag_error(p.dev_err, PKV_DEVERR_BLOCK_ID);

    const int c = lane % VPR;
    const int rsub = lane / VPR;
    const bool inter = p.interleaved != 0;
    const Place pl = place_of(c, lane, p.rot_dim, inter);
    const int ncs = inter ? 4 : 8;
    const int kv_tasks = 2 * p.num_kv_heads;
    const int hchunks = p.q != nullptr ? (p.num_heads + kHeadsPerTask - 1) / kHeadsPerTask : 0;
    const int tasks = kv_tasks + T * hchunks;
    for (int task = part * kWarps + warp; task < tasks; task += split * kWarps) {
        if (task < kv_tasks) {
            if (!good)
                continue;
            const int g = task >> 1;
            const bool is_v = task & 1;
            const uint16_t* src =
                reinterpret_cast<const uint16_t*>(is_v ? p.v : p.k) + (int64_t)g * D + c * 8;
            const int64_t stride = is_v ? p.v_stride : p.k_stride;
            uint4 w[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int t = i * RPI + rsub;
                w[i] = t < T ? ld_ro(src + (row0 + t) * stride) : make_uint4(0, 0, 0, 0);
            }
            char* tile = reinterpret_cast<char*>(is_v ? p.v_cache : p.k_cache) +
                         ((int64_t)phys * p.num_kv_heads + g) * (BS * D) * C;
            float inv = is_v ? p.v_inv_scale : p.k_inv_scale;
            if constexpr (MODE == kScaled) {
                float* sp = p.scales + ((int64_t)phys * p.num_kv_heads + g) * 2 + (is_v ? 1 : 0);
                const float old = off > 0 ? *sp : 0.f;
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float x[8];
                    unpack8<IT>(w[i], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = fabsf(x[e]);
                        mx = a < __int_as_float(0x7f800000) ? fmaxf(mx, a) : mx;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float need = power_of_two(is_v ? mx : mx * p.k_bound);
                const float sc = off > 0 ? fmaxf(old, need) : need;
                inv = 1.f / sc;
                if (off > 0 && sc != old) {
                    // the older tokens' codes follow the scale
                    const float f = old / sc;
                    for (int i = lane; i < off * (D / 8); i += 32) {
                        uint2* cp = reinterpret_cast<uint2*>(tile) + i;
                        const uint2 u = *cp;
                        float x[8];
                        const uint32_t ww[2] = {u.x, u.y};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t h0, h1;
                            e4m3x4_to_f16x2(ww[j], h0, h1);
                            const float2 a = f16x2_to_float2(h0);
                            const float2 b = f16x2_to_float2(h1);
                            x[4 * j] = a.x, x[4 * j + 1] = a.y;
                            x[4 * j + 2] = b.x, x[4 * j + 3] = b.y;
                        }
                        *cp = codes8(x, f);
                    }
                }
                if (lane == 0)
                    *sp = sc;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int t = i * RPI + rsub;
                if (i * RPI >= T)                     // warp-uniform
                    break;
                char* dst = tile + ((int64_t)(off + t) * D + c * 8) * C;
                float y[8];
                if (is_v || p.rot_dim == 0) {
                    if constexpr (MODE == kSame) {
                        if (t < T)
                            st_v4(dst, w[i]);
                        continue;
                    }
                    unpack8<IT>(w[i], y);
                } else {
                    const float2* cs = sh_cs + min(t, T - 1) * rh + pl.freq;
                    float2 z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = e < ncs && pl.rotated ? cs[e] : make_float2(1.f, 0.f);
                    rotate8<IT>(w[i], pl, z, y);
                }
                if (t < T) {
                    if constexpr (MODE == kSame)
                        st_v4(dst, pack8<IT>(y));
                    else
                        *reinterpret_cast<uint2*>(dst) = codes8(y, inv);
                }
            }
        } else {
            const int qt = task - kv_tasks;
            const int t = qt / hchunks;
            const int h0 = (qt - t * hchunks) * kHeadsPerTask;
            const int h1 = min(p.num_heads, h0 + kHeadsPerTask);
            const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + (row0 + t) * p.q_stride;
            uint16_t* dst = reinterpret_cast<uint16_t*>(p.q_out) + (row0 + t) * p.num_heads * D;
            const float2* cs = sh_cs + t * rh + pl.freq;
            float2 z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = e < ncs && pl.rotated ? cs[e] : make_float2(1.f, 0.f);
            constexpr int NQ = kHeadsPerTask / RPI;
            uint4 w[NQ];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int h = h0 + i * RPI + rsub;
                w[i] = h < h1 ? *reinterpret_cast<const uint4*>(src + (int64_t)h * D + c * 8)
                              : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const int h = h0 + i * RPI + rsub;
                float y[8];
                rotate8<IT>(w[i], pl, z, y);
                if (h < h1)
                    st_v4(dst + (int64_t)h * D + c * 8, pack8<IT>(y));
            }
        }
    }
}

template <int MODE, int IT, int D, int BS>
cudaError_t run(const RopeParams& p, int sms, cudaStream_t stream)
{
    const int64_t ntouch = (p.max_q_len + BS - 2) / BS + 1;
    // few blocks (a decode step): several CTAs share the rows of each block,
    // down to one warp task each
    const int T = p.max_q_len < BS ? p.max_q_len : BS;
    const int64_t hchunks = p.q ? (p.num_heads + kHeadsPerTask - 1) / kHeadsPerTask : 0;
    const int64_t tasks = 2 * p.num_kv_heads + T * hchunks;
    int64_t split = (4 * (int64_t)sms) / (ntouch * p.num_seqs);
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
