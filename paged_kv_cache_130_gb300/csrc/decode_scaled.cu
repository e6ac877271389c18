// decode_scaled.cu -- decode attention over an E4M3 cache with a scale per
// block and KV head.
//
// With code c and the block's scales ks, vs:
//   x_t = (scale ks) (q . ck_t),   out = sum_t exp(x_t - m) vs cv_t / sum_t exp(x_t - m).
// A scale belongs to a whole block of one head, so it never touches the
// elements: ks multiplies the token's score, vs its softmax weight.  The codes
// go to the tensor cores as fp16, in which every E4M3 value is exact.
//
// One CTA takes one partition of one sequence and KV head with up to 16 query
// heads; its warps stride over the partition in steps of 16 tokens.  Lane
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
//     fp16 (11 bits, relative 2^-12 at most each) after the multiplication by
//     vs / vref 2^6, vref = the largest vs so far: fp16 keeps that exact to
//     ratios of 2^-20, and what it loses below is 2^-31 of vref's block.
// The running maximum, sums and the output accumulators are fp32.
#include <cuda_runtime.h>

#include "decode_common.cuh"
#include "pkv_common.cuh"
#include "scaled_internal.h"

namespace pkv {
namespace {

using dec::ceil_div_i;
using dec::kNegInf;
using dec::PartitionWork;

constexpr int kWarps = 4;
constexpr int kRows = 16;              // query heads a CTA holds at most
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

template <int QT, int D, int BS, int NNT>
__global__ void __launch_bounds__(kWarps * 32, NNT == 1 ? 3 : 2)
    decode_scaled_kernel(const DecodeParams p, const float2* __restrict__ scales)
{
    constexpr int NKS = D / 16;                // k-steps of the scores
    constexpr int NM = D / 16;                 // m-tiles of the output
    constexpr int NKV = D / 64;                // 16-byte vectors of a K row per lane
    constexpr int BPS = BS == 8 ? 2 : 1;       // blocks per step
    constexpr int SPB = BS == 32 ? 2 : 1;      // steps per block

    extern __shared__ __align__(16) float smem[];
    float* sm_m = smem;                        // [kWarps][16]
    float* sm_l = sm_m + kWarps * kRows;
    float* sm_acc = sm_l + kWarps * kRows;     // [kWarps][16][D]
    __shared__ float sm_q[kRows];              // 1 / the heads' q scales
    __shared__ uint2 sm_qf[NNT * NKS * 32];    // q fragments by lane

    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int g = lane >> 2;
    const int t = lane & 3;
    const int G = p.group;
    int64_t idx = blockIdx.x;
    const int head = (int)(idx % p.num_kv_heads);
    idx /= p.num_kv_heads;
    const int srank = (int)(idx % p.num_seqs);
    const int part = (int)(idx / p.num_seqs);

    // longest context first for batches of up to 128 sequences (ties by index)
    int s = srank;
    if (p.num_seqs <= 128) {
        __shared__ int sh_ctx[128];
        __shared__ int sh_seq;
        for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x)
            sh_ctx[i] = __ldg(p.context_lens + i);
        __syncthreads();
        for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x) {
            const int ci = sh_ctx[i];
            int rank = 0;
            for (int j = 0; j < p.num_seqs; ++j)
                rank += (sh_ctx[j] > ci) || (sh_ctx[j] == ci && j < i);
            if (rank == srank)
                sh_seq = i;
        }
        __syncthreads();
        s = sh_seq;
    }
    pdl_launch_dependents();

    const PartitionWork w = dec::locate(p, s, part, threadIdx.x == 0);
    if (w.idle || w.zero_out || w.zero_partial) {
        if (!w.idle)
            dec::write_trivial<QT>(p, w, head * G, G, threadIdx.x, blockDim.x);
        return;
    }

    // q: each warp scales rows warp, warp + 4, ... by a power of two that
    // brings the largest element into [2^13, 2^14), and files the fragments
    for (int r = warp; r < 8 * NNT; r += kWarps) {
        constexpr int EPL = D / 32;            // elements per lane
        float x[EPL];
        float mx = 0.f;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) +
                              ((int64_t)s * p.num_heads + head * G + r) * D;
#pragma unroll
        for (int e = 0; e < EPL; e += 2) {
            const uint32_t u =
                r < G ? __ldg(reinterpret_cast<const uint32_t*>(src) + (lane * EPL + e) / 2) : 0u;
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

    const int t_begin = w.t_begin;
    const int t_end = w.t_end;
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
            if (g == 0) {
                sm_m[warp * kRows + r] = m_h[n][h];
                sm_l[warp * kRows + r] = l;
            }
            float* o = sm_acc + (int64_t)(warp * kRows + r) * D + g * (D / 8);
#pragma unroll
            for (int j = 0; j < NM; ++j) {
                o[2 * j] = acc[n][j][h] * ov;
                o[2 * j + 1] = acc[n][j][h + 2] * ov;
            }
        }
    __syncthreads();
    dec::finish_rows<QT, kWarps, kRows>(p, w, head * G, G, sm_m, sm_l, sm_acc, threadIdx.x,
                                        blockDim.x);
}

template <int QT, int D, int BS, int NNT>
cudaError_t run(const DecodeParams& p, const float* scales, cudaStream_t stream)
{
    auto kern = decode_scaled_kernel<QT, D, BS, NNT>;
    const int smem = (2 * kWarps * kRows + kWarps * kRows * D) * (int)sizeof(float);
    const int64_t ctas = (int64_t)p.grid_partitions * p.num_seqs * p.num_kv_heads;
    if (ctas > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)ctas, kWarps * 32, smem, stream>>>(p, reinterpret_cast<const float2*>(scales));
    return cudaGetLastError();
}

template <int QT, int D, int BS>
cudaError_t by_group(const DecodeParams& p, const float* scales, cudaStream_t st)
{
    return p.group <= 8 ? run<QT, D, BS, 1>(p, scales, st) : run<QT, D, BS, 2>(p, scales, st);
}

template <int QT, int D>
cudaError_t by_block(const DecodeParams& p, const float* scales, cudaStream_t st)
{
    switch (p.block_size) {
    case 8: return by_group<QT, D, 8>(p, scales, st);
    case 16: return by_group<QT, D, 16>(p, scales, st);
    case 32: return by_group<QT, D, 32>(p, scales, st);
    default: return cudaErrorNotSupported;
    }
}

template <int QT>
cudaError_t by_dim(const DecodeParams& p, const float* scales, cudaStream_t st)
{
    return p.head_dim == 128 ? by_block<QT, 128>(p, scales, st) : by_block<QT, 64>(p, scales, st);
}

}  // namespace

cudaError_t launch_decode_scaled(const DecodeParams& p, const float* scales, cudaStream_t stream)
{
    if (p.num_seqs <= 0)
        return cudaSuccess;
    if (p.group < 1 || p.group > kRows)
        return cudaErrorNotSupported;
    return p.q_dtype == kF16 ? by_dim<kF16>(p, scales, stream) : by_dim<kBF16>(p, scales, stream);
}

// Tokens per partition: one partition per context when the (sequence, KV head)
// items alone fill the GPU twice, else about 128 KiB of K and V codes per item.
int32_t decode_scaled_partition(const DecodeParams& p, int sms)
{
    const int32_t bs = p.block_size;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    if (items >= 6LL * sms && p.max_context_len <= 8192)
        return (p.max_context_len + bs - 1) / bs * bs;
    return (1 << 17) / (2 * p.head_dim);
}

}  // namespace pkv
