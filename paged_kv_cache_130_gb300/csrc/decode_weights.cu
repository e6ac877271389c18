// decode_weights.cu -- a decode step over a scaled cache that adds its attention
// weights to a running total per token and KV head.
//
//   p_h(t) = exp(x_ht - max x_h) / sum_t exp(x_ht - max x_h),  weights[t] += sum_h p_h(t)
// over the query heads h of a KV head.  The softmax is known only once the whole
// context has been seen, so the decode kernel files every score x (fp32, log2) as
// it goes; who has the maximum and the sum turns scores into weights: the CTA
// itself where it holds the context, else a kernel behind the reduce, which files
// every row's maximum and 1 / sum.
// Scores cost 4 bytes a query head and token, written and read (K and V: 256
// bytes a token at D = 128), the read mostly from L2; totals another 8 bytes.
// Measured: 64 sequences of 1,024..4,096 tokens (64 heads over 8) 80 us: decode 66, reduce 6,
// weights 10; 16 of 8,192..32,768 (32 heads of their own) 424: 402, 6, 21.  Weights
// added in the reduce's launch, a CTA per run of tokens: 87 and 443; the next item's
// first blocks fetched ahead: 407 instead of 375 without weights.
#include <cuda_runtime.h>

#include "decode_scaled_kernel.cuh"

namespace pkv {
namespace {

using namespace dsk;

constexpr int kAddThreads = 256;
constexpr int kAddTokens = 4;              // of a thread

// One CTA = kAddThreads * kAddTokens tokens of one (sequence, KV head).
template <int PITCH>
__global__ void __launch_bounds__(kAddThreads) add_weights_kernel(const DecodeParams p, const DecodeExtra x)
{
    constexpr int V = PITCH < 4 ? PITCH : 4;   // scores to a load
    __shared__ float2 fin[PITCH];
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads;
    const int64_t item = blockIdx.x % items;
    const int s = (int)(item / p.num_kv_heads);
    const int head = (int)(item - (int64_t)s * p.num_kv_heads);
    const int first = (int)(blockIdx.x / items) * (kAddThreads * kAddTokens) + threadIdx.x;
    int ctx = __ldg(p.context_lens + s);       // (older than the kernels before)
    if (ctx > p.max_context_len || ctx > p.max_blocks_per_seq * p.block_size)
        ctx = 0;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (first - (int)threadIdx.x >= ctx)
        return;
    const float* sc = x.scores + item * x.score_tokens * PITCH;
    float* w = x.weights + s * x.weights_seq + head * x.weights_head;
    float v[kAddTokens][PITCH], before[kAddTokens];
#pragma unroll
    for (int i = 0; i < kAddTokens; ++i) {
        const int t = first + i * kAddThreads;
        before[i] = t < ctx ? w[t] : 0.f;
#pragma unroll
        for (int r = 0; r < PITCH; r += V) {
            const float* at = sc + (int64_t)min(t, ctx - 1) * PITCH + r;
            if constexpr (V == 4) {
                const float4 u = __ldcg(reinterpret_cast<const float4*>(at));
                v[i][r] = u.x, v[i][r + 1] = u.y, v[i][r + 2] = u.z, v[i][r + 3] = u.w;
            } else if constexpr (V == 2) {
                const float2 u = __ldcg(reinterpret_cast<const float2*>(at));
                v[i][r] = u.x, v[i][r + 1] = u.y;
            } else {
                v[i][r] = __ldcg(at);
            }
        }
    }
    if (threadIdx.x < PITCH)
        fin[threadIdx.x] = (int)threadIdx.x < p.group
                               ? __ldcg(x.whole + (int64_t)s * p.num_heads + head * p.group + threadIdx.x)
                               : make_float2(0.f, 0.f);
    __syncthreads();
    float sum[kAddTokens] = {};
#pragma unroll
    for (int r = 0; r < PITCH; ++r) {
        const float2 f = fin[r];
        if (r < p.group)
#pragma unroll
            for (int i = 0; i < kAddTokens; ++i)
                if (v[i][r] != dec::kNegInf)
                    sum[i] = fmaf(exp2_fast(v[i][r] - f.x), f.y, sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kAddTokens; ++i)
        if (first + i * kAddThreads < ctx)
            w[first + i * kAddThreads] = before[i] + sum[i];
}

template <int QT, int D, int BS, int NNT>
cudaError_t run(const DecodeParams& p, const float* scales, const DecodeExtra& x, int sms,
                cudaStream_t stream)
{
    const float2* sc = reinterpret_cast<const float2*>(scales);
    if (p.partition_size > 0)
        return launch_early(decode_scaled_kernel<QT, D, BS, NNT, false, kWeights>,
                            (int64_t)p.num_seqs * p.num_kv_heads, kWarps * 32, stream, p, sc, x);
    const int64_t ctas = decode_scaled_ctas(p.group, sms);
    cudaError_t e = launch_early(decode_scaled_kernel<QT, D, BS, NNT, true, kWeights>, ctas,
                                 kWarps * 32, stream, p, sc, x);
    if (e != cudaSuccess)
        return e;
    const int64_t rows = (int64_t)p.num_seqs * p.num_heads;
    e = launch_early(reduce_shares_kernel<QT, D, kWeights>, (rows + kReduceRows - 1) / kReduceRows,
                     kReduceRows * 32, stream, p, ctas, 8 * NNT, x);
    if (e != cudaSuccess)
        return e;
    const int64_t chunks = ((int64_t)p.max_context_len + kAddThreads * kAddTokens - 1) / (kAddThreads * kAddTokens);
    const int64_t grid = chunks * p.num_seqs * p.num_kv_heads;
    switch (x.pitch) {
    case 1: return launch_early(add_weights_kernel<1>, grid, kAddThreads, stream, p, x);
    case 2: return launch_early(add_weights_kernel<2>, grid, kAddThreads, stream, p, x);
    case 4: return launch_early(add_weights_kernel<4>, grid, kAddThreads, stream, p, x);
    case 8: return launch_early(add_weights_kernel<8>, grid, kAddThreads, stream, p, x);
    default: return launch_early(add_weights_kernel<16>, grid, kAddThreads, stream, p, x);
    }
}

template <int QT, int D, int BS>
cudaError_t by_rows(const DecodeParams& p, const float* scales, const DecodeExtra& x, int sms, cudaStream_t st)
{
    return p.group <= 8 ? run<QT, D, BS, 1>(p, scales, x, sms, st)
                     : run<QT, D, BS, 2>(p, scales, x, sms, st);
}

template <int QT, int D>
cudaError_t by_block(const DecodeParams& p, const float* scales, const DecodeExtra& x, int sms, cudaStream_t st)
{
    switch (p.block_size) {
    case 8: return by_rows<QT, D, 8>(p, scales, x, sms, st);
    case 16: return by_rows<QT, D, 16>(p, scales, x, sms, st);
    case 32: return by_rows<QT, D, 32>(p, scales, x, sms, st);
    default: return cudaErrorNotSupported;
    }
}

template <int QT>
cudaError_t by_dim(const DecodeParams& p, const float* scales, const DecodeExtra& x, int sms, cudaStream_t st)
{
    return p.head_dim == 128 ? by_block<QT, 128>(p, scales, x, sms, st)
                             : by_block<QT, 64>(p, scales, x, sms, st);
}

}  // namespace

cudaError_t launch_decode_weights(const DecodeParams& p, const float* scales, const DecodeExtra& x,
                                  int sms, cudaStream_t stream)
{
    if (p.num_seqs <= 0)
        return cudaSuccess;
    if (p.group < 1 || p.group > kMaxGroup || p.num_seqs > kWeightsSeqs)
        return cudaErrorNotSupported;
    static_assert(kWeightsSeqs <= kMaxBalanced, "sequences that a CTA scans");
    return p.q_dtype == kF16 ? by_dim<kF16>(p, scales, x, sms, stream)
                             : by_dim<kBF16>(p, scales, x, sms, stream);
}

}  // namespace pkv
