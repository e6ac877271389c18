// decode_weights.cu -- a decode step over a scaled cache that adds its attention
// weights to a running total per token and KV head.
//
//   p_h(t) = exp(x_ht - max x_h) / sum_t exp(x_ht - max x_h),  weights[t] += sum_h p_h(t)
// over the query heads h of a KV head.  The softmax is known only once the whole
// context has been seen, so the decode kernel files every score x (fp32, log2) as
// it goes; who has the maximum and the sum turns scores into weights: the CTA
// itself where it holds the context, else CTAs of the reduce kernel's launch.
// Scores cost 4 bytes a query head and token, written and read (K and V: 256
// bytes a token at D = 128); the second read is mostly from L2.
#include <cuda_runtime.h>

#include "decode_scaled_kernel.cuh"

namespace pkv {
namespace {

using namespace dsk;

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
    const int64_t chunks = ((int64_t)p.max_context_len + kWeightTokens - 1) / kWeightTokens;
    return launch_early(reduce_shares_kernel<QT, D, kWeights>,
                        (rows + kReduceRows - 1) / kReduceRows +
                            chunks * p.num_seqs * p.num_kv_heads,
                        kReduceRows * 32, stream, p, ctas, 8 * NNT, x);
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
