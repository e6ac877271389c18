// decode_scaled.cu -- decode attention over a scaled cache: launches of the plain
// kernels, and how contexts are cut.
#include <cuda_runtime.h>

#include "decode_scaled_kernel.cuh"

namespace pkv {
namespace {

using namespace dsk;

template <int QT, int D, int BS, int NNT>
cudaError_t run(const DecodeParams& p, const float* scales, int sms, cudaStream_t stream)
{
    const float2* sc = reinterpret_cast<const float2*>(scales);
    if (p.partition_size > 0)
        return launch_early(decode_scaled_kernel<QT, D, BS, NNT, false, kPlain>,
                            (int64_t)p.grid_partitions * p.num_seqs * p.num_kv_heads, kWarps * 32,
                            stream, p, sc, DecodeExtra{});
    const int64_t ctas = decode_scaled_ctas(p.group, sms);
    cudaError_t e = launch_early(decode_scaled_kernel<QT, D, BS, NNT, true, kPlain>, ctas, kWarps * 32,
                                 stream, p, sc, DecodeExtra{});
    if (e != cudaSuccess)
        return e;
    const int64_t rows = (int64_t)p.num_seqs * p.num_heads;
    return launch_early(reduce_shares_kernel<QT, D, kPlain>, (rows + kReduceRows - 1) / kReduceRows,
                        kReduceRows * 32, stream, p, ctas, 8 * NNT, DecodeExtra{});
}

template <int QT, int D, int BS>
cudaError_t by_group(const DecodeParams& p, const float* scales, int sms, cudaStream_t st)
{
    return p.group <= 8 ? run<QT, D, BS, 1>(p, scales, sms, st)
                        : run<QT, D, BS, 2>(p, scales, sms, st);
}

template <int QT, int D>
cudaError_t by_block(const DecodeParams& p, const float* scales, int sms, cudaStream_t st)
{
    switch (p.block_size) {
    case 8: return by_group<QT, D, 8>(p, scales, sms, st);
    case 16: return by_group<QT, D, 16>(p, scales, sms, st);
    case 32: return by_group<QT, D, 32>(p, scales, sms, st);
    default: return cudaErrorNotSupported;
    }
}

template <int QT>
cudaError_t by_dim(const DecodeParams& p, const float* scales, int sms, cudaStream_t st)
{
    return p.head_dim == 128 ? by_block<QT, 128>(p, scales, sms, st)
                             : by_block<QT, 64>(p, scales, sms, st);
}

}  // namespace

cudaError_t launch_decode_scaled(const DecodeParams& p, const float* scales, int sms,
                                 cudaStream_t stream)
{
    if (p.num_seqs <= 0)
        return cudaSuccess;
    if (p.group < 1 || p.group > kMaxGroup)
        return cudaErrorNotSupported;
    return p.q_dtype == kF16 ? by_dim<kF16>(p, scales, sms, stream)
                             : by_dim<kBF16>(p, scales, sms, stream);
}

// Resident CTAs: the registers of three fit an SM with 8 heads, of two with 16.
int64_t decode_scaled_ctas(int32_t group, int sms) { return (group <= 8 ? 3 : 2) * (int64_t)sms; }

int64_t decode_scaled_partial_rows(int32_t group, int sms)
{
    return 2 * decode_scaled_ctas(group, sms) * (group <= 8 ? 8 : 16);
}

// One CTA per (sequence, KV head), in one launch, while the longest context is
// short; equal shares beyond, unless there are more sequences than a CTA scans.
// Measured, D = 128, one pass / shares in us: 32 items of 128..512 tokens 7.3 /
// 11.5, 128 (8 heads each) of 128..512 8.6 / 15.5, 1,024 of 256..1024 44 / 44, of
// 512..2048 76 / 71, of 1024..4096 137 / 120, 2,048 of 256..1024 70 / 69, of
// 1024..4096 232 / 216, 8,192 of 256..1024 249 / 248, of 2048..8192 1633 / 1634:
// the shares' second launch and walk against the imbalance of the last wave.
// Few items of exactly 256, 512, 768, 1,024 tokens, 8 heads each, D = 128:
//   1 item    6.7 /  8.5   9.3 / 11.3  11.8 / 12.4  14.1 / 11.9
//   8 items   6.5 / 13.0   9.1 / 12.9  11.6 / 13.6  13.9 / 13.4
//   32 items  6.7 / 13.5  10.5 / 14.1  13.8 / 14.7  17.0 / 15.1
// and D = 64: 1 item 5.5 / 7.2, 7.5 / 9.6, 9.4 / 10.7, 11.2 / 10.3; 32 items 5.6 /
// 11.4, 7.7 / 11.5, 9.8 / 12.0, 13.6 / 12.9.  One pass loses up to a sixth at its
// very end.  Explicit partitions of 256 tokens beat both there (D = 128: 7.7,
// 7.8 and 7.8 us for 1 item of 512, 768, 1,024; 32 items 8.4, 8.8 and 9.0).
int32_t decode_scaled_partition(const DecodeParams& p)
{
    const int32_t bs = p.block_size < 16 ? 16 : p.block_size;
    if (p.max_context_len <= kOnePass)
        return (p.max_context_len + bs - 1) / bs * bs;
    return p.num_seqs <= kMaxBalanced ? 0 : (1 << 19) / (2 * p.head_dim);
}

}  // namespace pkv
