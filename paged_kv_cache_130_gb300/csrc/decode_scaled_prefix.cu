// decode_scaled_prefix.cu -- decode over a scaled cache for groups of sequences that
// share their leading blocks.
//
// Attention over [0, c) splits at the end P of the shared prefix.  Both parts are
// items of the equal shares of decode_scaled_kernel.cuh: a prefix for every 8 or 16
// rows (members x query heads of a KV head) of its group, read for all of them
// at once, and each sequence's tokens from P on.  The reduce merges what belongs
// to a row.
#include <cuda_runtime.h>

#include "decode_scaled_kernel.cuh"

namespace pkv {
namespace {

using namespace dsk;

int rows_of(int32_t group, int32_t max_group_size)
{
    return group > 8 || (int64_t)group * max_group_size > 8 ? 16 : 8;
}

template <int QT, int D, int BS, int NNT>
cudaError_t run(const DecodeParams& p, const float* scales, int sms, cudaStream_t stream)
{
    const int64_t ctas = decode_scaled_ctas(8 * NNT, sms);
    cudaError_t e = launch_early(decode_scaled_kernel<QT, D, BS, NNT, true, kShared>, ctas,
                                 kWarps * 32, stream, p, reinterpret_cast<const float2*>(scales),
                                 DecodeExtra{});
    if (e != cudaSuccess)
        return e;
    const int64_t rows = (int64_t)p.num_seqs * p.num_heads;
    return launch_early(reduce_shares_kernel<QT, D, kShared>, (rows + kReduceRows - 1) / kReduceRows,
                        kReduceRows * 32, stream, p, ctas, 8 * NNT, DecodeExtra{});
}

template <int QT, int D, int BS>
cudaError_t by_rows(const DecodeParams& p, const float* scales, int sms, cudaStream_t st)
{
    return rows_of(p.group, p.max_group_size) == 8 ? run<QT, D, BS, 1>(p, scales, sms, st)
                     : run<QT, D, BS, 2>(p, scales, sms, st);
}

template <int QT, int D>
cudaError_t by_block(const DecodeParams& p, const float* scales, int sms, cudaStream_t st)
{
    switch (p.block_size) {
    case 8: return by_rows<QT, D, 8>(p, scales, sms, st);
    case 16: return by_rows<QT, D, 16>(p, scales, sms, st);
    case 32: return by_rows<QT, D, 32>(p, scales, sms, st);
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

cudaError_t launch_decode_scaled_prefix(const DecodeParams& p, const float* scales, int sms,
                                        cudaStream_t stream)
{
    if (p.num_seqs <= 0)
        return cudaSuccess;
    if (p.group < 1 || p.group > kMaxGroup || p.num_groups < 1 ||
        (int64_t)p.num_groups + p.num_seqs > kSharedEntries)
        return cudaErrorNotSupported;
    return p.q_dtype == kF16 ? by_dim<kF16>(p, scales, sms, stream)
                             : by_dim<kBF16>(p, scales, sms, stream);
}

// Two pieces a CTA, and the rows of items that one CTA held whole, prefixes and
// own tokens.
int64_t decode_prefix_rows(int32_t num_seqs, int32_t num_heads, int32_t group,
                           int32_t max_group_size, int sms)
{
    const int rt = rows_of(group, max_group_size);
    return 2 * decode_scaled_ctas(rt, sms) * rt + 2 * (int64_t)num_seqs * num_heads;
}

}  // namespace pkv
