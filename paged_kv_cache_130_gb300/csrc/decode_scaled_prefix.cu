// decode_scaled_prefix.cu -- decode over a scaled cache for groups of sequences that
// share their leading blocks.
//
// Attention over [0, c) splits at the end P of the shared prefix.  Few rows (members
// x query heads of a KV head): both parts are items of the equal shares of
// decode_scaled_kernel.cuh: a prefix for every 8 or 16 rows of its group, read for
// all of them at once, and each sequence's tokens from P on.  Many rows: the
// prefixes go to the tensor-memory kernel of prefill_scaled_kernel.cuh, 256 rows a
// CTA and the keys in runs, beside which the shares hold the own tokens only.  The
// reduce merges what belongs to a row.
//
// Bound by latency in small groups, by the start of an item (a CTA has ~8 of them)
// where prefixes are short, by the prefix kernel and the shares in turn (an SM holds
// one or the other) where one is long.  Measured: 16 prompts of 504 tokens with six
// samples of 16..512 tokens each (32 heads, D 128, fp16) 84 us (shares 77, reduce 10);
// 64 sequences of 64..1,024 tokens behind a prompt of 8,192 (64 heads over 8, bf16)
// 61 us (prefix 29, shares 24, reduce 10).  Items of up to 16 rows that hold the prefix
// and their own tokens in one softmax: 81 and 75.
#include <cuda_runtime.h>

#include <atomic>

#include "decode_scaled_kernel.cuh"
#include "prefill_scaled_kernel.cuh"

namespace pkv {
namespace {

using namespace dsk;

constexpr int kKeys = pfs::kKeys;
// Rows of a group beyond which prefixes have their own kernel.  Shares only / own
// kernel, us, 64 heads over 8, own tokens 32..64 (D 128, 16 tokens a block):
//   rows                            16       32       48       64       128
//   1 prefix of 2,048 tokens      21 / 23  23 / 23  23 / 23  24 / 23   26 / 24
//   1 of 16,384                   27 / 33  33 / 34  41 / 36  50 / 43   84 / 45
//   8 of 2,048                    26 / 31  36 / 41  47 / 41  60 / 41  114 / 52
//   15 of 1,024                   28 / 40  41 / 41  56 / 45  74 / 50  139 / 70
// Where groups x KV heads keep the GPU busy anyhow, beyond half as many: 16 heads of
// their own, rows                  16       24       32       48
//   8 of 2,048                    60 / 65  91 / 75 105 / 84 156 / 108
//   15 of 1,024                   90 / 90 135 / 110 162 / 129 239 / 168
//   1 of 16,384                   35 / 50  48 / 50  48 / 51  66 / 53
constexpr int kManyRows = 32;
constexpr int kManyItems = 128;
constexpr int kMinRun = 4 * kKeys;         // keys of a CTA of it

bool many_rows(int32_t num_groups, int32_t num_kv_heads, int32_t group, int32_t max_group_size)
{
    const bool busy = (int64_t)num_groups * num_kv_heads >= kManyItems;
    return (int64_t)group * max_group_size > (busy ? kManyRows / 2 : kManyRows);
}

// Rows of an item of the shares.
int rows_of(int32_t num_groups, int32_t num_kv_heads, int32_t group, int32_t max_group_size)
{
    const int64_t rows = many_rows(num_groups, num_kv_heads, group, max_group_size)
                             ? group
                             : (int64_t)group * max_group_size;
    return group > 8 || rows > 8 ? 16 : 8;
}

// CTAs of one run over every group's prefix, and the most runs: what fills the GPU
// once.
int64_t ctas_of_run(int32_t num_groups, int32_t num_kv_heads, int32_t group, int32_t max_group_size)
{
    const int span = 2 * (pfs::kRows / group);
    return (int64_t)num_groups * num_kv_heads * ((max_group_size + span - 1) / span);
}

int64_t most_runs(int32_t num_groups, int32_t num_kv_heads, int32_t group, int32_t max_group_size, int sms)
{
    const int64_t n = sms / ctas_of_run(num_groups, num_kv_heads, group, max_group_size);
    return n < 1 ? 1 : n;
}

// The prefixes' own kernel.
template <int QT, int D, int BS>
cudaError_t run_prefixes(const DecodeParams& p, const float* scales, int64_t first_row, cudaStream_t stream)
{
    using L = pfs::Layout<D>;
    auto kern = pfs::prefill_scaled_kernel<QT, D, BS, true>;
    static std::atomic<bool> configured[64];      // (threads may call at once)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::alloc);
        if (e != cudaSuccess)
            return e;
        configured[dev] = true;
    }
    ScaledPrefillParams sp{};
    sp.p.k_cache = p.k_cache;
    sp.p.v_cache = p.v_cache;
    sp.p.num_blocks = p.num_blocks;
    sp.p.num_kv_heads = p.num_kv_heads;
    sp.p.block_size = p.block_size;
    sp.p.head_dim = p.head_dim;
    sp.p.dtype = p.q_dtype;
    sp.p.q = p.q;
    sp.p.num_seqs = p.num_seqs;
    sp.p.num_heads = p.num_heads;
    sp.p.group = p.group;
    sp.p.block_tables = p.block_tables;
    sp.p.max_blocks_per_seq = p.max_blocks_per_seq;
    sp.p.qk_scale_log2 = p.qk_scale_log2;
    sp.p.dev_err = p.dev_err;
    sp.scales = scales;
    PrefixParams px{};
    px.grp_begin = p.grp_begin;
    px.grp_prefix_blocks = p.grp_prefix_blocks;
    px.num_groups = p.num_groups;
    px.max_group_size = p.max_group_size;
    px.max_prefix_blocks = p.max_prefix_blocks;
    px.run = p.prefix_partition;
    px.first_row = first_row;
    px.ws_m = p.ws_m;
    px.ws_l = p.ws_l;
    px.ws_o = p.ws_o;
    const int64_t runs = ((int64_t)p.max_prefix_blocks * p.block_size + px.run - 1) / px.run;
    const int64_t ctas = runs * ctas_of_run(p.num_groups, p.num_kv_heads, p.group, p.max_group_size);
    if (ctas > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)ctas, pfs::kThreads, L::alloc, stream>>>(sp, px);
    return cudaGetLastError();
}

template <int QT, int D, int BS, int NNT>
cudaError_t run(const DecodeParams& p0, const float* scales, int32_t* first, int sms, cudaStream_t stream)
{
    DecodeParams p = p0;
    const int64_t ctas = decode_scaled_ctas(8 * NNT, sms);
    const int64_t rows = (int64_t)p.num_seqs * p.num_heads;
    if (many_rows(p.num_groups, p.num_kv_heads, p.group, p.max_group_size)) {
        const int64_t n = most_runs(p.num_groups, p.num_kv_heads, p.group, p.max_group_size, sms);
        const int64_t tiles = ((int64_t)p.max_prefix_blocks * BS + kKeys - 1) / kKeys;
        const int64_t run = (tiles + n - 1) / n * kKeys;
        p.prefix_partition = (int32_t)(run < kMinRun ? kMinRun : run);
        cudaError_t e = run_prefixes<QT, D, BS>(p, scales, 2 * ctas * 8 * NNT + rows, stream);
        if (e != cudaSuccess)
            return e;
    }
    DecodeExtra x{};
    x.first = first;
    auto kern = decode_scaled_kernel<QT, D, BS, NNT, true, kShared>;
    static std::atomic<bool> configured[64];      // (threads may call at once)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)shared_entries_bytes(kSharedEntries, 1));
        if (e != cudaSuccess)
            return e;
        configured[dev] = true;
    }
    e = launch_early_smem(kern, ctas, kWarps * 32, shared_entries_bytes(p.num_groups, p.num_seqs), stream, p,
                          reinterpret_cast<const float2*>(scales), x);
    if (e != cudaSuccess)
        return e;
    return launch_early(reduce_shares_kernel<QT, D, kShared>, (rows + kReduceRows - 1) / kReduceRows,
                        kReduceRows * 32, stream, p, ctas, 8 * NNT, x);
}

template <int QT, int D, int BS>
cudaError_t by_rows(const DecodeParams& p, const float* scales, int32_t* first, int sms, cudaStream_t st)
{
    return rows_of(p.num_groups, p.num_kv_heads, p.group, p.max_group_size) == 8
               ? run<QT, D, BS, 1>(p, scales, first, sms, st)
               : run<QT, D, BS, 2>(p, scales, first, sms, st);
}

template <int QT, int D>
cudaError_t by_block(const DecodeParams& p, const float* scales, int32_t* first, int sms, cudaStream_t st)
{
    switch (p.block_size) {
    case 8: return by_rows<QT, D, 8>(p, scales, first, sms, st);
    case 16: return by_rows<QT, D, 16>(p, scales, first, sms, st);
    case 32: return by_rows<QT, D, 32>(p, scales, first, sms, st);
    default: return cudaErrorNotSupported;
    }
}

template <int QT>
cudaError_t by_dim(const DecodeParams& p, const float* scales, int32_t* first, int sms, cudaStream_t st)
{
    return p.head_dim == 128 ? by_block<QT, 128>(p, scales, first, sms, st)
                             : by_block<QT, 64>(p, scales, first, sms, st);
}

}  // namespace

cudaError_t launch_decode_scaled_prefix(const DecodeParams& p, const float* scales, int32_t* first, int sms,
                                        cudaStream_t stream)
{
    if (p.num_seqs <= 0)
        return cudaSuccess;
    if (p.group < 1 || p.group > kMaxGroup || p.num_groups < 1 ||
        (int64_t)p.num_groups + p.num_seqs > kSharedEntries)
        return cudaErrorNotSupported;
    return p.q_dtype == kF16 ? by_dim<kF16>(p, scales, first, sms, stream)
                             : by_dim<kBF16>(p, scales, first, sms, stream);
}

// Two pieces a CTA, the rows of sequences whose own tokens one CTA held, those of the
// prefixes: of what one CTA held, or of every run.
int64_t decode_prefix_rows(int32_t num_seqs, int32_t num_heads, int32_t group, int32_t num_groups,
                           int32_t max_group_size, int sms)
{
    const int rt = rows_of(num_groups, num_heads / group, group, max_group_size);
    const int64_t runs = many_rows(num_groups, num_heads / group, group, max_group_size)
                             ? most_runs(num_groups, num_heads / group, group, max_group_size, sms)
                             : 1;
    return 2 * decode_scaled_ctas(rt, sms) * rt + (1 + runs) * (int64_t)num_seqs * num_heads;
}

}  // namespace pkv
