// prefill_scaled.cu -- causal attention over a scaled cache: launches.
#include <cuda_runtime.h>

#include <atomic>

#include "prefill_scaled_kernel.cuh"

namespace pkv {
namespace {

using namespace pfs;

template <int QT, int D, int BS>
cudaError_t run(const ScaledPrefillParams& sp, cudaStream_t stream)
{
    using L = Layout<D>;
    const PrefillParams& p = sp.p;
    auto kern = prefill_scaled_kernel<QT, D, BS, false>;
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
    const int span = 2 * (kRows / p.group);
    const int64_t tiles = ((int64_t)p.max_q_len + span - 1) / span;
    const int64_t ctas = tiles * p.num_seqs * p.num_kv_heads;
    if (ctas > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    kern<<<(unsigned)ctas, kThreads, L::alloc, stream>>>(sp, PrefixParams{});
    return cudaGetLastError();
}

template <int QT, int D>
cudaError_t by_block(const ScaledPrefillParams& p, cudaStream_t st)
{
    switch (p.p.block_size) {
    case 8: return run<QT, D, 8>(p, st);
    case 16: return run<QT, D, 16>(p, st);
    case 32: return run<QT, D, 32>(p, st);
    default: return cudaErrorNotSupported;
    }
}

template <int QT>
cudaError_t by_dim(const ScaledPrefillParams& p, cudaStream_t st)
{
    return p.p.head_dim == 128 ? by_block<QT, 128>(p, st) : by_block<QT, 64>(p, st);
}

}  // namespace

cudaError_t launch_prefill_scaled(const ScaledPrefillParams& sp, cudaStream_t stream)
{
    if (sp.p.num_seqs <= 0 || sp.p.max_q_len <= 0)
        return cudaSuccess;
    if (sp.p.group < 1 || sp.p.group > kRows)
        return cudaErrorNotSupported;
    return sp.p.dtype == kF16 ? by_dim<kF16>(sp, stream) : by_dim<kBF16>(sp, stream);
}

}  // namespace pkv
