// copy_scaled.cu -- copy of whole blocks with their scales, every layer.
//
// A block of a scaled cache is its codes of K and of V (one contiguous run
// each) and num_kv_heads pairs of scales; a copy that left the scales behind
// would change every value.  Copy-on-write copies inside one pool
// (「KV 缓存与分页注意力」 §08), a swap copies between a device pool and one in
// pinned host memory (§09).  Bound by the bytes moved.  Grid: x = 16-KiB chunk
// of a block, y = (layer, K|V), z = pair, as in copy_blocks.cu; the CTA of a
// (layer, pair)'s first K chunk also moves the scales, so one launch does all.
// 80 pairs x 32 layers of 64-KiB K and V blocks: 672 MB in 97 us, 6.9 TB/s.
#include <cuda_runtime.h>

#include "pkv_common.cuh"
#include "scaled_internal.h"

namespace pkv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kVec = 4;
constexpr int64_t kChunk = (int64_t)kCopyThreads * kVec * 16;   // 16 KiB

__global__ void __launch_bounds__(kCopyThreads)
    copy_scaled_kernel(const __grid_constant__ ScaledCopyParams p)
{
    const int64_t pair = blockIdx.z;
    const int layer = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const int64_t src = __ldg(p.pairs + 2 * pair);
    const int64_t dst = __ldg(p.pairs + 2 * pair + 1);
    if (src < 0 || src >= p.src_blocks || dst < 0 || dst >= p.dst_blocks) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            flag_error(p.dev_err, PKV_DEVERR_COPY_PAIR);
        return;
    }
    const char* s = reinterpret_cast<const char*>(is_v ? p.src_v[layer] : p.src_k[layer]) +
                    src * p.block_bytes;
    char* d = reinterpret_cast<char*>(is_v ? p.dst_v[layer] : p.dst_k[layer]) +
              dst * p.block_bytes;
    const int64_t start = (int64_t)blockIdx.x * kChunk;
    uint4 buf[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int64_t off = start + ((int64_t)j * kCopyThreads + threadIdx.x) * 16;
        if (off < p.block_bytes)
            buf[j] = *reinterpret_cast<const uint4*>(s + off);
    }
    if (blockIdx.x == 0 && !is_v) {
        const float2* ss = reinterpret_cast<const float2*>(p.src_s[layer]) + src * p.num_kv_heads;
        float2* ds = reinterpret_cast<float2*>(p.dst_s[layer]) + dst * p.num_kv_heads;
        for (int i = threadIdx.x; i < p.num_kv_heads; i += kCopyThreads)
            ds[i] = ss[i];
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int64_t off = start + ((int64_t)j * kCopyThreads + threadIdx.x) * 16;
        if (off < p.block_bytes)
            st_v4(d + off, buf[j]);
    }
}

}  // namespace

cudaError_t launch_copy_scaled(const ScaledCopyParams& p, cudaStream_t stream)
{
    if (p.num_pairs <= 0 || p.num_layers <= 0)
        return cudaSuccess;
    if (p.num_pairs > 65535 || p.num_layers > kCopyMaxLayers)
        return cudaErrorInvalidConfiguration;
    const int64_t chunks = (p.block_bytes + kChunk - 1) / kChunk;
    if (chunks > 0x7fffffffLL)
        return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)chunks, (unsigned)(2 * p.num_layers), (unsigned)p.num_pairs);
    copy_scaled_kernel<<<grid, kCopyThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
