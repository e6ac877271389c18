// api_common.h -- checks of arguments shared by scaled_api.cu and context_api.cu.
// Not installed; not part of the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"

namespace pkv {
namespace api {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

inline bool is16(int32_t dt) { return dt == PKV_F16 || dt == PKV_BF16; }

inline pkv_status from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return PKV_OK;
    return e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
}

// A cache descriptor; with `scaled` an E4M3 cache whose k_scale / v_scale are
// not used.
inline pkv_status check_cache(const pkv_cache_desc* c, bool scaled)
{
    if (c == nullptr || c->k_cache == nullptr || c->v_cache == nullptr ||
        !aligned(c->k_cache, 16) || !aligned(c->v_cache, 16))
        return PKV_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->block_size <= 0 || c->head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (!is16(c->cache_dtype) && c->cache_dtype != PKV_FP8_E4M3)
        return PKV_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) ||
        (c->block_size != 8 && c->block_size != 16 && c->block_size != 32))
        return PKV_ERR_UNSUPPORTED;
    if (scaled)
        return c->cache_dtype == PKV_FP8_E4M3 ? PKV_OK : PKV_ERR_UNSUPPORTED;
    if (c->cache_dtype == PKV_FP8_E4M3 && (!(c->k_scale > 0.f) || !(c->v_scale > 0.f)))
        return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

// Sizes whose token arithmetic stays inside 32 bits.
inline bool lengths_ok(int32_t max_blocks_per_seq, int32_t max_context_len, int32_t block_size)
{
    return max_blocks_per_seq >= 0 && max_blocks_per_seq <= INT_MAX / block_size &&
           max_context_len >= 0 && max_context_len <= INT_MAX - 1024;
}

inline int device_sms()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 152;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v <= 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
            return 152;
        cache[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

}  // namespace api
}  // namespace pkv
