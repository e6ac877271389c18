// scaled_api.cu -- the C ABI of the calls for the 8-bit cache with a scale per
// block and KV head, and of the rotary append: argument checks, launch choice.
//
// As in pkv_api.cu every entry point checks what the host can see and returns
// before launching anything when a check fails; nothing here allocates, frees
// or synchronises.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"
#include "scaled_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

bool is16(int32_t dt) { return dt == PKV_F16 || dt == PKV_BF16; }

pkv_status from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return PKV_OK;
    return e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
}

// A cache descriptor; with `scaled` an E4M3 cache whose k_scale / v_scale are
// not used.
pkv_status check_cache(const pkv_cache_desc* c, bool scaled)
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
bool lengths_ok(int32_t max_blocks_per_seq, int32_t max_context_len, int32_t block_size)
{
    return max_blocks_per_seq >= 0 && max_blocks_per_seq <= INT_MAX / block_size &&
           max_context_len >= 0 && max_context_len <= INT_MAX - 1024;
}

int device_sms()
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

struct Layout {
    int64_t parts, l_off, o_off, bytes;
};

// The decode workspace: m, l, o partials of every (sequence, head) and
// partition as in pkv.h, or (partition 0) those of the equal shares.
Layout layout(int32_t num_seqs, int32_t num_heads, int32_t group, int32_t head_dim,
              int32_t max_context_len, int32_t partition)
{
    Layout w{};
    int64_t rows;
    if (partition == 0) {
        w.parts = 1;
        rows = pkv::decode_scaled_partial_rows(group, device_sms());
    } else {
        w.parts = ((int64_t)max_context_len + partition - 1) / partition;
        if (w.parts <= 1)
            return w;
        rows = (int64_t)num_seqs * num_heads * w.parts;
    }
    w.l_off = round_up(4 * rows, 256);
    w.o_off = 2 * w.l_off;
    w.bytes = w.o_off + round_up(4 * rows * head_dim, 256);
    return w;
}

int32_t partition_of(const pkv_cache_desc* c, int32_t num_seqs, int32_t num_heads,
                     int32_t max_context_len, int32_t requested)
{
    if (requested > 0)
        return requested;
    pkv::DecodeParams p{};
    p.num_kv_heads = c->num_kv_heads;
    p.block_size = c->block_size;
    p.head_dim = c->head_dim;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.max_context_len = max_context_len;
    return pkv::decode_scaled_partition(p);
}

bool sizes_known(const pkv_cache_desc* c, int32_t num_seqs, int32_t num_heads,
                 int32_t max_context_len, int32_t partition_size)
{
    return c != nullptr && c->num_kv_heads > 0 && c->block_size > 0 && c->head_dim > 0 &&
           num_seqs > 0 && num_heads >= c->num_kv_heads && max_context_len > 0 && partition_size >= 0 &&
           max_context_len <= INT_MAX - 1024;
}

// A pointer the GPU can dereference (device, managed or pinned host memory),
// as its device address; null otherwise.
void* device_address(const void* p)
{
    cudaPointerAttributes a{};
    if (p == nullptr || cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return a.type == cudaMemoryTypeUnregistered ? nullptr : a.devicePointer;
}

}  // namespace

extern "C" {

pkv_status pkv_rope_append(const pkv_cache_desc* cache, float* scales, const void* q,
                           int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, int32_t in_dtype, int32_t num_heads,
                           const double* inv_freq, int32_t rot_dim, int32_t interleaved,
                           float mscale, int32_t num_seqs, const int32_t* cu_seqlens_q,
                           int32_t total_q, int32_t max_q_len, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens,
                           int32_t max_context_len, int32_t* dev_err, void* q_out,
                           pkv_stream_t stream)
{
    const bool scaled = scales != nullptr;
    pkv_status st = check_cache(cache, scaled);
    if (st != PKV_OK)
        return st;
    if (!is16(in_dtype) || num_seqs < 0 || total_q < 0 || max_q_len < 0 ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size))
        return PKV_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > cache->head_dim || !(fabsf(mscale) < INFINITY))
        return PKV_ERR_INVALID_ARG;
    if (rot_dim % 16 != 0 || (cache->cache_dtype != PKV_FP8_E4M3 && cache->cache_dtype != in_dtype))
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0)
        return PKV_OK;
    const int64_t kv_row = (int64_t)cache->num_kv_heads * cache->head_dim;
    if (k == nullptr || v == nullptr || !aligned(k, 16) || !aligned(v, 16) || k_stride < kv_row ||
        v_stride < kv_row || k_stride % 8 != 0 || v_stride % 8 != 0)
        return PKV_ERR_INVALID_ARG;
    if (q != nullptr &&
        (num_heads <= 0 || q_out == nullptr || !aligned(q, 16) || !aligned(q_out, 16) ||
         q_stride < (int64_t)num_heads * cache->head_dim || q_stride % 8 != 0))
        return PKV_ERR_INVALID_ARG;
    if ((rot_dim > 0 && (inv_freq == nullptr || !aligned(inv_freq, 8))) ||
        cu_seqlens_q == nullptr || context_lens == nullptr || block_tables == nullptr ||
        max_blocks_per_seq == 0 || !aligned(scales, 8))
        return PKV_ERR_INVALID_ARG;
    pkv::RopeParams p{};
    p.k_cache = cache->k_cache;
    p.v_cache = cache->v_cache;
    p.scales = scales;
    p.num_blocks = cache->num_blocks;
    p.num_kv_heads = cache->num_kv_heads;
    p.block_size = cache->block_size;
    p.head_dim = cache->head_dim;
    p.cache_dtype = cache->cache_dtype;
    const bool one_scale = cache->cache_dtype == PKV_FP8_E4M3 && !scaled;
    p.k_inv_scale = one_scale ? 1.0f / cache->k_scale : 1.f;
    p.v_inv_scale = one_scale ? 1.0f / cache->v_scale : 1.f;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.in_dtype = in_dtype;
    p.num_heads = num_heads;
    p.inv_freq = inv_freq;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved != 0;
    p.mscale = mscale;
    static const uint64_t per_radian = (uint64_t)(ldexpl(1.0L, 65) / acosl(-1.0L));
    p.per_radian = per_radian;
    p.k_bound = 1.f;
    if (rot_dim > 0 && 1.41421356f * fabsf(mscale) > 1.f)
        p.k_bound = 1.41421356f * fabsf(mscale);
    p.num_seqs = num_seqs;
    p.cu_seqlens_q = cu_seqlens_q;
    p.total_q = total_q;
    p.max_q_len = max_q_len < total_q ? max_q_len : total_q;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.dev_err = dev_err;
    p.q_out = q_out;
    return from_cuda(
        pkv::launch_rope_append(p, device_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

int32_t pkv_decode_scaled_partition_size(const pkv_cache_desc* cache, int32_t num_seqs,
                                         int32_t num_heads, int32_t max_context_len,
                                         int32_t requested)
{
    if (!sizes_known(cache, num_seqs, num_heads, max_context_len, requested))
        return 0;
    return partition_of(cache, num_seqs, num_heads, max_context_len, requested);
}

size_t pkv_decode_scaled_workspace_bytes(const pkv_cache_desc* cache, int32_t num_seqs,
                                         int32_t num_heads, int32_t max_context_len,
                                         int32_t partition_size)
{
    if (!sizes_known(cache, num_seqs, num_heads, max_context_len, partition_size))
        return 0;
    const int32_t part =
        partition_of(cache, num_seqs, num_heads, max_context_len, partition_size);
    return (size_t)layout(num_seqs, num_heads, num_heads / cache->num_kv_heads, cache->head_dim,
                          max_context_len, part)
        .bytes;
}

pkv_status pkv_paged_attention_decode_scaled(const pkv_cache_desc* cache, const float* scales,
                                             const void* q, int32_t q_dtype, int32_t num_seqs,
                                             int32_t num_heads, const int32_t* block_tables,
                                             int32_t max_blocks_per_seq,
                                             const int32_t* context_lens, int32_t max_context_len,
                                             float scale, int32_t partition_size,
                                             void* workspace, size_t workspace_bytes,
                                             int32_t* dev_err, void* out, pkv_stream_t stream)
{
    pkv_status st = check_cache(cache, true);
    if (st != PKV_OK)
        return st;
    if (!is16(q_dtype) || num_seqs < 0 || num_heads <= 0 || num_heads % cache->num_kv_heads != 0 ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size) ||
        !(fabsf(scale) < INFINITY) || partition_size < 0 ||
        partition_size % cache->block_size != 0 || partition_size % 16 != 0)
        return PKV_ERR_INVALID_ARG;
    if (num_heads / cache->num_kv_heads > 16)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0)
        return PKV_OK;
    if (scales == nullptr || !aligned(scales, 8) || q == nullptr || out == nullptr ||
        context_lens == nullptr || !aligned(q, 16) || !aligned(out, 16) ||
        (max_context_len > 0 && (block_tables == nullptr || max_blocks_per_seq == 0)))
        return PKV_ERR_INVALID_ARG;
    const int32_t part =
        max_context_len > 0
            ? partition_of(cache, num_seqs, num_heads, max_context_len, partition_size)
            : 32;
    const Layout wl = layout(num_seqs, num_heads, num_heads / cache->num_kv_heads, cache->head_dim,
                             max_context_len, part);
    if (wl.bytes > 0 && (workspace == nullptr || !aligned(workspace, 256) ||
                         (int64_t)workspace_bytes < wl.bytes))
        return PKV_ERR_WORKSPACE;
    pkv::DecodeParams p{};
    p.k_cache = cache->k_cache;
    p.v_cache = cache->v_cache;
    p.num_blocks = cache->num_blocks;
    p.num_kv_heads = cache->num_kv_heads;
    p.block_size = cache->block_size;
    p.head_dim = cache->head_dim;
    p.cache_dtype = cache->cache_dtype;
    p.k_scale = 1.f;
    p.v_scale = 1.f;
    p.q = q;
    p.q_dtype = q_dtype;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.group = num_heads / cache->num_kv_heads;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.partition_size = part;
    p.max_partitions = wl.parts < 1 ? 1 : (int32_t)wl.parts;
    p.grid_partitions = p.max_partitions;
    p.qk_scale_log2 = scale * 1.4426950408889634f;
    char* ws = reinterpret_cast<char*>(workspace);
    if (wl.bytes > 0) {
        p.ws_m = reinterpret_cast<float*>(ws);
        p.ws_l = reinterpret_cast<float*>(ws + wl.l_off);
        p.ws_o = reinterpret_cast<float*>(ws + wl.o_off);
    }
    p.dev_err = dev_err;
    p.out = out;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    st = from_cuda(pkv::launch_decode_scaled(p, scales, device_sms(), cs));
    if (st != PKV_OK || wl.bytes == 0 || part == 0)
        return st;
    pkv::ReduceParams r{};
    r.num_seqs = num_seqs;
    r.num_heads = num_heads;
    r.head_dim = cache->head_dim;
    r.context_lens = context_lens;
    r.max_context_len = max_context_len;
    r.partition_size = part;
    r.max_partitions = (int32_t)wl.parts;
    r.ws_m = p.ws_m;
    r.ws_l = p.ws_l;
    r.ws_o = p.ws_o;
    r.out_dtype = q_dtype;
    r.out = out;
    return from_cuda(pkv::launch_lse_reduce(r, cs, true));
}

pkv_status pkv_paged_attention_prefill_scaled(
    const pkv_cache_desc* cache, const float* scales, const void* q, int32_t q_dtype,
    int32_t num_seqs, int32_t num_heads, const int32_t* cu_seqlens_q, int32_t total_q,
    int32_t max_q_len, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, int32_t max_context_len, float scale, int32_t* dev_err, void* out,
    pkv_stream_t stream)
{
    pkv_status st = check_cache(cache, true);
    if (st != PKV_OK)
        return st;
    if (!is16(q_dtype) || num_seqs < 0 || num_heads <= 0 || num_heads % cache->num_kv_heads != 0 ||
        total_q < 0 || max_q_len < 0 || !(fabsf(scale) < INFINITY) ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size))
        return PKV_ERR_INVALID_ARG;
    if (num_heads / cache->num_kv_heads > 128)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0)
        return PKV_OK;
    if (scales == nullptr || !aligned(scales, 8) || q == nullptr || out == nullptr ||
        cu_seqlens_q == nullptr || context_lens == nullptr || block_tables == nullptr ||
        max_blocks_per_seq == 0 || !aligned(q, 16) || !aligned(out, 16))
        return PKV_ERR_INVALID_ARG;
    pkv::ScaledPrefillParams sp{};
    pkv::PrefillParams& p = sp.p;
    p.k_cache = cache->k_cache;
    p.v_cache = cache->v_cache;
    p.num_blocks = cache->num_blocks;
    p.num_kv_heads = cache->num_kv_heads;
    p.block_size = cache->block_size;
    p.head_dim = cache->head_dim;
    p.dtype = q_dtype;
    p.q = q;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.group = num_heads / cache->num_kv_heads;
    p.cu_seqlens_q = cu_seqlens_q;
    p.total_q = total_q;
    p.max_q_len = max_q_len < total_q ? max_q_len : total_q;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.qk_scale_log2 = scale * 1.4426950408889634f;
    p.dev_err = dev_err;
    p.out = out;
    sp.scales = scales;
    return from_cuda(pkv::launch_prefill_scaled(sp, reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status pkv_copy_blocks_scaled(const pkv_cache_desc* src, float* const* src_scales,
                                  const pkv_cache_desc* dst, float* const* dst_scales,
                                  int32_t num_layers, const int64_t* block_pairs,
                                  int64_t num_pairs, int32_t* dev_err, pkv_stream_t stream)
{
    if (src == nullptr || src_scales == nullptr || (dst == nullptr) != (dst_scales == nullptr) ||
        num_layers <= 0 || num_pairs < 0)
        return PKV_ERR_INVALID_ARG;
    const bool between = dst != nullptr;
    const pkv_cache_desc* to = between ? dst : src;
    float* const* to_scales = between ? dst_scales : src_scales;
    const pkv_cache_desc& c0 = src[0];
    for (int32_t l = 0; l < num_layers; ++l) {
        pkv_status st = check_cache(&src[l], true);
        if (st == PKV_OK)
            st = check_cache(&to[l], true);
        if (st != PKV_OK)
            return st;
        const pkv_cache_desc& a = src[l];
        const pkv_cache_desc& b = to[l];
        if (a.num_kv_heads != c0.num_kv_heads || a.block_size != c0.block_size ||
            a.head_dim != c0.head_dim || a.num_blocks != c0.num_blocks ||
            b.num_kv_heads != c0.num_kv_heads || b.block_size != c0.block_size ||
            b.head_dim != c0.head_dim || b.num_blocks != to[0].num_blocks)
            return PKV_ERR_INVALID_ARG;
        if (src_scales[l] == nullptr || to_scales[l] == nullptr || !aligned(src_scales[l], 8) ||
            !aligned(to_scales[l], 8))
            return PKV_ERR_INVALID_ARG;
    }
    if (num_pairs == 0)
        return PKV_OK;
    if (block_pairs == nullptr)
        return PKV_ERR_INVALID_ARG;
    const int64_t* pairs = block_pairs;
    if (between) {
        // either side may be host memory: only what the GPU can reach
        pairs = reinterpret_cast<const int64_t*>(device_address(block_pairs));
        if (pairs == nullptr)
            return PKV_ERR_INVALID_ARG;
        for (int32_t l = 0; l < num_layers; ++l) {
            const void* all[6] = {src[l].k_cache, src[l].v_cache, src_scales[l],
                                  dst[l].k_cache, dst[l].v_cache, dst_scales[l]};
            for (const void* a : all)
                if (device_address(a) == nullptr)
                    return PKV_ERR_INVALID_ARG;
        }
    }
    pkv::ScaledCopyParams p{};
    p.num_kv_heads = c0.num_kv_heads;
    p.src_blocks = c0.num_blocks;
    p.dst_blocks = to[0].num_blocks;
    p.block_bytes = (int64_t)c0.num_kv_heads * c0.block_size * c0.head_dim;
    p.dev_err = dev_err;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int32_t l0 = 0; l0 < num_layers; l0 += pkv::kCopyMaxLayers) {
        p.num_layers =
            num_layers - l0 < pkv::kCopyMaxLayers ? num_layers - l0 : pkv::kCopyMaxLayers;
        for (int32_t i = 0; i < p.num_layers; ++i) {
            const int32_t l = l0 + i;
            auto at = [&](const void* a) { return between ? device_address(a) : const_cast<void*>(a); };
            p.src_k[i] = at(src[l].k_cache);
            p.src_v[i] = at(src[l].v_cache);
            p.src_s[i] = reinterpret_cast<const float*>(at(src_scales[l]));
            p.dst_k[i] = at(to[l].k_cache);
            p.dst_v[i] = at(to[l].v_cache);
            p.dst_s[i] = reinterpret_cast<float*>(at(to_scales[l]));
        }
        for (int64_t q0 = 0; q0 < num_pairs; q0 += 65535) {
            p.pairs = pairs + 2 * q0;
            p.num_pairs = num_pairs - q0 < 65535 ? num_pairs - q0 : 65535;
            const pkv_status st = from_cuda(pkv::launch_copy_scaled(p, s));
            if (st != PKV_OK)
                return st;
        }
    }
    return PKV_OK;
}

}  // extern "C"
