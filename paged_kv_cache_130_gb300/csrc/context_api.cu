// context_api.cu -- the C ABI of the calls that share and shrink long contexts:
// shared-prefix decode over the scaled cache, attention weights, the decode that
// adds its weights, eviction.  Argument checks and launch choice.
//
// As in pkv_api.cu every entry point checks what the host can see and returns
// before launching anything when a check fails; nothing here allocates, frees
// or synchronises.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "api_common.h"
#include "context_internal.h"
#include "pkv.h"
#include "scaled_internal.h"

namespace {

using namespace pkv::api;

constexpr float kLog2E = 1.4426950408889634f;

bool sizes_known(const pkv_cache_desc* c, int32_t num_seqs, int32_t num_heads, int32_t max_context_len)
{
    return c != nullptr && c->num_kv_heads > 0 && c->block_size > 0 && c->head_dim > 0 &&
           num_seqs > 0 && num_heads >= c->num_kv_heads && max_context_len > 0 &&
           max_context_len <= INT_MAX - 1024;
}

// n runs of m rows each of at least `len` entries, the runs `outer` apart and their rows
// `inner`, do not overlap.
bool rows_apart(int64_t outer, int64_t n, int64_t inner, int64_t m, int64_t len)
{
    return (m <= 1 || inner >= len) && (n <= 1 || (outer >= len && (m <= 1 || inner <= (outer - len) / (m - 1))));
}

// Rows of at least `len` entries that do not overlap, sequence by sequence or head by
// head (null where there are none).
bool weights_ok(const float* w, int64_t seq, int64_t head, int32_t num_seqs, int32_t heads, int64_t len)
{
    return (w != nullptr || len == 0) && aligned(w, 4) &&
           (rows_apart(seq, num_seqs, head, heads, len) || rows_apart(head, heads, seq, num_seqs, len));
}

// Two arrays of n entries that have none in common.
bool apart(const int32_t* a, const int32_t* b, int32_t n)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return (x < y ? y - x : x - y) >= sizeof(int32_t) * (uintptr_t)n;
}

pkv::DecodeParams decode_params(const pkv_cache_desc* cache, const void* q, int32_t q_dtype,
                                int32_t num_seqs, int32_t num_heads, const int32_t* block_tables,
                                int32_t max_blocks_per_seq, const int32_t* context_lens,
                                int32_t max_context_len, float scale, int32_t* dev_err, void* out)
{
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
    p.max_partitions = 1;
    p.grid_partitions = 1;
    p.qk_scale_log2 = scale * kLog2E;
    p.dev_err = dev_err;
    p.out = out;
    return p;
}

// Scratch of m, l and o partials: `rows` rows, and `more` bytes.
struct Partials {
    int64_t l_off, o_off, more_off, bytes;
};

Partials partials(int64_t rows, int32_t head_dim, int64_t more = 0)
{
    Partials w{};
    w.l_off = round_up(4 * rows, 256);
    w.o_off = 2 * w.l_off;
    w.more_off = w.o_off + round_up(4 * rows * head_dim, 256);
    w.bytes = w.more_off + more;
    return w;
}

void place(pkv::DecodeParams& p, const Partials& w, char* ws)
{
    p.ws_m = reinterpret_cast<float*>(ws);
    p.ws_l = reinterpret_cast<float*>(ws + w.l_off);
    p.ws_o = reinterpret_cast<float*>(ws + w.o_off);
}

// (behind them: units before each group and sequence)
Partials shared_layout(const pkv_cache_desc* c, int32_t num_seqs, int32_t num_heads, int32_t num_groups,
                       int32_t max_group_size)
{
    const int32_t members = max_group_size < num_seqs ? max_group_size : num_seqs;
    return partials(pkv::decode_prefix_rows(num_seqs, num_heads, num_heads / c->num_kv_heads, num_groups,
                                            members, device_sms()),
                    c->head_dim, round_up(4 * ((int64_t)num_groups + num_seqs + 1), 256));
}

// The decode that adds its weights: contexts up to kOnePass tokens are one CTA's
// work, longer ones equal shares; launches of up to kWeightsSeqs sequences, which
// share the scratch.
struct WeightsLayout {
    int32_t partition;
    int32_t seqs;              // of one launch
    int32_t pitch;
    Partials part;
    int64_t whole_off, scores_off, bytes;
};

WeightsLayout weights_layout(const pkv_cache_desc* c, int32_t num_seqs, int32_t num_heads,
                             int32_t max_context_len)
{
    WeightsLayout w{};
    const int32_t group = num_heads / c->num_kv_heads;
    w.seqs = num_seqs < pkv::kWeightsSeqs ? num_seqs : pkv::kWeightsSeqs;
    w.pitch = 1;
    while (w.pitch < group)
        w.pitch *= 2;
    pkv::DecodeParams p{};
    p.num_kv_heads = c->num_kv_heads;
    p.block_size = c->block_size;
    p.head_dim = c->head_dim;
    p.num_seqs = w.seqs;
    p.num_heads = num_heads;
    p.max_context_len = max_context_len;
    w.partition = pkv::decode_scaled_partition(p);
    if (w.partition == 0)
        w.part = partials(pkv::decode_scaled_partial_rows(group, device_sms()), c->head_dim);
    w.whole_off = w.part.bytes;
    w.scores_off = w.whole_off + round_up(8 * (int64_t)w.seqs * num_heads, 256);
    w.bytes = w.scores_off +
              round_up(4 * (int64_t)w.seqs * c->num_kv_heads * max_context_len * w.pitch, 256);
    return w;
}

// (row, query head) rows of a KV head: a sequence has no more rows than its context.
int64_t window_rows(const pkv_cache_desc* c, int32_t num_heads, int32_t window, int32_t max_context_len)
{
    return (int64_t)(window < max_context_len ? window : max_context_len) * (num_heads / c->num_kv_heads);
}

// The weights of a window: launches of up to kWindowSeqs sequences, which share the
// scratch.
struct WindowLayout {
    int32_t seqs;              // of one launch
    int32_t row_tiles, ctas;
    int64_t info_off, partials_off, finished_off, failed_off, bytes;
};

WindowLayout window_layout(const pkv_cache_desc* c, int32_t num_seqs, int32_t num_heads, int32_t window,
                           int32_t max_context_len)
{
    WindowLayout w{};
    w.seqs = num_seqs < pkv::kWindowSeqs ? num_seqs : pkv::kWindowSeqs;
    w.row_tiles = (int32_t)((window_rows(c, num_heads, window, max_context_len) + 127) / 128);
    w.ctas = device_sms();
    const int64_t tiles = (int64_t)w.seqs * c->num_kv_heads * w.row_tiles;
    w.info_off = tiles * 128 * c->head_dim * 2;
    w.partials_off = round_up(w.info_off + tiles * 260 * 4, 256);
    w.finished_off = w.partials_off + 2 * (int64_t)w.ctas * w.row_tiles * 128 * 4;
    w.failed_off = w.finished_off + 4 * (int64_t)w.seqs * c->num_kv_heads;
    w.bytes = round_up(w.failed_off + 4, 256);
    return w;
}

}  // namespace

extern "C" {

size_t pkv_decode_scaled_shared_prefix_workspace_bytes(const pkv_cache_desc* cache, int32_t num_seqs,
                                                       int32_t num_heads, int32_t num_groups,
                                                       int32_t max_group_size, int32_t max_context_len)
{
    if (!sizes_known(cache, num_seqs, num_heads, max_context_len) || num_groups < 0 || max_group_size < 0)
        return 0;
    const size_t plain = pkv_decode_scaled_workspace_bytes(cache, num_seqs, num_heads, max_context_len, 0);
    if (num_groups == 0 || max_group_size == 0 || num_heads / cache->num_kv_heads > 16)
        return plain;
    const size_t shared = (size_t)shared_layout(cache, num_seqs, num_heads, num_groups, max_group_size).bytes;
    return plain > shared ? plain : shared;
}

pkv_status pkv_paged_attention_decode_scaled_shared_prefix(
    const pkv_cache_desc* cache, const float* scales, const void* q, int32_t q_dtype, int32_t num_seqs,
    int32_t num_heads, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, int32_t max_context_len, int32_t num_groups,
    const int32_t* group_begin, const int32_t* group_prefix_blocks, int32_t max_group_size,
    int32_t max_prefix_blocks, float scale, void* workspace, size_t workspace_bytes, int32_t* dev_err,
    void* out, pkv_stream_t stream)
{
    pkv_status st = check_cache(cache, true);
    if (st != PKV_OK)
        return st;
    if (num_groups < 0 || max_group_size < 0 || max_prefix_blocks < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_groups == 0 || max_prefix_blocks == 0 || num_seqs == 0)
        return pkv_paged_attention_decode_scaled(cache, scales, q, q_dtype, num_seqs, num_heads,
                                                 block_tables, max_blocks_per_seq, context_lens,
                                                 max_context_len, scale, 0, workspace, workspace_bytes,
                                                 dev_err, out, stream);
    if (!is16(q_dtype) || num_seqs < 0 || num_heads <= 0 || num_heads % cache->num_kv_heads != 0 ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size) || !(fabsf(scale) < INFINITY))
        return PKV_ERR_INVALID_ARG;
    if (max_group_size == 0 || max_prefix_blocks > max_blocks_per_seq ||
        (int64_t)max_prefix_blocks * cache->block_size > max_context_len)
        return PKV_ERR_INVALID_ARG;
    if (num_heads / cache->num_kv_heads > 16 || (int64_t)num_groups + num_seqs > pkv::kSharedEntries)
        return PKV_ERR_UNSUPPORTED;
    if (scales == nullptr || !aligned(scales, 8) || q == nullptr || out == nullptr ||
        context_lens == nullptr || block_tables == nullptr || group_begin == nullptr ||
        group_prefix_blocks == nullptr || !aligned(q, 16) || !aligned(out, 16))
        return PKV_ERR_INVALID_ARG;
    const Partials wl = shared_layout(cache, num_seqs, num_heads, num_groups, max_group_size);
    if (workspace == nullptr || !aligned(workspace, 256) || (int64_t)workspace_bytes < wl.bytes)
        return PKV_ERR_WORKSPACE;
    pkv::DecodeParams p =
        decode_params(cache, q, q_dtype, num_seqs, num_heads, block_tables, max_blocks_per_seq,
                      context_lens, max_context_len, scale, dev_err, out);
    place(p, wl, reinterpret_cast<char*>(workspace));
    p.grp_begin = group_begin;
    p.grp_prefix_blocks = group_prefix_blocks;
    p.num_groups = num_groups;
    p.max_group_size = max_group_size < num_seqs ? max_group_size : num_seqs;
    p.max_prefix_blocks = max_prefix_blocks;
    int32_t* first = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(workspace) + wl.more_off);
    return from_cuda(pkv::launch_decode_scaled_prefix(p, scales, first, device_sms(),
                                                      reinterpret_cast<cudaStream_t>(stream)));
}

size_t pkv_attention_weights_workspace_bytes(const pkv_cache_desc* cache, int32_t num_seqs,
                                             int32_t num_heads, int32_t window, int32_t max_context_len)
{
    if (!sizes_known(cache, num_seqs, num_heads, max_context_len) || window <= 0 ||
        window_rows(cache, num_heads, window, max_context_len) > pkv::kWindowRows)
        return 0;
    return (size_t)window_layout(cache, num_seqs, num_heads, window, max_context_len).bytes;
}

pkv_status pkv_attention_weights(const pkv_cache_desc* cache, const float* scales, const void* q,
                                 int32_t q_dtype, int32_t num_seqs, int32_t num_heads,
                                 const int32_t* cu_seqlens_q, int32_t total_q, int32_t window,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* context_lens, int32_t max_context_len, float scale,
                                 float* weights, int64_t weights_seq, int64_t weights_head,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                 pkv_stream_t stream)
{
    const bool scaled = scales != nullptr;
    pkv_status st = check_cache(cache, scaled);
    if (st != PKV_OK)
        return st;
    if (!is16(q_dtype) || num_seqs < 0 || num_heads <= 0 || num_heads % cache->num_kv_heads != 0 ||
        total_q < 0 || window < 0 || !(fabsf(scale) < INFINITY) ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size))
        return PKV_ERR_INVALID_ARG;
    if (num_heads / cache->num_kv_heads > 128 ||
        window_rows(cache, num_heads, window, max_context_len) > pkv::kWindowRows ||
        (cache->cache_dtype != PKV_FP8_E4M3 && cache->cache_dtype != q_dtype))
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || window == 0 || max_context_len == 0)
        return PKV_OK;
    if (q == nullptr || !aligned(q, 16) || !aligned(scales, 8) || cu_seqlens_q == nullptr ||
        context_lens == nullptr || block_tables == nullptr || max_blocks_per_seq == 0 ||
        !weights_ok(weights, weights_seq, weights_head, num_seqs, cache->num_kv_heads, max_context_len))
        return PKV_ERR_INVALID_ARG;
    const WindowLayout wl = window_layout(cache, num_seqs, num_heads, window, max_context_len);
    if (workspace == nullptr || !aligned(workspace, 256) || (int64_t)workspace_bytes < wl.bytes)
        return PKV_ERR_WORKSPACE;
    char* ws = reinterpret_cast<char*>(workspace);
    pkv::WeightsParams p{};
    p.k_cache = cache->k_cache;
    p.scales = scales;
    p.num_blocks = cache->num_blocks;
    p.num_kv_heads = cache->num_kv_heads;
    p.block_size = cache->block_size;
    p.head_dim = cache->head_dim;
    p.cache_dtype = cache->cache_dtype;
    p.q = q;
    p.q_dtype = q_dtype;
    p.num_heads = num_heads;
    p.group = num_heads / cache->num_kv_heads;
    p.total_q = total_q;
    p.window = window < max_context_len ? window : max_context_len;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    const bool one_scale = cache->cache_dtype == PKV_FP8_E4M3 && !scaled;
    p.qk_scale_log2 = scale * kLog2E * (one_scale ? cache->k_scale : 1.f);
    if (!(fabsf(p.qk_scale_log2) < INFINITY))
        return PKV_ERR_INVALID_ARG;
    p.row_tiles = wl.row_tiles;
    p.ctas = wl.ctas;
    p.q_tiles = ws;
    p.row_info = reinterpret_cast<float*>(ws + wl.info_off);
    p.partials = reinterpret_cast<float*>(ws + wl.partials_off);
    p.finished = reinterpret_cast<int32_t*>(ws + wl.finished_off);
    p.failed = reinterpret_cast<int32_t*>(ws + wl.failed_off);
    p.weights_seq = weights_seq;
    p.weights_head = weights_head;
    p.dev_err = dev_err;
    p.wait_tries = pkv::decode_wait_tries();
    for (int32_t s0 = 0; s0 < num_seqs; s0 += wl.seqs) {
        p.num_seqs = num_seqs - s0 < wl.seqs ? num_seqs - s0 : wl.seqs;
        p.cu_seqlens_q = cu_seqlens_q + s0;
        p.block_tables = block_tables + (int64_t)s0 * max_blocks_per_seq;
        p.context_lens = context_lens + s0;
        p.weights = weights + s0 * weights_seq;
        st = from_cuda(pkv::launch_attention_weights(p, reinterpret_cast<cudaStream_t>(stream)));
        if (st != PKV_OK)
            return st;
    }
    return PKV_OK;
}

size_t pkv_decode_scaled_weights_workspace_bytes(const pkv_cache_desc* cache, int32_t num_seqs,
                                                 int32_t num_heads, int32_t max_context_len)
{
    if (!sizes_known(cache, num_seqs, num_heads, max_context_len))
        return 0;
    return (size_t)weights_layout(cache, num_seqs, num_heads, max_context_len).bytes;
}

pkv_status pkv_paged_attention_decode_scaled_weights(
    const pkv_cache_desc* cache, const float* scales, const void* q, int32_t q_dtype, int32_t num_seqs,
    int32_t num_heads, const int32_t* block_tables, int32_t max_blocks_per_seq,
    const int32_t* context_lens, int32_t max_context_len, float scale, float* weights,
    int64_t weights_seq, int64_t weights_head, void* workspace, size_t workspace_bytes,
    int32_t* dev_err, void* out, pkv_stream_t stream)
{
    pkv_status st = check_cache(cache, true);
    if (st != PKV_OK)
        return st;
    if (!is16(q_dtype) || num_seqs < 0 || num_heads <= 0 || num_heads % cache->num_kv_heads != 0 ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size) || !(fabsf(scale) < INFINITY))
        return PKV_ERR_INVALID_ARG;
    if (num_heads / cache->num_kv_heads > 16)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0)
        return PKV_OK;
    if (max_context_len == 0)                          // zeros, and no weights
        return pkv_paged_attention_decode_scaled(cache, scales, q, q_dtype, num_seqs, num_heads,
                                                 block_tables, max_blocks_per_seq, context_lens, 0, scale, 0,
                                                 nullptr, 0, dev_err, out, stream);
    if (scales == nullptr || !aligned(scales, 8) || q == nullptr || out == nullptr ||
        context_lens == nullptr || block_tables == nullptr || max_blocks_per_seq == 0 || !aligned(q, 16) ||
        !aligned(out, 16) ||
        !weights_ok(weights, weights_seq, weights_head, num_seqs, cache->num_kv_heads, max_context_len))
        return PKV_ERR_INVALID_ARG;
    const WeightsLayout wl = weights_layout(cache, num_seqs, num_heads, max_context_len);
    if (workspace == nullptr || !aligned(workspace, 256) || (int64_t)workspace_bytes < wl.bytes)
        return PKV_ERR_WORKSPACE;
    char* ws = reinterpret_cast<char*>(workspace);
    for (int32_t s0 = 0; s0 < num_seqs; s0 += wl.seqs) {
        const int64_t row = (int64_t)s0 * num_heads * cache->head_dim;
        pkv::DecodeParams p = decode_params(
            cache, reinterpret_cast<const uint16_t*>(q) + row, q_dtype,
            num_seqs - s0 < wl.seqs ? num_seqs - s0 : wl.seqs, num_heads,
            block_tables + (int64_t)s0 * max_blocks_per_seq, max_blocks_per_seq, context_lens + s0,
            max_context_len, scale, dev_err, reinterpret_cast<uint16_t*>(out) + row);
        p.partition_size = wl.partition;
        if (wl.partition == 0)
            place(p, wl.part, ws);
        pkv::DecodeExtra x{};
        x.scores = reinterpret_cast<float*>(ws + wl.scores_off);
        x.score_tokens = max_context_len;
        x.pitch = wl.pitch;
        x.weights = weights + s0 * weights_seq;
        x.weights_seq = weights_seq;
        x.weights_head = weights_head;
        x.whole = reinterpret_cast<float2*>(ws + wl.whole_off);
        st = from_cuda(pkv::launch_decode_weights(p, scales, x, device_sms(),
                                                  reinterpret_cast<cudaStream_t>(stream)));
        if (st != PKV_OK)
            return st;
    }
    return PKV_OK;
}

size_t pkv_evict_workspace_bytes(const pkv_cache_desc* cache, int32_t num_seqs, int32_t max_keep_len,
                                 int32_t max_context_len)
{
    if (!sizes_known(cache, num_seqs, cache != nullptr ? cache->num_kv_heads : 0, max_context_len) ||
        max_keep_len <= 0)
        return 0;
    const int32_t most = max_keep_len < max_context_len ? max_keep_len : max_context_len;
    return (size_t)round_up(4 * (int64_t)num_seqs * cache->num_kv_heads * most, 256);
}

pkv_status pkv_evict(const pkv_cache_desc* cache, float* scales, int32_t num_seqs,
                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                     const int32_t* context_lens, int32_t max_context_len, const float* weights,
                     int64_t weights_seq, int64_t weights_head, const int32_t* keep_lens,
                     int32_t max_keep_len, int32_t keep_first, int32_t keep_last,
                     const int32_t* dst_tables, int32_t max_dst_blocks, float* weights_out,
                     int64_t weights_out_seq, int64_t weights_out_head, int32_t weights_out_len,
                     int32_t* lens_out, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                     pkv_stream_t stream)
{
    const bool scaled = scales != nullptr;
    pkv_status st = check_cache(cache, scaled);
    if (st != PKV_OK)
        return st;
    if (num_seqs < 0 || max_keep_len < 0 || max_keep_len > INT_MAX - 1024 || keep_first < 0 ||
        keep_last < 0 || weights_out_len < 0 || max_dst_blocks < 0 ||
        !lengths_ok(max_blocks_per_seq, max_context_len, cache->block_size))
        return PKV_ERR_INVALID_ARG;
    // (a context keeps no more than it has)
    const int32_t most = max_keep_len < max_context_len ? max_keep_len : max_context_len;
    if (((int64_t)most + cache->block_size - 1) / cache->block_size > max_dst_blocks ||
        weights_out_len < most)
        return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0)
        return PKV_OK;
    if (context_lens == nullptr || keep_lens == nullptr || lens_out == nullptr || !aligned(scales, 8) ||
        (max_context_len > 0 && (block_tables == nullptr || max_blocks_per_seq == 0)) ||
        (most > 0 && dst_tables == nullptr) ||
        !weights_ok(weights, weights_seq, weights_head, num_seqs, cache->num_kv_heads, max_context_len) ||
        !weights_ok(weights_out, weights_out_seq, weights_out_head, num_seqs, cache->num_kv_heads,
                    weights_out_len) ||
        (weights == weights_out && weights != nullptr) || !apart(lens_out, context_lens, num_seqs) ||
        !apart(lens_out, keep_lens, num_seqs))
        return PKV_ERR_INVALID_ARG;
    const int64_t need = 4 * (int64_t)num_seqs * cache->num_kv_heads * most;
    if (need > 0 && (workspace == nullptr || !aligned(workspace, 256) || (int64_t)workspace_bytes < need))
        return PKV_ERR_WORKSPACE;
    pkv::EvictParams p{};
    p.k_cache = cache->k_cache;
    p.v_cache = cache->v_cache;
    p.scales = scales;
    p.num_blocks = cache->num_blocks;
    p.num_kv_heads = cache->num_kv_heads;
    p.block_size = cache->block_size;
    p.row_bytes = cache->head_dim * (cache->cache_dtype == PKV_FP8_E4M3 ? 1 : 2);
    p.num_seqs = num_seqs;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.weights = weights;
    p.weights_seq = weights_seq;
    p.weights_head = weights_head;
    p.keep_lens = keep_lens;
    p.max_keep_len = max_keep_len;
    p.most = most;
    p.keep_first = keep_first;
    p.keep_last = keep_last;
    p.dst_tables = dst_tables;
    p.max_dst_blocks = max_dst_blocks;
    p.weights_out = weights_out;
    p.weights_out_seq = weights_out_seq;
    p.weights_out_head = weights_out_head;
    p.weights_out_len = weights_out_len;
    p.lens_out = lens_out;
    p.kept = reinterpret_cast<int32_t*>(workspace);
    p.dev_err = dev_err;
    return from_cuda(pkv::launch_evict(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
