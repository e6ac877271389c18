// context_internal.h -- launch interface of the kernels that weigh and evict cached
// tokens, between context_api.cu and the kernel files.  Not installed; not part of
// the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

constexpr int kWindowSeqs = 512;       // sequences a launch of attention weights takes
constexpr int64_t kWindowRows = 1 << 30;   // (row, query head) rows of a KV head that its 32 bits hold

struct WeightsParams {
    const void* k_cache;
    const float* scales;           // [num_blocks][num_kv_heads][2], or null
    int64_t num_blocks;
    int32_t num_kv_heads;
    int32_t block_size;
    int32_t head_dim;
    int32_t cache_dtype;
    const void* q;                 // [total_q][num_heads][head_dim]
    int32_t q_dtype;
    int32_t num_seqs;
    int32_t num_heads;
    int32_t group;
    const int32_t* cu_seqlens_q;
    int32_t total_q;
    int32_t window;                // last rows of a sequence that count
    const int32_t* block_tables;
    int32_t max_blocks_per_seq;
    const int32_t* context_lens;
    int32_t max_context_len;
    float qk_scale_log2;           // scale * log2(e), times the cache's one scale
    int32_t row_tiles;             // q tiles of 128 rows of a KV head: ceil(window * group / 128)
    int32_t ctas;                  // of a pass: one an SM
    void* q_tiles;                 // [num_seqs][num_kv_heads][row_tiles] operand tiles
    float* row_info;               // [num_seqs][num_kv_heads][row_tiles][260]: factors, -log sums, a flag
    float* partials;               // [2 ctas][row_tiles * 128]: log sums
    int32_t* finished;             // [num_seqs][num_kv_heads]: segments done
    int32_t* failed;               // a wait of the pass for the sums ran out
    float* weights;                // element (s, h, t) at s weights_seq + h weights_head + t
    int64_t weights_seq;
    int64_t weights_head;
    int32_t* dev_err;
    uint32_t wait_tries;           // polls of a wait for the sums; 0: the kernel's own limit
};

cudaError_t launch_attention_weights(const WeightsParams& p, cudaStream_t stream);

struct EvictParams {
    void* k_cache;
    void* v_cache;
    float* scales;                 // [num_blocks][num_kv_heads][2], or null
    int64_t num_blocks;
    int32_t num_kv_heads;
    int32_t block_size;
    int32_t row_bytes;             // head_dim elements
    int32_t num_seqs;
    const int32_t* block_tables;
    int32_t max_blocks_per_seq;
    const int32_t* context_lens;
    int32_t max_context_len;
    const float* weights;
    int64_t weights_seq;
    int64_t weights_head;
    const int32_t* keep_lens;
    int32_t max_keep_len;
    int32_t most;                  // min(max_keep_len, max_context_len): bound of what stays
    int32_t keep_first;
    int32_t keep_last;
    const int32_t* dst_tables;
    int32_t max_dst_blocks;
    float* weights_out;
    int64_t weights_out_seq;
    int64_t weights_out_head;
    int32_t weights_out_len;       // entries of a row that are written
    int32_t* lens_out;
    int32_t* kept;                 // [num_seqs][num_kv_heads][most]: kept tokens in order
    int32_t* dev_err;
};

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace pkv
