// scaled_internal.h -- launch interface of the kernels for the 8-bit cache with
// a scale per block and KV head, between scaled_api.cu and the kernel files.
// Not installed; not part of the C ABI.
#pragma once

#include "pkv_internal.h"

namespace pkv {

struct RopeParams {
    void* k_cache;
    void* v_cache;
    float* scales;                 // [num_blocks][num_kv_heads][2], or null
    int64_t num_blocks;
    int32_t num_kv_heads;
    int32_t block_size;
    int32_t head_dim;
    int32_t cache_dtype;
    float k_inv_scale;             // E4M3 cache without `scales`
    float v_inv_scale;
    const void* q;                 // null: no q
    const void* k;
    const void* v;
    int64_t q_stride;              // elements between tokens
    int64_t k_stride;
    int64_t v_stride;
    int32_t in_dtype;
    int32_t num_heads;
    const double* inv_freq;        // [rot_dim / 2], radians per position
    int32_t rot_dim;
    int32_t interleaved;
    float mscale;
    uint64_t per_radian;           // 2^65 / pi: 2^66ths of a turn in a radian
    float k_bound;                 // |rotated K| <= k_bound * max |K|
    int32_t num_seqs;
    const int32_t* cu_seqlens_q;
    int32_t total_q;
    int32_t max_q_len;
    const int32_t* block_tables;
    int32_t max_blocks_per_seq;
    const int32_t* context_lens;
    int32_t max_context_len;
    const int32_t* position_offsets;   // [num_seqs], or null: position - place in the context
    int32_t* dev_err;
    void* q_out;                   // [total_q][num_heads][head_dim]
};

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t stream);

// Decode over a scaled cache: `p` with k_scale = v_scale = 1; partition_size 0:
// equal shares, whose partials take decode_scaled_partial_rows rows of ws_m,
// ws_l and ws_o, and which launches its own reduce.
cudaError_t launch_decode_scaled(const DecodeParams& p, const float* scales, int sms,
                                 cudaStream_t stream);
int64_t decode_scaled_ctas(int32_t group, int sms);
int64_t decode_scaled_partial_rows(int32_t group, int sms);
// The library's choice: tokens per partition, or 0 for equal shares.
int32_t decode_scaled_partition(const DecodeParams& p);

// What the decode that adds its weights has beside DecodeParams (scratch in
// `scores`, `whole`): weights[s][h][t] += the softmax weight of token t, summed
// over the query heads of KV head h.
struct DecodeExtra {
    float* scores;                 // [num_seqs][num_kv_heads][score_tokens][pitch], log2
    int64_t score_tokens;
    int32_t pitch;                 // query heads of a KV head, to the next power of two
    float* weights;
    int64_t weights_seq;           // elements between sequences, KV heads
    int64_t weights_head;
    float2* whole;                 // [num_seqs][num_heads]: (maximum, 1 / sum) of items one CTA held
    int32_t* first;                // shared prefixes: units before each group and sequence
};

constexpr int kWeightsSeqs = 1024;     // sequences a launch takes

// partition_size > 0: contexts of at most that many tokens, one launch; 0: equal
// shares (at most kWeightsSeqs sequences).
cudaError_t launch_decode_weights(const DecodeParams& p, const float* scales, const DecodeExtra& x,
                                  int sms, cudaStream_t stream);

// Shared prefixes (p.grp_*): ws_m, ws_l, ws_o of decode_prefix_rows rows, `first` of
// one more entry than groups and sequences.
constexpr int kSharedEntries = 2048;   // groups and sequences a launch takes
cudaError_t launch_decode_scaled_prefix(const DecodeParams& p, const float* scales, int32_t* first, int sms,
                                        cudaStream_t stream);
int64_t decode_prefix_rows(int32_t num_seqs, int32_t num_heads, int32_t group, int32_t num_groups,
                           int32_t max_group_size, int sms);

struct ScaledPrefillParams {
    PrefillParams p;               // dtype = that of q and out
    const float* scales;
};

// The prefixes that groups of sequences share, as launch_prefill_scaled's kernel
// takes them: partials of the rows of q over runs of `run` keys, the rows of run i
// from first_row + i num_seqs num_heads on.
struct PrefixParams {
    const int32_t* grp_begin;
    const int32_t* grp_prefix_blocks;
    int32_t num_groups;
    int32_t max_group_size;
    int32_t max_prefix_blocks;
    int32_t run;                   // a multiple of 128
    int64_t first_row;
    float* ws_m;
    float* ws_l;
    float* ws_o;
};

cudaError_t launch_prefill_scaled(const ScaledPrefillParams& p, cudaStream_t stream);

struct ScaledCopyParams {
    const void* src_k[kCopyMaxLayers];
    const void* src_v[kCopyMaxLayers];
    const float* src_s[kCopyMaxLayers];
    void* dst_k[kCopyMaxLayers];
    void* dst_v[kCopyMaxLayers];
    float* dst_s[kCopyMaxLayers];
    int32_t num_layers;
    int32_t num_kv_heads;
    int64_t src_blocks;
    int64_t dst_blocks;
    int64_t block_bytes;
    const int64_t* pairs;
    int64_t num_pairs;
    int32_t* dev_err;
};

cudaError_t launch_copy_scaled(const ScaledCopyParams& p, cudaStream_t stream);

}  // namespace pkv
