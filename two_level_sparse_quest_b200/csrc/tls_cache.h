// tls_cache.h -- host-side launchers of the 4-bit KV cache, the accumulated
// attention weight and the eviction (internal, not ABI).
#pragma once

#include "tls_internal.h"

namespace tls {

// 4-bit KV cache (tls_kv4.cuh: the record).  Rows of tokens [old_lens[b], new_lens[b]) in or out.
struct Kv4RowsArgs {
  const void *K, *V;  // bf16 [B*H_kv][row_stride][d]: row r is token old_lens[b] + r (read: the outputs, or null)
  const int32_t *old_lens, *new_lens;
  void *cache;
  const int32_t *label_idx;
  void *meta, *slab;  // nullable (append only)
  int *err;
  int batch, n_kv_heads, d, block_size, n_blocks_max, max_ctx, n_label, row_stride;
  int blocks_per_cta;  // set by the launch
};
cudaError_t launch_kv4_append(Kv4RowsArgs a, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4RowsArgs &a, cudaStream_t st);

struct Kv4AttnArgs {
  const void *q, *cache;
  const int32_t *token_idx;      // null: every token below seq_lens
  const int32_t *seq_lens;
  const int32_t *slot_of_block;  // null: the cache is indexed by token
  int n_slots;
  void *out;
  float *lse;
  float *part;
  int *err;
  int batch, n_q_heads, n_kv_heads, d, block_size, n_blocks_max, max_ctx, k_t, out_dtype;
  float scale_log2;
  int num_sms;
  int head_chunk, n_head_chunks, cluster, n_split;  // set by the launch (kv4_plan)
};
size_t kv4_attn_part_floats(int heads_per_group, int d, int num_sms);  // workspace floats of any call
cudaError_t launch_kv4_attention(Kv4AttnArgs a, cudaStream_t st);

// Softmax weights of a decode step added to one number per token (tls_weights.cu).
struct WeightsArgs {
  const void *q, *keys;          // keys: K rows, or 4-bit records
  const int32_t *token_idx;      // null: every token below seq_lens
  const int32_t *seq_lens;
  const float *lse;              // [B][H_q]
  float *weights;                // [B][H_kv][max_ctx]
  int batch, n_q_heads, n_kv_heads, d, max_ctx, k_t;
  int keys_kind;                 // 0 fp32, 1 bf16, 2 4-bit records
  float scale;                   // softmax scale
  int num_sms;
};
cudaError_t launch_accum_weights(const WeightsArgs &a, cudaStream_t st);

// Eviction by those numbers (tls_evict.cu).
struct EvictArgs {
  const float *weights;
  const int32_t *seq_lens;
  int32_t *keep_idx, *new_lens;
  int batch, n_kv_heads, max_ctx, budget, n_sink, n_recent, num_sms;
};
cudaError_t launch_evict_select(const EvictArgs &a, cudaStream_t st);
constexpr int kMaxEvictRows = 8;
struct CompactArgs {
  void *rows[kMaxEvictRows + 1];
  int row_bytes[kMaxEvictRows + 1];
  int n_rows;
  float *weights;  // nullable: one of rows, whose tail is zeroed
  const int32_t *keep_idx, *seq_lens;
  int batch, n_kv_heads, max_ctx, budget, num_sms;
};
cudaError_t launch_evict_compact(const CompactArgs &a, cudaStream_t st);

}  // namespace tls
