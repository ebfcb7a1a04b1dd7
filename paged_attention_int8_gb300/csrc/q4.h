// Internal launch interface of the 4-bit cache, the read-back of all formats and
// the attention over whole prompts for the C ABI (api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace paq8 {

struct KvStoreQ4 {
  const uint16_t *key, *value;
  int64_t key_stride, value_stride;
  const int64_t *slot_mapping;
  int32_t num_tokens, hk, d;
  uint8_t *k_cache, *v_cache;
  uint16_t *k_scale, *v_scale;
  int32_t num_blocks, block_size;
  uint32_t *status;
};

cudaError_t launch_kv_store_q4(const KvStoreQ4 &p, cudaStream_t stream);

enum class CacheFormat { q8, f8v4, q4 };

// a .. c: the format's arrays in the order of its store (q8 and q4: k_cache,
// k_scale, v_cache, v_scale; f8v4: k_cache, v_cache, v_scale, v_zero).
struct KvLoad {
  uint16_t *key, *value;
  int64_t key_stride, value_stride;
  const int32_t *cu_seqlens_k, *load_lens;  // load_lens: or null
  int32_t num_seqs, num_rows;
  const int32_t *block_table;
  int32_t table_stride, table_columns;
  int32_t hk, d;
  const void *array[4];
  int32_t num_blocks, block_size;
  uint32_t *status;
};

cudaError_t launch_kv_load(const KvLoad &p, CacheFormat format, cudaStream_t stream);

struct AttnQ4 {
  const uint16_t *q;
  const uint8_t *k_cache, *v_cache;
  const uint16_t *k_scale, *v_scale;
  const int32_t *cu, *seq_lens, *block_table;
  int32_t table_stride, table_columns, num_seqs, num_tokens, hq, hk, d, num_blocks, bs;
  int32_t max_query_len, max_seq_len, num_splits;
  float softmax_scale;
  const float *sinks;
  int32_t window;
  bool causal;
  uint16_t *out;
  float *lse;
  uint8_t *workspace;
};

// Query tokens that a row block takes, and the automatic number of key segments.
int32_t q4_block_tokens(int32_t qpk, int32_t max_query_len, int32_t d);
int32_t q4_auto_splits(int32_t num_seqs, int32_t num_tokens, int32_t hq, int32_t hk, int32_t d,
                       int32_t max_query_len, int32_t max_seq_len);
cudaError_t launch_attention_q4(const AttnQ4 &p, cudaStream_t stream);

}  // namespace paq8
