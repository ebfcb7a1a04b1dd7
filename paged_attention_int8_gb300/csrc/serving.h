// Internal launch interface of the shared-prefix serving calls for the C ABI
// (api.cu): block tables from request lengths (block_tables.cu), block copies
// (copy_blocks.cu) and attention over a shared prefix (attn_shared*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace paq8 {

struct BlockTables {
  const int32_t *context_lens, *query_lens;
  int32_t num_seqs;
  const int32_t *source_table;
  int32_t source_stride, num_source_rows;
  const int32_t *source_rows, *shared_lens;  // or null
  const int32_t *free_blocks;
  int32_t num_free;
  const int32_t *free_head;  // or null: 0
  int32_t num_blocks, block_size;
  int32_t *block_table;
  int32_t table_stride;
  int32_t *cu_seqlens_q, *seq_lens;
  int64_t *slot_mapping, *positions;  // positions: or null
  int32_t num_tokens;
  int32_t *copy_pairs, *next_free;  // or null
  uint32_t *status;
};

cudaError_t launch_build_block_tables(const BlockTables &p, cudaStream_t stream);

// Copies whole blocks of up to four arrays: array i holds num_blocks blocks
// of bytes[i] (a multiple of 16) each.
struct BlockCopy {
  const int32_t *pairs;  // [num_pairs][2] (source, destination)
  int32_t num_pairs, num_blocks;
  uint8_t *base[4];
  int64_t bytes[4];
  uint32_t *status;
};

cudaError_t launch_copy_blocks(const BlockCopy &p, cudaStream_t stream);

struct SharedLaunch {
  const void *q, *k_cache, *k_scale, *v_cache, *v_scale, *v_zero;
  const int32_t *cu, *seq_lens, *block_table, *cu_groups, *prefix_lens;
  int32_t bt_stride, bt_cols, num_seqs, num_tokens, num_groups, hq, hk, d, num_blocks, bs;
  int32_t max_query_len, max_prefix_len, max_suffix_len;
  int32_t prefix_splits, suffix_splits;
  float softmax_scale;
  const float *sinks;
  void *out;
  float *lse;
  uint8_t *workspace;
  bool f8v4;
};

// Key segments of the prefix and of the suffix that fill the GPU for these
// host-side bounds.
struct SharedSplits {
  int32_t prefix, suffix;
};
SharedSplits shared_splits(int32_t num_seqs, int32_t num_tokens, int32_t num_groups, int32_t hq,
                           int32_t hk, int32_t d, int32_t max_query_len, int32_t max_prefix_len,
                           int32_t max_suffix_len);

cudaError_t launch_shared_prefix(const SharedLaunch &L, cudaStream_t stream);

}  // namespace paq8
