// Internal launch interface of the attention over whole prompts for the C ABI (api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace paq8 {

struct PromptAttention {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements from token to token
  const int32_t *cu_q, *cu_k;
  int32_t num_seqs, num_tokens, num_keys, hq, hk, d;
  int32_t max_query_len, max_key_len;
  float softmax_scale;
  const float *sinks;
  int32_t window;
  bool causal;
  uint16_t *out;
  float *lse;
  uint8_t *workspace;
  size_t workspace_bytes;
};

// Key segments that a call of these sizes takes.
int32_t prompt_splits(int32_t num_seqs, int32_t num_tokens, int32_t hq, int32_t hk, int32_t d,
                      int32_t max_key_len);
cudaError_t launch_prompt_attention(const PromptAttention &p, cudaStream_t stream);

}  // namespace paq8
