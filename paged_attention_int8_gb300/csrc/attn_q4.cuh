// What the kernels of the attention over the 4-bit cache share: their arguments, and which
// keys and key segments a block of query rows has.
#pragma once

#include "common.cuh"
#include "q4.h"
#include "segments.cuh"

namespace paq8 {
namespace q4 {

struct Q4Args {
  AttnQ4 p;
  uint32_t *status;
  float *part_acc;   // [T * Hq][splits][D]
  float2 *part_ml;   // [T * Hq][splits]
  int32_t qpk, qpk_inverse, block_tokens, num_items, num_splits;
  float scale_log2;
  int32_t seg_start[kMaxSegments];  // 16-key blocks of a range before each segment
};

// Visible keys of the block of rows that starts at token tok0 of a sequence, in
// 16-key blocks: what the kernel and the join agree on.
struct KeyRange {
  int begin, end;        // keys
  int first, blocks;     // 16-key blocks
};

__device__ __forceinline__ KeyRange key_range(const Q4Args &a, int seq_len, int q_len, int tok0) {
  const int n_tok = min(a.block_tokens, q_len - tok0);
  const int last0 = a.p.causal ? seq_len - q_len + tok0 : seq_len - 1;
  const int last1 = a.p.causal ? last0 + n_tok - 1 : last0;
  KeyRange r;
  // (keys past the table's columns have no page: left out here, flagged by the kernel)
  r.end = static_cast<int>(min(static_cast<int64_t>(last1) + 1, int64_t{a.p.table_columns} * a.p.bs));
  r.begin = a.p.window > 0 ? max(0, last0 - a.p.window + 1) : 0;
  r.first = r.begin / 16;
  r.blocks = r.end > r.begin ? (r.end - 1) / 16 + 1 - r.first : 0;
  return r;
}

__device__ __forceinline__ int segments(const Q4Args &a, int blocks) {
  int n = 1;
  while (n < a.num_splits && a.seg_start[n] < blocks) ++n;
  return n;
}

// The bounds of a sequence's metadata that the kernels rely on.
__device__ __forceinline__ bool valid_sequence(const Q4Args &a, int q0, int q_len, int seq_len) {
  return q0 >= 0 && q_len >= 0 && q0 <= a.p.num_tokens - q_len && seq_len >= (a.p.causal ? q_len : 0) &&
         (a.p.max_query_len > 1 || q_len <= 1);
}

// No item need be that of a sequence whose bounds are bad: item i looks at sequences i, i +
// num_items, ... (single tokens: its own), by one thread of one block.
__device__ __forceinline__ void flag_bad_sequences(const Q4Args &a, int item, int h, int sigma) {
  if (h != 0 || sigma != 0) return;
  for (int64_t s = item; s < a.p.num_seqs; s += a.num_items) {
    const int q0 = a.p.cu[s], q_len = a.p.cu[s + 1] - q0;
    if (q_len != 0 && !valid_sequence(a, q0, q_len, a.p.seq_lens[s])) flag_status(a.status, PA_DEV_BAD_SEQ);
  }
}

// Queries enter the products as fp16.  They are multiplied by the power of two that brings the
// largest of a block to 2^15 .. 2^16 (32 of them over 32 stay within fp16), which the scores'
// factors take back: bf16 values down to 2^-28 of the largest keep their bits, as q and as q / 16.
// Of a block with values from 65520 on (flagged) the power is 1.
struct QueryScale {
  float up, codes, zeros;  // of q; of sum_g s_g (q c 2^-24) and of sum_g z_g (q sum / 32)
};
__device__ __forceinline__ QueryScale query_scale(float largest, float scale_log2) {
  const int e = static_cast<int>(__float_as_uint(fminf(largest, 65504.0f)) >> 23) - 127;
  const int f = min(15 - e, 120);
  const auto power = [](int x) { return __uint_as_float(static_cast<uint32_t>(x + 127) << 23); };
  return {power(f), scale_log2 * power(24 - f), scale_log2 * power(5 - f)};
}
// The largest |x| of eight bf16 values (a NaN is passed over).
__device__ __forceinline__ float largest_of(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmax3(m, fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i])));
  return m;
}

// The largest of a warp's values >= 0, whose bits are in their order.
__device__ __forceinline__ float warp_largest(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// The tcgen05 kernel of a call (D 128, blocks of up to kTcRows rows); its triples and results are
// those of the mma.sync kernel.
constexpr int kTcRows = 64;
cudaError_t launch_attention_tc(const Q4Args &a, cudaStream_t stream);

}  // namespace q4
}  // namespace paq8
