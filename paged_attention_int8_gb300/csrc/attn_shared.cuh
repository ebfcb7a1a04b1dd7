// Pieces shared by the kernels of attention over a shared prefix: arguments,
// the work a block takes, and where its partial results go.
//
// The sequences of a batch stand in groups (cu_groups, consecutive sequences);
// the first prefix_lens[g] keys of every sequence of group g are the same and
// are read once for all of the group's queries, through the block-table row
// of the group's first sequence.  The call's work is two sets of items over
// the same cache:
//   prefix: all query tokens of a group x keys [0, P), every query sees all;
//   suffix: the query tokens of one sequence x keys [P, seq_len), causal.
// Each item's keys are cut into segments of whole 64-key tiles, and each
// segment leaves one triple per row (a row = query token x q head):
//   m = max_j s_j (log2 units), l = sum_j 2^(s_j - m), acc = sum_j 2^(s_j - m) v_j,
// which the join kernel (attn_shared.cu) merges:
//   M = max m_k, w_k = 2^(m_k - M), out = sum w_k acc_k / sum w_k l_k,
//   lse = (M + log2 sum w_k l_k) ln 2,
// a sink joining as one more term with no value.  Triples are fp32.
#pragma once

#include "attn_common.cuh"
#include "attn_f8v4.cuh"
#include "launch.h"
#include "serving.h"

namespace paq8 {

constexpr int kSegTile = 64;  // keys per tile of the segment rule, for every kernel
constexpr int kFewRows = 8;   // rows per kv head that the rows kernel takes

struct SharedArgs {
  AttnArgs a;  // q, caches, tables, partials (part_acc, part_ml), status, scale, sinks
  const int32_t *cu_groups;    // [G + 1] first sequence of each group
  const int32_t *prefix_lens;  // [G]
  int32_t num_groups;
  int32_t ns_p, ns_s;          // prefix and suffix segments: triples of a row
  int32_t seg_p, seg_s;        // 64-key tiles per segment
  int32_t n_pblocks, n_sblocks;  // row blocks of the prefix and suffix items in the grid
  int32_t few_rows;            // suffixes of at most this many rows are the rows kernel's
  int32_t max_rows;            // no suffix kernel takes more rows than this
};

// Warp-cooperative search: the last i in [0, n) with key(i) <= target, key
// non-decreasing (find_seq over any key).
template <class K>
__device__ __forceinline__ int find_last(int n, int target, int lane, K &&key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int idx = lo + lane * step;
    const bool le = idx < hi && key(idx) <= target;
    const unsigned ball = __ballot_sync(0xffffffffu, le);
    const int k = ball ? 31 - __clz(ball) : 0;
    lo = lo + k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// First query token of group g (cu_seqlens_q of its first sequence).
__device__ __forceinline__ int group_token(const SharedArgs &s, int g) {
  const int q = s.cu_groups[g];
  return q < 0 || q > s.a.num_seqs ? 0x7fffffff : s.a.cu_seqlens_q[q];
}

// The prefix length that sequence seq shares, -1 when no group holds it or
// the group's entries are out of range.
__device__ __forceinline__ int prefix_of(const SharedArgs &s, int seq, int lane) {
  const int g = find_last(s.num_groups, seq, lane, [&](int i) { return s.cu_groups[i]; });
  if (s.cu_groups[g] > seq || s.cu_groups[g + 1] <= seq) return -1;
  return s.prefix_lens[g];
}

// Query rows per kv head of a sequence of q_len tokens (saturating).
__device__ __forceinline__ int rows_of(const SharedArgs &s, int q_len) {
  return q_len > (1 << 26) ? 1 << 30 : q_len * s.a.qpk;
}

// Segments of keys [begin, end): the rule every kernel and the join share.
__device__ __forceinline__ int shared_segments(int begin, int end, int seg_tiles, int ns) {
  return end <= begin ? 0 : segments_of(begin, end, kSegTile, seg_tiles, ns);
}

// What a block works on: rows of n_tok query tokens from token q0 on, keys
// [kv_begin, kv_end) of block-table row `row`.  Token i of the block sees keys
// up to limit0 + i * limit_step.  Its rows' triples go to segment slot `slot`
// of their ns_p + ns_s.
struct SharedWork {
  int row, q0, n_tok, kv_begin, kv_end, limit0, limit_step, slot;
};

// Keys of segment sigma of [begin, end).
__device__ __forceinline__ bool segment_keys(int begin, int end, int seg_tiles, int ns, int sigma,
                                             SharedWork &w) {
  const int n = shared_segments(begin, end, seg_tiles, ns);
  if (sigma >= n) return false;
  const int t0 = begin / kSegTile;
  w.kv_begin = max(begin, (t0 + sigma * seg_tiles) * kSegTile);
  w.kv_end = sigma == ns - 1 ? end
                             : static_cast<int>(min(static_cast<int64_t>(end),
                                   (static_cast<int64_t>(t0) + static_cast<int64_t>(sigma + 1) * seg_tiles) *
                                       kSegTile));
  return w.kv_begin < w.kv_end;
}

// Prefix item: row block `blk` (block_q tokens of one group), segment sigma.
// Executed by whole warps; false: nothing to do.
__device__ __forceinline__ bool prefix_work(const SharedArgs &s, int blk, int sigma, int block_q,
                                            int lane, SharedWork &w) {
  const AttnArgs &a = s.a;
  const int g = find_last(s.num_groups, blk, lane, [&](int i) {
    const int t = group_token(s, i);
    return t == 0x7fffffff ? t : t / block_q + i;
  });
  const int c0 = group_token(s, g), c1 = group_token(s, g + 1);
  const int P = s.prefix_lens[g];
  if (c0 < 0 || c1 > a.num_tokens || c0 > c1 || P < 0) {
    if (threadIdx.x == 0) flag_status(a.status, PA_DEV_BAD_SEQ);
    return false;
  }
  const int tok0 = (blk - (c0 / block_q + g)) * block_q;
  if (tok0 < 0 || tok0 >= c1 - c0 || P == 0) return false;
  w.row = s.cu_groups[g];
  w.q0 = c0 + tok0;
  w.n_tok = min(block_q, c1 - c0 - tok0);
  w.slot = sigma;
  if (!segment_keys(0, P, s.seg_p, s.ns_p, sigma, w)) return false;
  w.limit0 = w.kv_end - 1;
  w.limit_step = 0;
  return true;
}

// Suffix item: row block `blk` (block_q tokens of one sequence), segment sigma.
__device__ __forceinline__ bool suffix_work(const SharedArgs &s, int blk, int sigma, int block_q,
                                            int lane, SharedWork &w) {
  const AttnArgs &a = s.a;
  const int seq = find_seq(a.cu_seqlens_q, a.num_seqs, block_q, blk, lane);
  const int c0 = a.cu_seqlens_q[seq], c1 = a.cu_seqlens_q[seq + 1];
  const int first = block_q == 1 ? c0 : c0 / block_q + seq;
  const int tok0 = (blk - first) * block_q;
  if (tok0 < 0 || tok0 >= c1 - c0) return false;
  if (rows_of(s, c1 - c0) <= s.few_rows) return false;
  const int seq_len = a.seq_lens[seq], ctx = seq_len - (c1 - c0);
  const int P = prefix_of(s, seq, lane);
  if (c0 < 0 || c1 > a.num_tokens || P < 0 || ctx < P) {
    if (sigma == 0 && tok0 == 0 && threadIdx.x == 0) flag_status(a.status, PA_DEV_BAD_SEQ);
    return false;
  }
  w.row = seq;
  w.q0 = c0 + tok0;
  w.n_tok = min(block_q, c1 - c0 - tok0);
  w.slot = s.ns_p + sigma;
  if (!segment_keys(P, ctx + tok0 + w.n_tok, s.seg_s, s.ns_s, sigma, w)) return false;
  w.limit0 = ctx + tok0;
  w.limit_step = 1;
  return true;
}

// Triple of row (token, q head), segment slot k.
__device__ __forceinline__ int64_t triple_at(const SharedArgs &s, int token, int hh, int k) {
  return (static_cast<int64_t>(token) * s.a.hq + hh) * (s.ns_p + s.ns_s) + k;
}

}  // namespace paq8
