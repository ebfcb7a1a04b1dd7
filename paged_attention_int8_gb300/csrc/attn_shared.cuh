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
//   m (log2 units), l = sum_j 2^(s_j - m), acc = sum_j 2^(s_j - m) v_j,
// m one of the scores s_j, at most 15 below the largest (so that every 2^(s_j - m)
// is inside fp16), which the join kernel (attn_shared.cu) merges:
//   M = max m_k, w_k = 2^(m_k - M), out = sum w_k acc_k / sum w_k l_k,
//   lse = (M + log2 sum w_k l_k) ln 2,
// a sink joining as one more term with no value.  Triples are fp32.
//
// What is rounded, as in the package's other attention kernels: P and V' (code * scale;
// idx * scale + zero) to fp16, one rounding each, since the tensor cores take 16-bit
// operands (tf32 ones at half the rate) and 11 bits are 3 more than the bf16 output
// keeps; l sums the P before its rounding.  q to fp16, exact down to 2^-14.  Keys are
// exact (fp8: every code is an fp16 value; q8: integer codes, or two fp16 parts), so
// that the LSE is an fp32 sum's.  Against 64 bits the output's error is 1.68e-3 of its
// size (rms), of which the bf16 rounding alone is 1.66e-3 (64 to 128 requests, D = 128).
#pragma once

#include "attn_common.cuh"
#include "attn_f8v4.cuh"
#include "launch.h"
#include "programmatic.cuh"
#include "serving.h"

namespace paq8 {

constexpr int kSegTile = 64;  // keys per tile of the segment rule, for every kernel
constexpr int kFewRows = 32;  // rows per kv head that the rows kernel takes

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
  int32_t row_passes;          // rows kernel: passes over the keys that cover them
  int32_t capacity;            // keys that the columns of a table row hold: none past them is walked,
                               // so that no look-up passes the columns, whatever the row stride
  int32_t first;               // row-tile kernel: it is the call's first
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

// The last i in [0, n) with v[i] <= target (0 if there is none), by one thread.
__device__ __forceinline__ int last_at_most(const int32_t *v, int n, int target) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= target) lo = mid;
    else hi = mid;
  }
  return lo;
}

// First query token of group g (cu_seqlens_q of its first sequence).
__device__ __forceinline__ int group_token(const SharedArgs &s, int g) {
  const int q = s.cu_groups[g];
  return q < 0 || q > s.a.num_seqs ? 0x7fffffff : s.a.cu_seqlens_q[q];
}

// The prefix length that sequence seq shares (what a table row holds at most), -1
// when no group holds it or the group's entries are out of range.
__device__ __forceinline__ int prefix_of(const SharedArgs &s, int seq, int lane) {
  if (s.num_groups <= 32) {  // a lane a group: one round of loads
    int first = 0x7fffffff, end = 0, len = 0;
    if (lane < s.num_groups) {
      first = s.cu_groups[lane];
      end = s.cu_groups[lane + 1];
      len = s.prefix_lens[lane];
    }
    const unsigned ball = __ballot_sync(0xffffffffu, first <= seq);
    const int g = ball ? 31 - __clz(ball) : 0;
    if (__shfl_sync(0xffffffffu, first, g) > seq || __shfl_sync(0xffffffffu, end, g) <= seq) return -1;
    return min(__shfl_sync(0xffffffffu, len, g), s.capacity);
  }
  const int g = find_last(s.num_groups, seq, lane, [&](int i) { return s.cu_groups[i]; });
  if (s.cu_groups[g] > seq || s.cu_groups[g + 1] <= seq) return -1;
  return min(s.prefix_lens[g], s.capacity);
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

// Prefix item `item` of the grid: a row block (block_q tokens of one group) and
// a segment, segment-major.  Up to 32 groups are counted exactly (one lane
// each), so that the grid's unused items stand at its end; more are found by
// search over the key first_token / block_q + g, which leaves gaps.  Executed
// by whole warps; false: nothing to do.
__device__ __forceinline__ bool prefix_work(const SharedArgs &s, int item, int block_q, int lane,
                                            SharedWork &w) {
  const AttnArgs &a = s.a;
  int g, tok0, sigma, c0, c1, P;
  if (s.num_groups <= 32) {
    int b0 = 0, b1 = 0, first = 0, len = 0;
    if (lane < s.num_groups) {
      len = s.prefix_lens[lane];
      first = s.cu_groups[lane];
      b0 = group_token(s, lane);
      b1 = group_token(s, lane + 1);
    }
    const int mine = b0 >= 0 && b1 <= a.num_tokens && b0 < b1 ? (b1 - b0 + block_q - 1) / block_q : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    if (total == 0 || item >= total * s.ns_p) return false;
    const int blk = item % total;
    sigma = item / total;
    const unsigned past = __ballot_sync(0xffffffffu, upto > blk);
    g = __ffs(past) - 1;
    c0 = __shfl_sync(0xffffffffu, b0, g);
    c1 = __shfl_sync(0xffffffffu, b1, g);
    w.row = __shfl_sync(0xffffffffu, first, g);
    P = __shfl_sync(0xffffffffu, len, g);
    tok0 = (blk - __shfl_sync(0xffffffffu, upto - mine, g)) * block_q;
  } else {
    const int blk = item % s.n_pblocks;
    sigma = item / s.n_pblocks;
    if (sigma >= s.ns_p) return false;
    g = find_last(s.num_groups, blk, lane, [&](int i) {
      const int t = group_token(s, i);
      return t == 0x7fffffff ? t : t / block_q + i;
    });
    c0 = group_token(s, g);
    c1 = group_token(s, g + 1);
    if (c0 < 0 || c1 > a.num_tokens) return false;  // the suffix items flag it
    tok0 = (blk - (c0 / block_q + g)) * block_q;
    if (tok0 < 0 || tok0 >= c1 - c0) return false;
    w.row = s.cu_groups[g];
    P = s.prefix_lens[g];
  }
  if (P <= 0 || w.row >= a.num_seqs) return false;
  if (P > s.capacity) {  // pages past the table's columns: flagged and left out
    if (threadIdx.x == 0) flag_status(a.status, PA_DEV_BAD_BLOCK);
    P = s.capacity;
  }
  w.q0 = c0 + tok0;
  w.n_tok = min(block_q, c1 - c0 - tok0);
  w.slot = sigma;
  if (!segment_keys(0, P, s.seg_p, s.ns_p, sigma, w)) return false;
  w.limit0 = w.kv_end - 1;
  w.limit_step = 0;
  return true;
}

// Row blocks of all groups at most: the items of one prefix segment.
inline int prefix_blocks(int num_tokens, int num_groups, int block_q) {
  return num_groups <= 32
             ? static_cast<int>((num_tokens + static_cast<int64_t>(num_groups) * (block_q - 1)) / block_q)
             : num_tokens / block_q + num_groups;
}

// Rows that the rows kernel takes a pass over the keys, for sequences of at most `most`
// rows: two 8-row tiles where the registers hold them without spills.  D = 128, 48
// requests of up to 32 rows and 2000 keys: two passes of two 69 us (q8) and 62 (fp8 /
// 4-bit), one of four 83 and 75; D = 64, of 32 rows 46 and 45, one of four 56 and 51;
// D = 256, of 12 rows: two passes of one 64 and 64, one of two 73 and 69.
inline int rows_per_pass(int d, int64_t most) { return d == 256 || most <= 8 ? 8 : 16; }

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
  const int end = ctx + tok0 + w.n_tok;
  if (end > s.capacity && threadIdx.x == 0) flag_status(a.status, PA_DEV_BAD_BLOCK);
  if (!segment_keys(P, min(end, s.capacity), s.seg_s, s.ns_s, sigma, w)) return false;
  w.limit0 = ctx + tok0;
  w.limit_step = 1;
  return true;
}

// Where triples stand.  A row of kv head h is token * qpk + (q head - h * qpk),
// so the rows of a block are consecutive; acc is [slot][h][D / 4][row][4], which
// a block of any kernel writes (and the join reads) in whole sectors, and
// (m, l) is [slot][h][row].
__device__ __forceinline__ int64_t rows_total(const SharedArgs &s) {
  return static_cast<int64_t>(s.a.num_tokens) * s.a.qpk;
}
// First row of slot k, head h in (m, l) pairs.
__device__ __forceinline__ int64_t ml_at(const SharedArgs &s, int k, int h) {
  return (static_cast<int64_t>(k) * s.a.hk + h) * rows_total(s);
}
// acc of slot k, head h: channel c of row r at + (c / 4) * rows_total * 4 + r * 4 + c % 4.
template <int D>
__device__ __forceinline__ float *acc_at(const SharedArgs &s, int k, int h) {
  return s.a.part_acc + ml_at(s, k, h) * D;
}

// q rows r0 .. r0 + 31 of a block (row r: q head h qpk + r % qpk of query token
// q0 + r / qpk; rows at and past n_rows are left out) to shared memory at dst, by
// one warp: whole lines, all in flight, and no registers held.  A lane that reads
// its own row from global memory touches a line per piece: the 4096 lookups of a
// block's rows took 4 us.  Pieces of 16 bytes stand swizzled for reads by row.
template <int D>
__device__ __forceinline__ uint32_t q_piece(uint32_t dst, int r, int piece) {
  return dst + r * (2 * D) + ((piece * 16) ^ ((r & 7) << 4));
}
template <int D>
__device__ __forceinline__ void copy_q_rows(const AttnArgs &a, uint32_t dst, int q0, int h, int r0,
                                            int n_rows, int lane) {
  constexpr int kPieces = D / 8, kStep = 32 / kPieces;
  const int magic = (65536 + a.qpk - 1) / a.qpk;  // r / qpk = r magic / 65536 for r < 256, qpk <= 16
  const uint16_t *base = a.q + (static_cast<int64_t>(q0) * a.hq + h * a.qpk) * D + lane % kPieces * 8;
#pragma unroll 8
  for (int i = 0; i < 32; i += kStep) {
    const int r = i + lane / kPieces;
    const int tok = ((r0 + r) * magic) >> 16;
    if (r0 + r < n_rows)
      cp_async16(q_piece<D>(dst, r, lane % kPieces),
                 base + (static_cast<int64_t>(tok) * (a.hq - a.qpk) + r0 + r) * D);
  }
  cp_async_commit();
}

}  // namespace paq8
