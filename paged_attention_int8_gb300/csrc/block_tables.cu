// build_block_tables: a serving step's block table, slot map, positions and
// length arrays from its request lengths.
//
// Per sequence s (context c, query length q, page size bs):
//   seq_len = c + q, cu[s] = sum of q before s,
//   held = ceil(c / bs), end = ceil((c + q) / bs),
//   private copy: q > 0, c % bs != 0 and the page of position c holds shared
//     tokens (shared_len > floor(c / bs) * bs),
//   first = floor(c / bs) with a private copy, else held,
//   page p < first: the source row's entry; first <= p < end: the free list's
//     entry free_head + (new pages of earlier sequences) + p - first;
//   slot of position x = page(x / bs) * bs + x % bs.
//
// A block takes 8 sequences (one warp each) and one chunk of their tokens and
// pages (grid y), so that a long prompt or a wide table row is spread over
// blocks; every grid-y-th chunk where one each would be more than kMaxBlocks.
// The sums over earlier sequences are formed by every block that needs them,
// straight from the lengths (12 bytes a sequence, L2 resident): one launch, no
// scan across blocks, no order that could change results.  A block whose chunk
// holds neither tokens nor new pages copies old entries only and takes no sum.
#include "common.cuh"
#include "launch.h"
#include "programmatic.cuh"
#include "serving.h"

namespace paq8 {

namespace {

constexpr int kWarps = 8;          // sequences per block
constexpr int kTokenChunk = 256;   // tokens of a sequence per block
constexpr int kPageChunk = 1024;   // pages of a sequence per block
constexpr int kMaxBlocks = 65535;  // about; grid y has no more rows

struct SeqPlan {
  int ctx, q, first, end;  // pages [first, end) are new
  bool cow, ok;
};

__device__ __forceinline__ SeqPlan plan_of(const BlockTables &p, int s) {
  SeqPlan r;
  r.ctx = p.context_lens[s];
  r.q = p.query_lens[s];
  r.ok = r.ctx >= 0 && r.q >= 0 && r.q <= p.num_tokens && r.ctx <= 0x7fffffff - 64 - r.q;
  if (!r.ok) r.ctx = r.q = 0;
  const int bs = p.block_size;
  const int floor_page = r.ctx / bs;
  const int held = (r.ctx + bs - 1) / bs;
  r.cow = r.q > 0 && held != floor_page && p.shared_lens && p.shared_lens[s] > floor_page * bs;
  r.first = r.cow ? floor_page : held;
  r.end = (r.ctx + r.q + bs - 1) / bs;
  return r;
}

__device__ __forceinline__ int clamp_i32(int64_t v) {
  return static_cast<int>(v > 0x7fffffff ? 0x7fffffff : v);
}

// kLoop: a block takes more chunks than one.  A kernel of its own, since the loop alone
// costs registers (112 against 64): 1024 samples of 131072 tokens 15.4 us against 12.0.
template <bool kLoop>
__global__ void __launch_bounds__(kWarps * 32) block_tables_kernel(const BlockTables p) {
  __shared__ int64_t sum_q[kWarps], sum_n[kWarps];
  __shared__ int own_q[kWarps], own_n[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s0 = static_cast<int>(blockIdx.x) * kWarps;
  const int s = s0 + warp;
  const bool last_x = blockIdx.x == gridDim.x - 1;
  const int y = static_cast<int>(blockIdx.y), dy = static_cast<int>(gridDim.y);
  const bool active = s < p.num_seqs;

  wait_for_predecessor();  // the lengths, and every reader of what is written here
  SeqPlan me = {0, 0, 0, 0, false, true};
  if (active) me = plan_of(p, s);
  const int n_new = me.end - me.first;  // 0 when q == 0: end == held == first
  // chunks of this sequence's tokens and table entries; the block's are y, y + dy, ...
  const int n_chunks = max(1, max((me.q + kTokenChunk - 1) / kTokenChunk,
                                  (min(me.end, p.table_stride) + kPageChunk - 1) / kPageChunk));
  // the sums are needed for the heads of the arrays (chunk 0), for tokens and
  // new pages of a chunk, and for the padding rows behind the last token
  const bool need = y == 0 || last_x || y * kTokenChunk < me.q || (kLoop && y + dy < n_chunks) ||
                    (y * kPageChunk < me.end && (y + 1) * kPageChunk > me.first);
  int64_t before_q = 0, before_n = 0;
  int64_t total_q = 0, total_n = 0;
  if (__syncthreads_or(need)) {
    int64_t aq = 0, an = 0;
    for (int i = threadIdx.x; i < s0; i += kWarps * 32) {
      const SeqPlan o = plan_of(p, i);
      aq += o.q;
      an += o.end - o.first;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      aq += __shfl_xor_sync(0xffffffffu, aq, o);
      an += __shfl_xor_sync(0xffffffffu, an, o);
    }
    if (lane == 0) {
      sum_q[warp] = aq;
      sum_n[warp] = an;
      own_q[warp] = me.q;
      own_n[warp] = n_new;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      total_q += sum_q[w] + own_q[w];
      total_n += sum_n[w] + own_n[w];
      before_q += sum_q[w] + (w < warp ? own_q[w] : 0);
      before_n += sum_n[w] + (w < warp ? own_n[w] : 0);
    }
  }

  const int head = p.free_head ? *p.free_head : 0;
  uint32_t bad = me.ok ? 0u : PA_DEV_BAD_SEQ;
  if (active) {
    // the source row, or -1: none
    const int row = p.source_rows ? p.source_rows[s] : s;
    const bool row_ok = row >= 0 && row < p.num_source_rows;
    const uint32_t bad_old = row_ok ? PA_DEV_BAD_BLOCK : PA_DEV_BAD_SEQ;  // an old page is missing
    if (!row_ok && me.ctx > 0) bad |= PA_DEV_BAD_SEQ;
    const int32_t *src = p.source_table + static_cast<int64_t>(row_ok ? row : 0) * p.source_stride;
    int32_t *dst = p.block_table + static_cast<int64_t>(s) * p.table_stride;
    auto old_entry = [&](int page) {
      return row_ok && page < p.source_stride ? src[page] : -1;
    };
    // the free list's entry of new page `page`, -1 when there is none
    auto new_entry = [&](int page) {
      const int64_t at = head + before_n + (page - me.first);
      if (head < 0 || at >= p.num_free) {
        bad |= PA_DEV_NO_BLOCKS;
        return -1;
      }
      const int b = p.free_blocks[at];
      if (b < 0 || b >= p.num_blocks) {
        bad |= PA_DEV_BAD_BLOCK;
        return -1;
      }
      return b;
    };

    if (y == 0 && lane == 0) {
      p.cu_seqlens_q[s] = clamp_i32(before_q);
      p.seq_lens[s] = me.ctx + me.q;
      if (me.end > p.table_stride) bad |= PA_DEV_BAD_BLOCK;
      if (before_q + me.q > p.num_tokens) bad |= PA_DEV_BAD_SEQ;
    }
    // the pair comes from the block that owns the private page's entry (it is
    // replaced below, in place perhaps: read here before)
    const int pair_chunk = me.cow ? min(me.first, p.table_stride - 1) / kPageChunk : 0;
#pragma unroll 1
    for (int chunk = y; chunk < n_chunks; chunk = kLoop ? chunk + dy : n_chunks) {
      const int64_t tok_lo = static_cast<int64_t>(chunk) * kTokenChunk;
      const int64_t page_lo = static_cast<int64_t>(chunk) * kPageChunk;
      if (p.copy_pairs && chunk == pair_chunk && lane == 0) {
        int from = -1, to = -1;
        if (me.cow) {
          from = old_entry(me.first);
          to = me.first < p.table_stride ? new_entry(me.first) : -1;
          if (from < 0 || from >= p.num_blocks) bad |= bad_old;
          if (from < 0 || from >= p.num_blocks || to < 0) from = to = -1;
        }
        p.copy_pairs[2 * s] = from;
        p.copy_pairs[2 * s + 1] = to;
      }
      __syncwarp();

      // ---- table entries of this chunk
      const int pl = static_cast<int>(min(page_lo, static_cast<int64_t>(me.end)));
      const int ph = min(min(me.end, pl + kPageChunk), p.table_stride);
      const bool in_place = dst == src;
      const int split = max(pl, min(ph, me.first));  // old entries end here
      if (!in_place) {
        // entries that the source row has, a batch of loads ahead of their stores
        const int have = row_ok ? max(pl, min(split, p.source_stride)) : pl;
        const int n = have - pl;
        constexpr int kBatch = 8;
        int i = lane;
        if (((reinterpret_cast<uintptr_t>(dst + pl) | reinterpret_cast<uintptr_t>(src + pl)) & 15u) == 0) {
          const int4 *from = reinterpret_cast<const int4 *>(src + pl);
          int4 *to = reinterpret_cast<int4 *>(dst + pl);
          for (; i < n / 4; i += 32 * kBatch) {
            int4 v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              if (i + 32 * j < n / 4) v[j] = from[i + 32 * j];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              if (i + 32 * j < n / 4) to[i + 32 * j] = v[j];
          }
          i = (n & ~3) + lane;
        }
        for (; i < n; i += 32 * kBatch) {
          int v[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (i + 32 * j < n) v[j] = src[pl + i + 32 * j];
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (i + 32 * j < n) dst[pl + i + 32 * j] = v[j];
        }
        for (int page = have + lane; page < split; page += 32) dst[page] = -1;
      }
      for (int page = split + lane; page < ph; page += 32) dst[page] = new_entry(page);

      // ---- slots and positions of this chunk
      const int th = static_cast<int>(min(static_cast<int64_t>(me.q), tok_lo + kTokenChunk));
      for (int i = static_cast<int>(min(tok_lo, static_cast<int64_t>(th))) + lane; i < th; i += 32) {
        const int64_t t = before_q + i;
        if (t >= p.num_tokens) break;  // flagged above
        const int x = me.ctx + i;
        const int page = x / p.block_size;
        int b = -1;
        if (page < p.table_stride) {
          b = page < me.first ? old_entry(page) : new_entry(page);
          if (page < me.first && (b < 0 || b >= p.num_blocks)) {
            bad |= bad_old;
            b = -1;
          }
        }
        p.slot_mapping[t] =
            b < 0 ? -1 : static_cast<int64_t>(b) * p.block_size + (x - page * p.block_size);
        if (p.positions) p.positions[t] = x;
      }
    }
  }
  if (last_x) {
    if (y == 0 && threadIdx.x == 0) {
      p.cu_seqlens_q[p.num_seqs] = clamp_i32(total_q);
      if (p.next_free) *p.next_free = head < 0 ? head : clamp_i32(head + total_n);
    }
    // padding rows behind the last token: no slot, position 0
    static_assert(kTokenChunk == kWarps * 32, "a thread a row");
    for (int64_t t = total_q + static_cast<int64_t>(y) * kTokenChunk + threadIdx.x; t < p.num_tokens;
         t += kLoop ? static_cast<int64_t>(dy) * kTokenChunk : p.num_tokens) {
      p.slot_mapping[t] = -1;
      if (p.positions) p.positions[t] = 0;
    }
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad && lane == 0) flag_status(p.status, bad);
}

}  // namespace

cudaError_t launch_build_block_tables(const BlockTables &p, cudaStream_t stream) {
  const int xs = p.num_seqs / kWarps + (p.num_seqs % kWarps != 0);
  const unsigned x = static_cast<unsigned>(xs > 0 ? xs : 1);  // padding rows without any sequence
  // chunks that cover every token of one sequence and every page of one row
  const int tc = (p.num_tokens + kTokenChunk - 1) / kTokenChunk;
  const int pc = (p.table_stride + kPageChunk - 1) / kPageChunk;
  const unsigned chunks = static_cast<unsigned>(tc > pc ? tc : pc);
  const unsigned most = x < kMaxBlocks ? kMaxBlocks / x : 1;
  if (chunks <= most)
    return launch_kernel(block_tables_kernel<false>, dim3(x, chunks), kWarps * 32, 0, stream, p);
  return launch_kernel(block_tables_kernel<true>, dim3(x, most), kWarps * 32, 0, stream, p);
}

}  // namespace paq8
