// Attention over whole prompts: packed bf16 rows q [T, Hq, D], k, v [Tk, Hk, D] of
// sequences of different lengths, no cache.  For query i of a sequence of q_len
// queries and k_len keys, row (i, q head):
//   out = sum_j p_j v_j / sum_j p_j,  lse = ln sum_j exp(scale q . k_j),
//   p_j = exp(scale q . k_j - m), over keys j <= k_len - q_len + i (causal; the last
//   `window` of them with a sliding window) or all keys.
//
// Bound by the tensor cores: 4 D Hq flops a query-key pair, on tcgen05 with fp32
// accumulators in TMEM.  128-row tiles (128 / qpk tokens x the qpk q heads of a kv head)
// against 128-key tiles:
//   S = Q K^T   both operands in shared memory, as TMA brings them (bf16, exact products)
//   P = 2^(S scale - m) by one thread a row, bf16, back into S's TMEM columns
//   O += P V    P from TMEM, V as it lies in memory (channels contiguous: the MMA's
//               N-major form)
// D 64 / 128: two row tiles a block share every K/V tile; while one's softmax runs the
// tensor core works on the other's products (TMEM: S/P 128 columns and O D columns
// each).  D 256: one row tile, whose S alternates between two buffers (O takes 256
// columns): QK(j + 1) runs behind the softmax of j.
// K and V pass through one ring of slots of a tile each (D 256: a quarter, 64 channels of
// a K tile or 32 keys of a V tile), freed by the commit of its last MMA.
// The maximum that P is taken against moves only when a tile's passes it by 2^8; O in TMEM
// is then rescaled by the softmax warps.  P is handed over in two halves, so that its
// product begins while the second is formed.  P is rounded to bf16 (the MMA's operands
// are of one type); sums and O are fp32.
// Warps: 4 softmax warps a row tile (one a TMEM lane quarter), one that issues the MMAs
// from one elected thread (one a row tile lost the alternation of the two and 20 %), one
// that issues the copies.
#include <algorithm>

#include "attn_common.cuh"
#include "launch.h"
#include "programmatic.cuh"
#include "prompt.h"
#include "segments.cuh"
#include "tcgen05.cuh"

namespace paq8 {

namespace {

struct PromptArgs {
  PromptAttention p;
  uint32_t *status;
  int32_t qpk, tile_tokens, block_tokens;  // tokens a row tile, a block
  int32_t num_items, num_splits;
  float scale_log2;
  float *part_acc;   // [T * Hq][splits][D]
  float2 *part_ml;   // [T * Hq][splits]
};

template <int D>
struct PromptCfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;      // row tiles a block
  static constexpr int kKeys = 128;                    // keys a tile
  static constexpr int kParts = D == 256 ? 4 : 1;      // slots of a K tile, and of a V tile
  static constexpr int kKChunks = D / 64 / kParts;     // 64-channel chunks of a K slot
  static constexpr int kVKeys = kKeys / kParts;        // keys of a V slot
  static constexpr int kSlotBytes = kKeys * D * 2 / kParts;
  static constexpr int kSlots = 10 * 16384 / kSlotBytes;
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kQOff = kSlots * kSlotBytes;
  static constexpr int kBarOff = kQOff + kTiles * kQBytes;
  static constexpr int kItemOff = kBarOff + 384;       // two items, the answer
  static constexpr int kSmem = kItemOff + 256 + 1024;
  static constexpr int kSoftmaxWarps = 4 * kTiles;
  // two row tiles: warps in whole groups of four, so that registers can move from the
  // last group (168 a thread at launch, 88 after) to the softmax (208)
  static constexpr int kThreads = kTiles == 2 ? 384 : (kSoftmaxWarps + 2) * 32;
  static constexpr float kMargin = 8.0f;  // log2 of the largest p
  // TMEM columns of S/P and of O, by row tile (D 64, 128) or by S buffer (D 256)
  __device__ static __forceinline__ uint32_t s_col(int i) { return D == 256 ? 256 + 128 * i : 256 * i; }
  __device__ static __forceinline__ uint32_t o_col(int i) { return D == 256 ? 0 : 256 * i + 128; }
  static_assert(kSmem <= 232448, "shared memory");
};

// barriers (8 bytes each)
constexpr int kBarFull = 0;    // [slots] copy -> MMA
constexpr int kBarEmpty = 10;  // [slots] commit of a slot's last MMA -> copy
constexpr int kBarQ = 20;      // [2] copies of a row tile's q -> MMA
constexpr int kBarS = 22;      // [2] commit of QK -> softmax
constexpr int kBarP = 24;      // [2][half] 64 columns of P in TMEM (4 warps) -> MMA
constexpr int kBarO = 28;      // [2] commit of the last PV -> epilogue (D 256: [1], of every PV -> rescale)
constexpr int kBarDrain = 30;  // commit of all that was issued, before the end
constexpr int kBarQFree = 31;  // [2] commit of a row tile's last QK -> copy
constexpr int kBarItem = 33;   // [2] an item's bounds stand in shared memory -> MMA, softmax
constexpr int kBarItemFree = 35;  // [2] they were read (MMA, softmax warps) -> copy
constexpr int kBarNext = 37;   // the answer to the request for another block's work -> copy
constexpr int kNumBars = 38;

// kind::f16 with bf16 operands, fp32 accumulator; n_major: B's N dimension contiguous.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool n_major) {
  return tc::idesc_f16(m, n) | (1u << 7) | (1u << 10) | (n_major ? 1u << 16 : 0u);
}

// A box of a tiled map at (x, y, z[, w]) into shared memory.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// What a block works on: two row tiles (D 256: one) of a sequence and kv head.
struct alignas(64) Item {
  int nt;              // 128-key tiles from t0 on, of the row tile that sees most; -1: no more items
  int tiles[2];        // of each row tile
  int end[2];          // keys before it are seen by some row of the row tile
  int t0, k0, k_len;
  int shift;           // last key of query i: shift (causal: + i)
  int q0, tok0, n_tok;
  int h, segment;
};
static_assert(sizeof(Item) == 64, "two of them, and the answer on a 16-byte boundary");

// The tiles and keys of the row tiles of a block that starts at token tok0 of a sequence:
// what the kernel and the join agree on.
struct Rows {
  int first_tile, tiles[2], end[2], nt;
};
template <int TILES>
__device__ __forceinline__ Rows rows_of(const PromptArgs &a, int q_len, int k_len, int tok0) {
  Rows r;
  const int shift = a.p.causal ? k_len - q_len : k_len - 1;
  const auto last_of = [&](int i) { return a.p.causal ? shift + i : shift; };
  const int n_tok = min(a.block_tokens, q_len - tok0);
  const int last0 = last_of(tok0);
  const int first0 = a.p.window > 0 ? max(0, last0 - a.p.window + 1) : 0;
  // (a row whose last key is negative sees none)
  r.first_tile = min(first0, max(0, last_of(tok0 + n_tok - 1))) / 128;
  r.tiles[1] = r.end[1] = 0;
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    const int n = min(a.tile_tokens, n_tok - i * a.tile_tokens);  // tokens of the row tile
    r.end[i] = n > 0 ? max(0, last_of(tok0 + i * a.tile_tokens + n - 1) + 1) : 0;
    r.tiles[i] = max(0, (r.end[i] + 127) / 128 - r.first_tile);
  }
  r.nt = max(r.tiles[0], r.tiles[1]);
  return r;
}
// Tiles a segment of a block of nt tiles, and how many segments that makes.
__device__ __forceinline__ int segment_tiles(const PromptArgs &a, int nt) {
  return max(1, (nt + a.num_splits - 1) / a.num_splits);
}
__device__ __forceinline__ int segment_count(const PromptArgs &a, int nt) {
  const int t = segment_tiles(a, nt);
  return max(1, (nt + t - 1) / t);
}

// Asks for the work of a block of this grid that has not started: its number (or none) is
// written to 16 bytes of shared memory, completing on bar.
__device__ __forceinline__ void ask_for_block(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          answer),
      "r"(bar)
      : "memory");
}
// The answer: false where no block was left.
__device__ __forceinline__ bool answered_block(uint32_t answer, uint32_t &block) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r;\n\t}"
      : "=r"(block), "=r"(got)
      : "r"(answer)
      : "memory");
  return got != 0;
}

template <int D>
__global__ void __launch_bounds__(PromptCfg<D>::kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using C = PromptCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (smem_base - smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kMmaWarp = C::kSoftmaxWarps, kCopyWarp = C::kSoftmaxWarps + 1;

  const uint32_t bars = smem_base + C::kBarOff;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t tmem_slot = bars + 8 * kNumBars;
  volatile Item *items = reinterpret_cast<volatile Item *>(smem + C::kItemOff);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBarQ + s), 1);
      mbar_init(bar(kBarS + s), 1);
      mbar_init(bar(kBarP + 2 * s), 4);
      mbar_init(bar(kBarP + 2 * s + 1), 4);
      mbar_init(bar(kBarO + s), 1);
      mbar_init(bar(kBarQFree + s), 1);
      mbar_init(bar(kBarItem + s), 1);
      mbar_init(bar(kBarItemFree + s), C::kSoftmaxWarps + 1);
    }
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarNext), 1);
    fence_barrier_init();
  }
  wait_for_predecessor();
  if (warp == kMmaWarp) tc::alloc(tmem_slot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kBarOff + 8 * kNumBars);
  bool ok = true;

  // An item's slots in the order of use: K(0), then (D 256: K(1)), then V(j), K(j + 1 or 2), ...
  constexpr int kAhead = D == 256 ? 2 : 1;

  if (warp == kCopyWarp) {
    // ============================================================ copies
    if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (lane == 0) {
      prefetch_tensormap(&map_q);
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
    }
    const uint32_t answer = smem_base + C::kItemOff + 2 * sizeof(Item);
    int used = 0;        // slots filled so far
    int q_used[2] = {0, 0};
    int count = 0, asked = 0;
    uint32_t block = blockIdx.x;
    const auto fits = [&](int q0, int q_len, int k0, int k_len) {
      return q_len > 0 && q0 >= 0 && q0 <= a.p.num_tokens - q_len && k0 >= 0 && k_len >= 0 &&
             k0 <= a.p.num_keys - k_len;
    };
    // 2 to 32 sequences: the one with most keys first, lane s holding sequence s and where its
    // items stand in that order (4 chunks behind prefixes of 1 to 6000 keys, D 256: 124 us, 133 in
    // the order of the batch).  A sequence whose bounds are out of range has none, and is flagged.
    const bool ranked = a.p.num_seqs > 1 && a.p.num_seqs <= 32;
    int start = 0, items_of = 0, q0_of = 0, k0_of = 0, q_len_of = 0, k_len_of = 0;
    if (ranked) {
      int keys = -1;
      if (lane < a.p.num_seqs) {
        q0_of = a.p.cu_q[lane];
        k0_of = a.p.cu_k[lane];
        q_len_of = a.p.cu_q[lane + 1] - q0_of;
        k_len_of = a.p.cu_k[lane + 1] - k0_of;
        if (fits(q0_of, q_len_of, k0_of, k_len_of)) {
          items_of = (q_len_of - 1) / a.block_tokens + 1;
          keys = k_len_of;
        } else if (q_len_of != 0) {
          flag_status(a.status, PA_DEV_BAD_SEQ);
        }
      }
#pragma unroll 1
      for (int s = 0; s < a.p.num_seqs; ++s) {
        const int other = __shfl_sync(0xffffffffu, keys, s), n = __shfl_sync(0xffffffffu, items_of, s);
        if (other > keys || (other == keys && s < lane)) start += n;
      }
    }
    for (bool more = true; more && ok;) {
      // ---- which rows, which keys; the heaviest first (later queries see more keys)
      Item it;
      it.h = static_cast<int>(block % static_cast<uint32_t>(a.p.hk));
      const int rest = static_cast<int>(block / static_cast<uint32_t>(a.p.hk));
      it.segment = rest / a.num_items;
      int q_len;
      if (ranked) {
        const int item = rest % a.num_items - start;
        const unsigned mine = __ballot_sync(0xffffffffu, item >= 0 && item < items_of);
        const int seq = mine ? __ffs(mine) - 1 : 0;
        it.q0 = __shfl_sync(0xffffffffu, q0_of, seq);
        it.k0 = __shfl_sync(0xffffffffu, k0_of, seq);
        q_len = __shfl_sync(0xffffffffu, q_len_of, seq);
        it.k_len = __shfl_sync(0xffffffffu, k_len_of, seq);
        // of a sequence, the last queries first
        const int tok0 = __shfl_sync(0xffffffffu, items_of - 1 - item, seq) * a.block_tokens;
        it.tok0 = mine ? tok0 : -1;
      } else {
        const int item = a.num_items - 1 - rest % a.num_items;
        const int seq = find_seq(a.p.cu_q, a.p.num_seqs, a.block_tokens, item, lane);
        it.q0 = a.p.cu_q[seq];
        it.k0 = a.p.cu_k[seq];
        q_len = a.p.cu_q[seq + 1] - it.q0;
        it.k_len = a.p.cu_k[seq + 1] - it.k0;
        it.tok0 = (item - (a.block_tokens == 1 ? it.q0 : it.q0 / a.block_tokens + seq)) * a.block_tokens;
      }
      bool valid = it.tok0 >= 0 && it.tok0 < q_len && fits(it.q0, q_len, it.k0, it.k_len);
      Rows rows;
      if (valid) {
        rows = rows_of<C::kTiles>(a, q_len, it.k_len, it.tok0);
        valid = it.segment < segment_count(a, rows.nt);
      }
      if (valid) {
        it.shift = a.p.causal ? it.k_len - q_len : it.k_len - 1;
        it.n_tok = min(a.block_tokens, q_len - it.tok0);
        const int most = segment_tiles(a, rows.nt), skipped = it.segment * most;
        it.t0 = rows.first_tile + skipped;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          it.end[i] = rows.end[i];
          it.tiles[i] = min(most, max(0, rows.tiles[i] - skipped));
        }
        it.nt = max(it.tiles[0], it.tiles[1]);
        const int b = count & 1;
        if (lane == 0) {
          if (count >= 2) ok = mbar_wait(bar(kBarItemFree + b), ((count >> 1) - 1) & 1);
          if (ok) {
            volatile int *dst = reinterpret_cast<volatile int *>(items + b);
            const int *src = reinterpret_cast<const int *>(&it);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(Item) / 4); ++i) dst[i] = src[i];
            mbar_arrive(bar(kBarItem + b));
          }
          auto take = [&]() -> int {
            const int s = used % C::kSlots;
            if (used >= C::kSlots && !mbar_wait(bar(kBarEmpty + s), ((used / C::kSlots) - 1) & 1)) return -1;
            ++used;
            mbar_arrive_expect_tx(bar(kBarFull + s), C::kSlotBytes);
            return s;
          };
          auto load_q = [&](int i) -> bool {
            if (it.tiles[i] == 0) return true;
            if (q_used[i] > 0 && !mbar_wait(bar(kBarQFree + i), (q_used[i] - 1) & 1)) return false;
            ++q_used[i];
            mbar_arrive_expect_tx(bar(kBarQ + i), a.tile_tokens * a.qpk * D * 2);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(smem_base + C::kQOff + i * C::kQBytes + c * (128 * 128), &map_q, c * 64,
                          it.h * a.qpk, it.q0 + it.tok0 + i * a.tile_tokens, bar(kBarQ + i));
            return true;
          };
          auto load_k = [&](int j) -> bool {
#pragma unroll
            for (int c = 0; c < C::kParts; ++c) {
              const int s = take();
              if (s < 0) return false;
              tma_load_4d(smem_base + s * C::kSlotBytes, &map_k, 0, it.k0 + (it.t0 + j) * C::kKeys,
                          c * C::kKChunks, it.h, bar(kBarFull + s));
            }
            return true;
          };
          auto load_v = [&](int j) -> bool {
#pragma unroll
            for (int c = 0; c < C::kParts; ++c) {
              const int s = take();
              if (s < 0) return false;
              tma_load_4d(smem_base + s * C::kSlotBytes, &map_v, 0,
                          it.k0 + (it.t0 + j) * C::kKeys + c * C::kVKeys, 0, it.h, bar(kBarFull + s));
            }
            return true;
          };
          // K(0), K(1) before V(0) at D 256; V(j), K(j + 1 or 2) then
          if (ok) ok = load_q(0);
          if (ok && C::kTiles == 2) ok = load_q(1);
#pragma unroll 1
          for (int j = -kAhead; ok && j < it.nt; ++j) {
            if (j >= 0) ok = load_v(j);
            if (ok && j + kAhead < it.nt) ok = load_k(j + kAhead);
          }
        }
        ++count;
      }
      // ---- the next block's number: asked for when this item's copies are on their way (at its
      // start a block would hold the next while others are idle)
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kBarNext), 16);
        ask_for_block(answer, bar(kBarNext));
      }
      // (in the batch's order no item need be that of a sequence with bad bounds: item n looks at
      // sequence n (and n + num_items, ...))
      if (!ranked && it.h == 0 && it.segment == 0) {
        const int64_t n = rest % a.num_items;
        for (int64_t s = n + int64_t{lane} * a.num_items; s < a.p.num_seqs; s += int64_t{32} * a.num_items) {
          const int q0 = a.p.cu_q[s], k0 = a.p.cu_k[s];
          const int len = a.p.cu_q[s + 1] - q0;
          if (len != 0 && !fits(q0, len, k0, a.p.cu_k[s + 1] - k0)) flag_status(a.status, PA_DEV_BAD_SEQ);
        }
      }
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(kBarNext), asked & 1));
      ++asked;
      more = ok && answered_block(answer, block);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    }
    if (lane == 0) {
      const int b = count & 1;
      if (ok && count >= 2) ok = mbar_wait(bar(kBarItemFree + b), ((count >> 1) - 1) & 1);
      if (ok) {
        items[b].nt = -1;
        mbar_arrive(bar(kBarItem + b));
      }
      // no block gives up its shared memory before its own copies have landed
      for (int i = max(0, used - C::kSlots); i < used; ++i)
        mbar_wait(bar(kBarFull + i % C::kSlots), (i / C::kSlots) & 1);
      for (int i = 0; i < C::kTiles; ++i)
        if (q_used[i] > 0) mbar_wait(bar(kBarQ + i), (q_used[i] - 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ============================================================ MMA issue
    if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (tc::elect_one()) {
      constexpr uint32_t id_qk = idesc_bf16(128, C::kKeys, false);
      constexpr uint32_t id_pv = idesc_bf16(128, D, true);
      const uint64_t q_desc = tc::desc_sw128(smem_base + C::kQOff);
      const uint64_t k_desc = tc::desc_sw128(smem_base);
      const uint64_t v_desc = tc::desc_mn_major(smem_base, C::kVKeys * 128);
      // (a phase that is complete, the common case, costs a test half of what a waiting test
      // does; the tensor core's queue holds five MMAs, 320 cycles, to hide it behind)
      auto wait = [&](int i, uint32_t parity) {
        return mbar_test(bar(i), parity) || (ok = mbar_wait(bar(i), parity));
      };
      int nt, t0, k_len;           // of the item
      int tile_count[2] = {0, 0};  // tiles of the items before, by row tile
      int q_count[2] = {0, 0};
      struct Place {  // in the ring
        int slot;
        uint32_t parity;
        __device__ __forceinline__ Place next() const {
          return slot + 1 == C::kSlots ? Place{0, parity ^ 1u} : Place{slot + 1, parity};
        }
      };
      Place place = {0, 0u};  // of the next slot that comes into use
      auto wait_slot = [&](const Place &at) { return wait(kBarFull + at.slot, at.parity); };
      // S(buffer i) = Q K(j)^T, K(j) at `at` (D 256: and the three slots after it, waited for
      // here); free: the tile's slots have no later use
      auto issue_qk = [&](int tile, int i, Place &at, bool free) -> bool {
        const uint32_t s_tmem = tmem + C::s_col(i);
        const uint64_t qd = q_desc + tile * (C::kQBytes >> 4);
#pragma unroll
        for (int c = 0; c < C::kParts; ++c) {
          if (C::kTiles == 1) {
            if (!wait_slot(at)) return false;
            tc::fence_after();
          }
          const uint64_t kd = k_desc + at.slot * (C::kSlotBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < 4 * C::kKChunks; ++ks) {  // 64 channels: 16 KB of Q and of K
            const int step = c * 4 * C::kKChunks + ks;
            tc::mma_f16(s_tmem, qd + ((step >> 2) * 1024 + 2 * (step & 3)),
                        kd + ((ks >> 2) * 1024 + 2 * (ks & 3)), id_qk, step > 0 ? 1u : 0u);
          }
          if (free) tc::commit(bar(kBarEmpty + at.slot));
          if (C::kTiles == 1) at = at.next();
        }
        tc::commit(bar(kBarS + i));
        return true;
      };
      // O(tile) += P(buffer i) V(j), over the 16-key steps below `end`, V(j) at `at`
      auto issue_pv = [&](int j, int tile, int i, uint32_t p_parity, int end, Place &at, bool free,
                          bool last) -> bool {
        const uint32_t p_tmem = tmem + C::s_col(i), o_tmem = tmem + C::o_col(tile);
        const int keys = end - (t0 + j) * C::kKeys;
        const int past = k_len - (t0 + j) * C::kKeys;  // keys from here on are another sequence's
        uint64_t vd = v_desc + at.slot * (C::kSlotBytes >> 4);
        if (!wait(kBarP + 2 * i, p_parity)) return false;
        tc::fence_after();
        auto second_half = [&]() {
          if (!wait(kBarP + 2 * i + 1, p_parity)) return false;
          tc::fence_after();
          return true;
        };
#pragma unroll
        for (int c = 0; c < C::kParts; ++c) {
          if (C::kParts > 1 && c == C::kParts / 2 && !second_half()) return false;
          if (C::kTiles == 1) {
            if (!wait_slot(at)) return false;
            tc::fence_after();
            vd = v_desc + at.slot * (C::kSlotBytes >> 4);
          }
          if (keys >= C::kKeys) {
#pragma unroll
            for (int ks = 0; ks < C::kVKeys / 16; ++ks) {
              const int step = c * (C::kVKeys / 16) + ks;
              if (C::kParts == 1 && ks == 4 && !second_half()) return false;
              tc::mma_f16_ts(o_tmem, p_tmem + step * 8, vd + ks * 128, id_pv, (j > 0 || step > 0) ? 1u : 0u);
            }
          } else {
            if (C::kParts == 1 && !second_half()) return false;
            // rows of the last step that lie past the sequence meet P = 0, but may hold
            // infinities: zeros in their place
            if (past < keys + 15 && past % 16 && past / 16 * 16 / C::kVKeys == c) {
              const uint32_t v = smem_base + at.slot * C::kSlotBytes;
              const int r0 = past - c * C::kVKeys, r1 = (past / 16 + 1) * 16 - c * C::kVKeys;
#pragma unroll 1
              for (int r = r0; r < r1; ++r)
#pragma unroll 1
                for (int b = 0; b < D * 2; b += 16)
                  sts128(v + (b >> 7) * (C::kVKeys * 128) + r * 128 + (b & 127), make_uint4(0u, 0u, 0u, 0u));
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
#pragma unroll 1
            for (int ks = 0; ks < C::kVKeys / 16; ++ks) {
              const int step = c * (C::kVKeys / 16) + ks;
              if (step * 16 < keys)
                tc::mma_f16_ts(o_tmem, p_tmem + step * 8, vd + ks * 128, id_pv, (j > 0 || step > 0) ? 1u : 0u);
            }
          }
          if (free) tc::commit(bar(kBarEmpty + at.slot));
          if (C::kTiles == 1) at = at.next();
        }
        if (C::kTiles == 1 || last) tc::commit(bar(kBarO + tile));
        return true;
      };
#pragma unroll 1
      for (int count = 0;; ++count) {
        const int b = count & 1;
        if (!wait(kBarItem + b, (count >> 1) & 1)) break;
        nt = items[b].nt;
        t0 = items[b].t0;
        k_len = items[b].k_len;
        const int n0 = items[b].tiles[0], n1 = items[b].tiles[1];
        const int end0 = items[b].end[0], end1 = items[b].end[1];
        mbar_arrive(bar(kBarItemFree + b));
        if (nt < 0) break;
        if (nt == 0) continue;
        if constexpr (C::kTiles == 2) {
          // What both row tiles need is waited for while the queue is full, so that nothing
          // stands between a P and its MMAs: V(j) behind QK(j) of the first tile, K(j + 1)
          // behind PV(j - 1) of the second.  A row tile's S buffer is free once its PV is
          // issued: MMAs of one thread execute in order.  A slot is freed by the last row
          // tile that uses it.
          Place k_at = place, v_at = place;  // of K(j), V(j - 1)
          wait_slot(k_at);
#pragma unroll 1
          for (int j = 0; ok && j <= nt; ++j) {
            const Place v_next = k_at.next(), k_next = v_next.next();
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              const int n = i ? n1 : n0, other = i ? 0 : n1, end = i ? end1 : end0;
              const int before = i ? tile_count[1] : tile_count[0];
              if (ok && j >= 1 && j - 1 < n)
                issue_pv(j - 1, i, i, (before + j - 1) & 1, end, v_at, i == 1 || j - 1 >= other, j == n);
              if (i == 1 && ok && j + 1 < nt) wait_slot(k_next);
              if (ok && j < n && (j > 0 || wait(kBarQ + i, (i ? q_count[1] : q_count[0]) & 1))) {
                tc::fence_after();
                issue_qk(i, i, k_at, i == 1 || j >= other);
                if (j == n - 1) tc::commit(bar(kBarQFree + i));
              }
              if (i == 0 && ok && j < nt) wait_slot(v_next);
            }
            v_at = v_next;
            if (j < nt) place = k_at = k_next;  // (two slots a tile)
          }
          tile_count[1] += n1;
          q_count[1] += n1 > 0;
        } else {
          if (wait(kBarQ, q_count[0] & 1)) tc::fence_after();
#pragma unroll 1
          for (int j = 0; ok && j < nt + 2; ++j) {
            const int g = tile_count[0] + j;  // S buffers alternate from item to item
            if (j >= 2) issue_pv(j - 2, 0, g & 1, ((g - 2) >> 1) & 1, end0, place, true, true);
            if (ok && j < nt) issue_qk(0, g & 1, place, true);
            if (ok && j == nt - 1) tc::commit(bar(kBarQFree));
          }
        }
        tile_count[0] += n0;
        q_count[0] += n0 > 0;
        if (!ok) break;
      }
      // no block gives up its shared memory and TMEM before its own MMAs have ended
      tc::commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0);
    }
    __syncwarp();
  } else if (warp < C::kSoftmaxWarps) {
    // ============================================================ softmax
    if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int tile = warp >> 2;
    const int quarter = warp & 3;  // TMEM lanes of this warp
    const int row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = a.scale_log2;
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity)) != 0; };
    int before = 0, with_tiles = 0;  // tiles, and items with tiles, of this row tile so far
#pragma unroll 1
    for (int count = 0;; ++count) {
      const int b = count & 1;
      if (!wait(kBarItem + b, (count >> 1) & 1)) { ok = false; break; }
      const int nt = items[b].nt, t0 = items[b].t0, n = items[b].tiles[tile], shift = items[b].shift;
      const int row_tok = row / a.qpk;
      const int tok = items[b].tok0 + tile * a.tile_tokens + row_tok;
      const bool valid = row < a.tile_tokens * a.qpk && tok < items[b].tok0 + items[b].n_tok;
      const int head = items[b].h * a.qpk + row - row_tok * a.qpk, out_tok = items[b].q0 + tok;
      const int segment = items[b].segment;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarItemFree + b));
      if (nt < 0) break;
      // visible keys [lo, limit]; rows that are not written take all, unmasked
      const int limit = !valid ? 0x7fffffff : a.p.causal ? shift + tok : shift;
      const int lo = valid && a.p.window > 0 ? max(0, limit - a.p.window + 1) : 0;
      float m_used = -INFINITY;  // the maximum O is scaled to (log2 units)
      float l = 0.0f;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const int g = before + j;
        const int i = C::kTiles == 2 ? tile : g & 1;  // S buffer
        const uint32_t use = C::kTiles == 2 ? g : g >> 1;
        if (!wait(kBarS + i, use & 1)) { ok = false; break; }
        tc::fence_after();
        const uint32_t t_s = t_lane + C::s_col(i);
        const int key0 = (t0 + j) * C::kKeys;
        // scores that are masked, or whose factor would turn the order around, are scaled first
        const bool first_scaled = key0 + C::kKeys - 1 > limit || key0 < lo || sl2 <= 0.0f;
        const float mul = first_scaled ? 1.0f : sl2;
        uint32_t sr[4][32];
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) tc::ld32(t_s + cb * 32, sr[cb]);
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) tc::wait_loaded(sr[cb]);
        const auto scale_first = [&](uint32_t(&x)[32], int first) {  // keys from `first` on
#pragma unroll
          for (int c = 0; c < 32; ++c)
            x[c] = __float_as_uint(first + c > limit || first + c < lo ? -INFINITY : __uint_as_float(x[c]) * sl2);
        };
        if (first_scaled) {
#pragma unroll
          for (int cb = 0; cb < 4; ++cb) scale_first(sr[cb], key0 + cb * 32);
        }
        float mx4[4];
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) {
          mx4[cb] = fmaxf(__uint_as_float(sr[cb][0]), __uint_as_float(sr[cb][1]));
#pragma unroll
          for (int c = 2; c < 32; c += 2)
            mx4[cb] = fmax3(mx4[cb], __uint_as_float(sr[cb][c]), __uint_as_float(sr[cb][c + 1]));
        }
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * mul;
        // D 256: every PV's phase is waited for, in order, before O is rescaled or behind this
        // tile's P; D 64, 128: PV(j - 1) was before S(j)
        bool await_pv = C::kTiles == 1 && j > 0;
        const bool grow = valid && mx > m_used + C::kMargin;
        if (__any_sync(0xffffffffu, grow)) {
          float f = 1.0f;  // factor of what O and l hold
          if (grow) {
            f = fast_exp2(m_used - mx);
            l *= f;
            m_used = mx;
          }
          if (await_pv) {
            if (!wait(kBarO, (g - 1) & 1)) { ok = false; break; }
            tc::fence_after();
            await_pv = false;
          }
          if (j > 0) {
#pragma unroll 1
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t orr[32];
              tc::ld32(t_lane + C::o_col(tile) + cb * 32, orr);
              tc::wait_loaded(orr);
#pragma unroll
              for (int c = 0; c < 32; ++c) orr[c] = __float_as_uint(__uint_as_float(orr[c]) * f);
              tc::st32(t_lane + C::o_col(tile) + cb * 32, orr);
            }
            tc::wait_st();
          }
        }
        // P against m_used as bf16 pairs, and its sum in fp32, 64 columns at a time
        const float neg_m = m_used == -INFINITY ? 0.0f : -m_used;  // (no key yet: all masked)
        const uint64_t mul2 = f32x2_pack(mul, mul), neg_m2 = f32x2_pack(neg_m, neg_m);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pw[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const uint32_t(&x)[32] = sr[2 * half + (c >> 5)];
            float x0, x1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(x[c & 31]), __uint_as_float(x[(c & 31) + 1])),
                                   mul2, neg_m2),
                         x0, x1);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            sum[(c >> 1) & 1] = f32x2_add(sum[(c >> 1) & 1], f32x2_pack(p0, p1));
            pw[c >> 1] = pack_bf162(p0, p1);
          }
          tc::st32(t_s + half * 32, pw);
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarP + 2 * i + half));
        }
        float s0, s1, s2, s3;
        f32x2_unpack(sum[0], s0, s1);
        f32x2_unpack(sum[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        if (await_pv && !wait(kBarO, (g - 1) & 1)) { ok = false; break; }
      }
      // ---- epilogue: O / l as bf16, lse; the sink as one term more of the sum
      if (ok && n > 0) ok = wait(kBarO + tile, C::kTiles == 1 ? (before + n - 1) & 1 : with_tiles & 1);
      before += n;
      with_tiles += n > 0;
      if (!ok) break;
      {
        tc::fence_after();
        const int64_t at = static_cast<int64_t>(out_tok) * a.p.hq + head;
        const bool seen = valid && limit >= 0 && n > 0;  // else no key: out = 0
        if (a.num_splits > 1) {
          const int64_t prow = at * a.num_splits + segment;
          float *dst = a.part_acc + prow * D;
#pragma unroll 1
          for (int cb = 0; n > 0 && cb < D / 32; ++cb) {
            uint32_t orr[32];
            tc::ld32(t_lane + C::o_col(tile) + cb * 32, orr);
            tc::wait_loaded(orr);
            if (seen) {
#pragma unroll
              for (int c = 0; c < 32; c += 4)
                *reinterpret_cast<uint4 *>(dst + cb * 32 + c) = make_uint4(orr[c], orr[c + 1], orr[c + 2], orr[c + 3]);
            }
          }
          if (valid) a.part_ml[prow] = seen ? make_float2(m_used, l) : make_float2(-INFINITY, 0.0f);
          continue;
        }
        float o_mul = 1.0f;
        if (a.p.sinks && valid) {
          const float sk = a.p.sinks[head] * kLog2e;
          const float mn = fmaxf(m_used, sk);
          if (mn > -INFINITY) {
            o_mul = fast_exp2(m_used - mn);
            l = l * o_mul + fast_exp2(sk - mn);
            m_used = mn;
          }
        }
        const float inv = seen && l != 0.0f ? o_mul / l : 0.0f;  // (l is 0 where every score is -inf)
        // Four neighbouring lanes exchange 16-byte pieces, so that they write 64 bytes of one row
        // after another (a lane writing its own row kept the memory pipe for 3000 cycles and more,
        // and the waits behind it).
        int out_row[4];  // rows of this lane's four, -1: not written
#pragma unroll
        for (int r = 0; r < 4; ++r)
          out_row[r] = __shfl_sync(0xffffffffu, valid ? static_cast<int>(at) : -1, (lane & ~3) + r);
        const bool odd = lane & 1, high = lane & 2;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t orr[32];
          if (n > 0) {
            tc::ld32(t_lane + C::o_col(tile) + cb * 32, orr);
            tc::wait_loaded(orr);
          }
          uint32_t piece[4][4];  // [row of the four][word] of piece lane & 3
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t x[4];  // word k of this row's pieces
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = seen ? pack_bf162(__uint_as_float(orr[8 * i + 2 * k]) * inv,
                                       __uint_as_float(orr[8 * i + 2 * k + 1]) * inv)
                          : 0u;
            const uint32_t a01 = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[1], 1);
            const uint32_t a23 = __shfl_xor_sync(0xffffffffu, odd ? x[2] : x[3], 1);
            const uint32_t e0 = odd ? a01 : x[0], o0 = odd ? x[1] : a01;  // even and odd rows
            const uint32_t e1 = odd ? a23 : x[2], o1 = odd ? x[3] : a23;
            const uint32_t be = __shfl_xor_sync(0xffffffffu, high ? e0 : e1, 2);
            const uint32_t bo = __shfl_xor_sync(0xffffffffu, high ? o0 : o1, 2);
            piece[0][k] = high ? be : e0;
            piece[1][k] = high ? bo : o0;
            piece[2][k] = high ? e1 : be;
            piece[3][k] = high ? o1 : bo;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (out_row[r] >= 0)
              *reinterpret_cast<uint4 *>(a.p.out + static_cast<int64_t>(out_row[r]) * D + cb * 32 + (lane & 3) * 8) =
                  make_uint4(piece[r][0], piece[r][1], piece[r][2], piece[r][3]);
        }
        if (valid && a.p.lse) a.p.lse[at] = l == 0.0f ? -INFINITY : (m_used + log2f(l)) * kLn2;
      }
    }
  } else {
    if constexpr (C::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  }
  if (!ok) flag_status(a.status, PA_DEV_TIMEOUT);

  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// Joins the triples of a row (token, q head), one warp a row.
template <int D>
__global__ void __launch_bounds__(128) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  // (the prompt kernel lets nothing start early)
  wait_for_predecessor();
  if (at >= static_cast<int64_t>(a.p.num_tokens) * a.p.hq) return;
  const int tok = static_cast<int>(at / a.p.hq);
  const int head = static_cast<int>(at % a.p.hq);
  const int seq = find_seq(a.p.cu_q, a.p.num_seqs, 1, tok, lane);
  const int q0 = a.p.cu_q[seq], q_len = a.p.cu_q[seq + 1] - q0;
  const int k0 = a.p.cu_k[seq], k_len = a.p.cu_k[seq + 1] - k0;
  if (tok < q0 || tok - q0 >= q_len || q0 < 0 || q0 > a.p.num_tokens - q_len || k0 < 0 || k_len < 0 ||
      k0 > a.p.num_keys - k_len)
    return;
  const int tok0 = (tok - q0) / a.block_tokens * a.block_tokens;
  const int n = segment_count(a, rows_of<PromptCfg<D>::kTiles>(a, q_len, k_len, tok0).nt);
  const float sink = a.p.sinks ? a.p.sinks[head] * kLog2e : -INFINITY;
  const int64_t prow = at * a.num_splits;
  join_row<D>(a.part_acc + prow * D, a.part_ml + prow, n, sink, a.p.out + at * D,
              a.p.lse ? a.p.lse + at : nullptr, lane);
}

// Rows x heads x channels of bf16 as a tiled map with 128-byte swizzle.
bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box) {
  const EncodeTiledFn fn = encode_tiled_fn();
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box,
                  step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const PromptAttention &p, cudaStream_t stream) {
  using C = PromptCfg<D>;
  PromptArgs a;
  a.p = p;
  a.status = reinterpret_cast<uint32_t *>(p.workspace);
  a.qpk = p.hq / p.hk;
  a.tile_tokens = 128 / a.qpk;
  a.block_tokens = a.tile_tokens * C::kTiles;
  a.num_items = a.block_tokens == 1 ? p.num_tokens : p.num_tokens / a.block_tokens + p.num_seqs;
  if (p.window >= p.num_keys) a.p.window = 0;  // no query leaves a key out
  a.scale_log2 = p.softmax_scale * kLog2e;
  CUtensorMap mq, mk, mv;
  const cuuint64_t qd[3] = {D, static_cast<cuuint64_t>(p.hq), static_cast<cuuint64_t>(p.num_tokens)};
  const cuuint64_t qs[2] = {D * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
  const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(a.qpk), static_cast<cuuint32_t>(a.tile_tokens)};
  // K and V rows as [kv head][64-channel chunk][key][64 channels]
  // (without keys no copy is made: any valid map)
  const bool none = p.num_keys == 0;
  const cuuint64_t kd[4] = {64, static_cast<cuuint64_t>(none ? 1 : p.num_keys), D / 64, static_cast<cuuint64_t>(p.hk)};
  const cuuint64_t ks[3] = {static_cast<cuuint64_t>(none ? p.q_stride : p.k_stride) * 2, 128, D * 2};
  const cuuint64_t vs[3] = {static_cast<cuuint64_t>(none ? p.q_stride : p.v_stride) * 2, 128, D * 2};
  const cuuint32_t kb[4] = {64, C::kKeys, C::kKChunks, 1};
  const cuuint32_t vb[4] = {64, C::kVKeys, D / 64, 1};
  if (!encode(&mq, p.q, 3, qd, qs, qb) || !encode(&mk, none ? p.q : p.k, 4, kd, ks, kb) ||
      !encode(&mv, none ? p.q : p.v, 4, kd, vs, vb))
    return cudaErrorInvalidValue;
  static DeviceOnce configured;
  const cudaError_t e = configured.get(nullptr, [](int, int *) {
    const cudaError_t r = registers_cover(reinterpret_cast<const void *>(prompt_kernel<D>), C::kThreads,
                                          C::kTiles == 2 ? 256 * 208 + 128 * 88 : 0);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  a.num_splits = prompt_splits(p.num_seqs, p.num_tokens, p.hq, p.hk, p.d, p.max_key_len);
  const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.hq;
  while (a.num_splits > 1 &&
         p.workspace_bytes < 256 + static_cast<size_t>(rows) * a.num_splits * (D + 2) * sizeof(float))
    --a.num_splits;
  a.part_acc = reinterpret_cast<float *>(p.workspace + 256);
  a.part_ml = reinterpret_cast<float2 *>(a.part_acc + rows * a.num_splits * D);
  const int64_t blocks = static_cast<int64_t>(a.num_items) * p.hk * a.num_splits;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const cudaError_t launched = launch_kernel(prompt_kernel<D>, dim3(static_cast<unsigned>(blocks)), C::kThreads,
                                             C::kSmem, stream, a, mq, mk, mv);
  if (launched != cudaSuccess || a.num_splits == 1) return launched;
  return launch_kernel(prompt_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, stream, a);
}

}  // namespace

// Key segments: blocks that leave a quarter of the SMs idle, and more, are split until two stand
// in line for each, or one where segments of 512 keys at least do not make two.  Whole rounds: 512
// queries on 4096 keys (32/8 heads, D 128) take 72 us in 4 segments (256 blocks), 85 in 5 (320),
// 79 in one; 256 on 8192 at D 256 91 us in 4, 111 in 5, 121 in one; 16 on 8192 at D 128 43 and 117.
int32_t prompt_splits(int32_t num_seqs, int32_t num_tokens, int32_t hq, int32_t hk, int32_t d,
                      int32_t max_key_len) {
  const int64_t block_tokens = 128 / (hq / hk) * (d == 256 ? 1 : 2);
  const int64_t blocks = std::max<int64_t>(num_seqs, (num_tokens + block_tokens - 1) / block_tokens) * hk;
  if (4 * blocks >= 3 * 152) return 1;
  const int64_t two = 2 * 152 / blocks;
  int64_t ns = std::min<int64_t>({two, max_key_len / 512, kMaxSegments});
  if (ns < two && ns * blocks > 152) ns = 152 / blocks;
  return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(ns, kMaxSegments)));
}

cudaError_t launch_prompt_attention(const PromptAttention &p, cudaStream_t stream) {
  switch (p.d) {
    case 64: return launch_d<64>(p, stream);
    case 128: return launch_d<128>(p, stream);
    case 256: return launch_d<256>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paq8
