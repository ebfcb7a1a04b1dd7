// Attention over a shared prefix on the 5th-generation tensor cores (tcgen05,
// TMEM): the prefix items of attn_shared.cuh for D = 64, 128.
//
// One block = 256 rows (256 / qpk query tokens of one group x the qpk q heads
// of one kv head) x one key segment, in 64-key tiles; every row sees every key,
// so only the last tile of a prefix is masked.  The pipeline is the one of the
// causal kernel (attn_prefill_tc.cu), whose measurements chose it: two 128-row
// halves share every converted K/V tile, both MMA A operands (q, P) live in
// TMEM, and warp 5 stages pages by TMA (6-stage ring), warps 0, 2, 3, 14 turn
// keys into fp16 hi and lo parts (q8: k = code * scale is exact as hi + lo; fp8
// keys are exact in one part), warps 4 and 15 turn values into fp16, warp 1
// issues the MMAs of the two halves alternately, and warps 6-13 run one row
// per thread of the online softmax, P taken against the maximum O is scaled to,
// which moves (O rescaled in TMEM) only when a tile's P sum would pass 2^15.
// Instead of the finished output a block leaves its rows' fp32 triples.
//
// Why a kernel of its own beside the causal one: its keys are split over
// blocks (64 requests on one prefix are 256 rows of 8 kv heads: 8 blocks
// without a split, 152 SMs to fill), its rows come from many sequences, and
// its result is a triple.
#include <type_traits>

#include "attn_shared.cuh"
#include "tcgen05.cuh"

namespace paq8 {

// Every block asks for all of an SM's shared memory, so that no block of the rows
// kernel comes beside it: with one a tile took 2700 cycles (fp8 / 4-bit, 16 rows:
// 4500), alone it takes 2000, and the rows run better on the SMs that a prefix cut
// into fewer segments leaves (4 groups of 96 requests: 42 us against 47; draft
// batches 58 against 62; 128 requests on 32768 keys 200 against 210).
constexpr int kSmemOfSm = 232448;

template <int D, int BS, bool F8>
struct SharedTcCfg {
  static constexpr int kTile = 64;
  static constexpr int kHalves = 2;
  static constexpr int kRows = 128 * kHalves;
  static constexpr int kSt = 6;  // staging stages (TMA)
  static constexpr int kWarps = 16;
  static constexpr int kKWarps = F8 ? 2 : 4, kVWarps = F8 ? 4 : 2;  // converters
  using L = std::conditional_t<F8, StageF8V4<D, BS, kTile>, StageLayout<D, BS, kTile>>;
  static constexpr int kKBytes = kTile * D * 2;  // one of K_hi, K_lo: [D/64][64 keys][128 B]
  static constexpr int kKSlot = 2 * kKBytes;     // K ring slot: hi then lo
  static constexpr int kVBytes = D * kTile * 2;  // V' ring slot: [D rows][64 keys]
  static constexpr int align1k(int x) { return (x + 1023) / 1024 * 1024; }
  static constexpr int kKOff = align1k(kSt * L::kBytes);
  static constexpr int kVOff = kKOff + 2 * kKSlot;
  static constexpr int kBarOff = kVOff + 2 * kVBytes;
  static constexpr int kSmem = kBarOff + 256 + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kHalfCols = 256;  // per half: S/P at +0, q at +64, O at +128
  static constexpr uint32_t kQCol = 64;
  static constexpr uint32_t kOCol = 128;
  static constexpr float kMaxTileSum = 32768.0f;  // bound on a tile's P sum (so on every P)
  static_assert(D == 64 || D == 128, "the tcgen05 kernel handles D = 64, 128");
  static_assert(kSmem <= kSmemOfSm, "shared memory");
  static_assert(kKSlot + 2 * kVBytes >= kRows * 2 * D, "q rows in K slot 1 and the V slots");
};

// barrier indices (8 bytes each, from kBarOff)
enum : int {
  kBarStFull = 0,    // [6] producer -> dequant (tx bytes)
  kBarStEmpty = 6,   // [6] dequant -> producer (6 warps)
  kBarKFull = 12,    // [2] K dequant -> MMA (kKWarps)
  kBarKEmpty = 14,   // [2] commit after both halves' QK -> K dequant
  kBarVFull = 16,    // [2] V dequant -> MMA (kVWarps)
  kBarVEmpty = 18,   // [2] commit after both halves' PV -> V dequant
  kBarSFull = 20,    // [half] commit after QK -> softmax of the half
  kBarPFull = 22,    // [half] softmax (P in TMEM) -> MMA (4 warps)
  kBarPvDone = 24,   // [half] commit after the last PV -> epilogue
  kBarQFull = 26,    // softmax (q written to TMEM) -> MMA (8 warps)
  kBarIdle = 27,     // commit after the last MMA issued -> MMA issuer
  kNumBars = 28
};

template <int D, int BS, bool F8>
__global__ void __launch_bounds__(512, 1)
    shared_tc_kernel(const __grid_constant__ SharedArgs sa, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v) {
  using C = SharedTcCfg<D, BS, F8>;
  using L = typename C::L;
  const AttnArgs &a = sa.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (smem_base - smem_u32(smem_raw));

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(sa.a.hk));

  if (threadIdx.x == 5 * 32) {
    prefetch_tensormap(&tmap_k);
    if constexpr (!F8) prefetch_tensormap(&tmap_v);
  }
  wait_for_predecessor();
  launch_dependents();
  SharedWork w;
  if (!prefix_work(sa, static_cast<int>(blockIdx.x / static_cast<unsigned>(a.hk)), a.block_q, lane, w))
    return;
  const int n_rows = w.n_tok * a.qpk;
  const int kv_end = w.kv_end;  // kv_begin starts a tile
  const int t0 = w.kv_begin / C::kTile;
  const int nt = (kv_end + C::kTile - 1) / C::kTile - t0;
  // the softmax warps' 32 rows of q each, in flight during the set-up: they stand
  // in K slot 1 and the V slots until they are in TMEM
  const int row0 = ((warp - 6) >> 2) * 128 + (warp & 3) * 32;
  const uint32_t q_smem = smem_base + C::kKOff + C::kKSlot + row0 * (2 * D);
  if (warp >= 6 && warp < 14) copy_q_rows<D>(a, q_smem, w.q0, h, row0, n_rows, lane);
  // half 1 holds no valid row when the block is short: it is then skipped
  const int halves = n_rows > 128 ? 2 : 1;

  const uint32_t bars = smem_base + C::kBarOff;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t tmem_slot = bars + 8 * kNumBars;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSt; ++s) {
      mbar_init(bar(kBarStFull + s), 1);
      mbar_init(bar(kBarStEmpty + s), 6);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBarKFull + s), C::kKWarps);
      mbar_init(bar(kBarKEmpty + s), 1);
      mbar_init(bar(kBarVFull + s), C::kVWarps);
      mbar_init(bar(kBarVEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBarSFull + s), 1);
      mbar_init(bar(kBarPFull + s), 4);
      mbar_init(bar(kBarPvDone + s), 1);
    }
    mbar_init(bar(kBarQFull), 8);
    mbar_init(bar(kBarIdle), 1);
    fence_barrier_init();
  }
  if (warp == 1) tc::alloc(tmem_slot, C::kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kBarOff + 8 * kNumBars);
  bool ok = true;

  if (warp == 5) {
    // ============================================================ producer
    // A lane per page and array issues that array's copy: one lane for all of them
    // took longer over the small copies of fp8 / 4-bit scales than a tile's MMAs.
    // Block-table entries are read 32 pages at a time; pages at or past the prefix's
    // end are not staged.
    const int n_pages = (kv_end + BS - 1) / BS;
    const int32_t *bt_row = a.block_table + static_cast<int64_t>(w.row) * a.bt_stride;
    const int my_page = lane >> 2, what = lane & 3;
    constexpr uint32_t kPageTx = F8 ? BS * D + BS * D / 2 + 4 * BS : 2 * BS * D + 4 * BS * (D / 32);
    int page_base = -(1 << 30), my_blk = -1;
    int stage = 0, phase = 1;  // of the ring; the parity of its being empty
    int j = 0;
    for (; ok && j < nt; ++j) {
      if (j >= C::kSt) {
        int there = 1;
        if (lane == 0) there = mbar_wait(bar(kBarStEmpty + stage), phase);
        if (!__shfl_sync(0xffffffffu, there, 0)) { ok = false; break; }
      }
      const int lp0 = (t0 + j) * L::kPages;
      if (lp0 - page_base >= 32) {
        page_base = lp0;
        const int lp = page_base + lane;
        my_blk = -1;
        if (lp < n_pages) {
          const int b = lp < a.bt_stride ? bt_row[lp] : -1;
          if (b >= 0 && b < a.num_blocks) my_blk = b;
          else flag_status(a.status, PA_DEV_BAD_BLOCK);
        }
      }
      const int blk = __shfl_sync(0xffffffffu, my_blk, lp0 + min(my_page, L::kPages - 1) - page_base);
      const bool mine = my_page < L::kPages && blk >= 0;
      const uint32_t full = bar(kBarStFull + stage);
      const int n_valid = __popc(__ballot_sync(0xffffffffu, mine && what == 0));
      if (lane == 0) mbar_arrive_expect_tx(full, n_valid * kPageTx);
      __syncwarp();
      if (mine) {
        const int64_t page = static_cast<int64_t>(blk) * a.hk + h;
        const uint32_t st = smem_base + stage * L::kBytes;
        if (what == 0)
          tma_load_2d(st + my_page * (BS * L::kRowBytes), &tmap_k, 0, static_cast<int32_t>(page * BS), full);
        if constexpr (F8) {
          if (what == 1)
            bulk_load(st + L::kVOff + my_page * (D * BS / 2),
                      reinterpret_cast<const uint8_t *>(a.v_cache) + page * (D * BS / 2), D * BS / 2, full);
          if (what == 2) bulk_load(st + L::kVsOff + my_page * (BS * 2), a.v_scale + page * BS, BS * 2, full);
          if (what == 3) bulk_load(st + L::kVzOff + my_page * (BS * 2), a.v_zero + page * BS, BS * 2, full);
        } else {
          constexpr int G = D / 32;
          if (what == 1)
            tma_load_2d(st + L::kVOff + my_page * (D * BS), &tmap_v, 0, static_cast<int32_t>(page * D), full);
          if (what == 2)
            bulk_load(st + L::kKsOff + my_page * (BS * G * 2), a.k_scale + page * BS * G, BS * G * 2, full);
          if (what == 3)
            bulk_load(st + L::kVsOff + my_page * (BS * G * 2), a.v_scale + page * BS * G, BS * G * 2, full);
        }
      }
      if (++stage == C::kSt) {
        stage = 0;
        phase ^= 1;
      }
      __syncwarp();
    }
    // the block holds its shared memory until its copies have landed, whoever gave up
    for (int i = max(0, j - C::kSt); lane == 0 && i < j; ++i)
      ok &= mbar_wait(bar(kBarStFull + i % C::kSt), (i / C::kSt) & 1);
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    // One elected lane runs the whole loop: under `elect` the compiler knows that
    // one thread is there and an MMA costs 5 instructions (18 under a predicate
    // or a branch on an earlier election, so that the issue, not the tensor core,
    // set the pace: 148 us against 138 on 128 requests and 32768 keys).
    if (tc::elect_one()) {
      constexpr uint32_t id_qk = tc::idesc_f16(128, 64);
      constexpr uint32_t id_qk_neg = id_qk | (1u << 14);  // negate B: K_lo is stored as -lo
      constexpr uint32_t id_pv = tc::idesc_f16(128, D);
      // O(half) += P(i, half) V'(i): A = P from the half's S/P columns
      auto issue_pv = [&](int i, int hf) -> bool {
        const int b = i & 1;
        if (hf == 0 && !mbar_wait(bar(kBarVFull + b), (i >> 1) & 1)) return false;
        if (!mbar_wait(bar(kBarPFull + hf), i & 1)) return false;
        tc::fence_after();
        const uint64_t v_desc = tc::desc_sw128(smem_base + C::kVOff + b * C::kVBytes);
        const uint32_t base = tmem + hf * C::kHalfCols;
#pragma unroll
        for (int ks = 0; ks < C::kTile / 16; ++ks)  // +32 bytes of K per step
          tc::mma_f16_ts(base + C::kOCol, base + ks * 8, v_desc + 2 * ks, id_pv,
                         (i > 0 || ks > 0) ? 1u : 0u);
        return true;
      };
      // S(half) = q K_hi(j)^T - q (-K_lo(j))^T: A = q from the half's TMEM columns
      auto issue_qk = [&](int j, int hf) {
        const uint64_t k_desc = tc::desc_sw128(smem_base + C::kKOff + (j & 1) * C::kKSlot);
        const uint32_t base = tmem + hf * C::kHalfCols;
#pragma unroll
        for (int part = 0; part < (F8 ? 1 : 2); ++part)  // F8: exact keys, no K_lo part
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t koff = part * C::kKBytes + (ks >> 2) * (64 * 128) + (ks & 3) * 32;
            tc::mma_f16_ts(base, base + C::kQCol + ks * 8, k_desc + (koff >> 4),
                           part ? id_qk_neg : id_qk, (part > 0 || ks > 0) ? 1u : 0u);
          }
        tc::commit(bar(kBarSFull + hf));
      };
      ok = mbar_wait(bar(kBarQFull), 0);
      tc::fence_after();
      for (int j = 0; ok && j < nt; ++j) {
        const int b = j & 1;
        for (int hf = 0; hf < halves; ++hf) {
          // the half's S/P buffer is free once PV(j - 1) is issued: MMAs from
          // this thread execute in order
          if (j >= 1 && !issue_pv(j - 1, hf)) { ok = false; break; }
          if (hf == 0 && !mbar_wait(bar(kBarKFull + b), (j >> 1) & 1)) { ok = false; break; }
          tc::fence_after();
          issue_qk(j, hf);
        }
        if (!ok) break;
        tc::commit(bar(kBarKEmpty + b));
        if (j >= 1) tc::commit(bar(kBarVEmpty + (b ^ 1)));
      }
      for (int hf = 0; ok && hf < halves; ++hf) {
        if (!issue_pv(nt - 1, hf)) { ok = false; break; }
        tc::commit(bar(kBarPvDone + hf));
      }
      // and its TMEM until its MMAs are done
      tc::commit(bar(kBarIdle));
      ok &= mbar_wait(bar(kBarIdle), 0);
    }
    ok = __all_sync(0xffffffffu, ok);
  } else if (warp < 6 || warp >= 14) {
    // ============================================================ dequant
    // q8: warps 0, 2, 3, 14: K (hi and lo parts), thread = one key row, D/2 channels;
    // warps 4, 15: V', thread = D / 64 channel rows of one scale group, all 64 keys.
    // fp8 / 4-bit, whose keys take a third of the work and whose values more: warps
    // 0, 2: K, thread = one key row; warps 4, 15, 3, 14: V', 32 keys a thread (two V'
    // warps took 1960 cycles a tile and set the pace).
    const bool k_side = F8 ? warp == 0 || warp == 2 : warp != 4 && warp != 15;
    const int t = (k_side ? (warp == 14 ? 3 : warp == 0 ? 0 : warp - 1)
                          : (warp == 4 ? 0 : warp == 15 ? 1 : warp == 3 ? 2 : 3)) * 32 +
                  lane;  // K: 0 .. 32 kKWarps - 1, V: 0 .. 32 kVWarps - 1
    constexpr int kChannels = 64 * D / (32 * C::kKWarps);  // of a K thread
    constexpr int kKeys = 64 * 64 / (32 * C::kVWarps);     // of a V' thread
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      const int sb = j % C::kSt, b = j & 1;
      if (!mbar_wait(bar(kBarStFull + sb), (j / C::kSt) & 1)) { ok = false; break; }
      const uint32_t st = smem_base + sb * L::kBytes;
      const int key0 = (t0 + j) * C::kTile;
      // keys at and past kv_end may hold stale bytes: converted as zeros
      const bool tail = key0 + C::kTile > kv_end;
      // K slot 1 and the V slots hold q until it is in TMEM
      if (j == (k_side ? 1 : 0) && !mbar_wait(bar(kBarQFull), 0)) { ok = false; break; }
      if (k_side) {
        if (j >= 2 && !mbar_wait(bar(kBarKEmpty + b), ((j - 2) >> 1) & 1)) { ok = false; break; }
        const uint32_t kdst = smem_base + C::kKOff + b * C::kKSlot;
        const int r = t & 63;
        const int c0 = (t >> 6) * kChannels;
        const bool dead = tail && key0 + r >= kv_end;
        if constexpr (F8) {
          // e4m3 -> fp16 exactly; a row outside the visible keys becomes zeros
#pragma unroll
          for (int c = c0; c < c0 + kChannels; c += 16) {
            const uint4 codes = dead ? make_uint4(0u, 0u, 0u, 0u) : lds128(st + L::k_off(r, c));
            const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
            uint32_t hw[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hw[2 * i] = e4m3x2_to_half2(cw[i]);
              hw[2 * i + 1] = e4m3x2_to_half2(cw[i] >> 16);
            }
            const int c16 = c / 8;
            sts128(kdst + tc::sw128_chunk(r, c16, 64), make_uint4(hw[0], hw[1], hw[2], hw[3]));
            sts128(kdst + tc::sw128_chunk(r, c16 + 1, 64), make_uint4(hw[4], hw[5], hw[6], hw[7]));
          }
        } else {
#pragma unroll
          for (int c = c0; c < c0 + kChannels; c += 16) {
            const uint4 codes = lds128(st + L::k_off(r, c));
            const uint32_t sbits = lds16(st + L::ks_off(r, c / 32));
            const uint32_t s2 = dead ? 0u : (sbits | (sbits << 16));
            const uint32_t ns2 = s2 ^ 0x80008000u;  // -scale
            uint32_t hw[8], lw[8];
            const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t lo, hi;
              codes4_to_half2(cw[i], lo, hi);
              // hi = fp16(code * s); lw = code * (-s) + hi = -lo (one rounding, exact);
              // the QK MMA of the lo part negates B, so it adds q . lo
              hw[2 * i] = hmul2_u32(lo, s2);
              hw[2 * i + 1] = hmul2_u32(hi, s2);
              asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(lw[2 * i]) : "r"(lo), "r"(ns2), "r"(hw[2 * i]));
              asm("fma.rn.f16x2 %0, %1, %2, %3;"
                  : "=r"(lw[2 * i + 1])
                  : "r"(hi), "r"(ns2), "r"(hw[2 * i + 1]));
            }
            const int c16 = c / 8;
            sts128(kdst + tc::sw128_chunk(r, c16, 64), make_uint4(hw[0], hw[1], hw[2], hw[3]));
            sts128(kdst + tc::sw128_chunk(r, c16 + 1, 64), make_uint4(hw[4], hw[5], hw[6], hw[7]));
            sts128(kdst + C::kKBytes + tc::sw128_chunk(r, c16, 64),
                   make_uint4(lw[0], lw[1], lw[2], lw[3]));
            sts128(kdst + C::kKBytes + tc::sw128_chunk(r, c16 + 1, 64),
                   make_uint4(lw[4], lw[5], lw[6], lw[7]));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarKFull + b));
          mbar_arrive(bar(kBarStEmpty + sb));
        }
      } else {
        if (j >= 2 && !mbar_wait(bar(kBarVEmpty + b), ((j - 2) >> 1) & 1)) { ok = false; break; }
        const uint32_t vrow = smem_base + C::kVOff + b * C::kVBytes;
        // D / 64 channel rows per thread, all in one scale group (for D = 128:
        // lanes 0-15 take channels 32w + lane and 32w + lane + 16), so the
        // per-key scales are loaded once for both rows
        constexpr int R = D / 64;
        int ch[R];
        if constexpr (R == 2) {
          ch[0] = ((t & 63) >> 4) * 32 + (t & 15);
          ch[1] = ch[0] + 16;
        } else {
          ch[0] = t & 63;
        }
        const int key_lo = (t >> 6) * kKeys;
        if constexpr (F8) {
#pragma unroll
          for (int key = key_lo; key < key_lo + kKeys; key += 16) {  // 16 keys: 8 bytes per channel row
            // the keys' scales and zeros, fp16 pairs (keys 2i, 2i+1); zero
            // outside the visible keys (stale bytes may sit there)
            const uint4 s01 = lds128(st + L::vs_off(key)), s23 = lds128(st + L::vs_off(key + 8));
            const uint4 z01 = lds128(st + L::vz_off(key)), z23 = lds128(st + L::vz_off(key + 8));
            uint32_t sc[8] = {s01.x, s01.y, s01.z, s01.w, s23.x, s23.y, s23.z, s23.w};
            uint32_t zr[8] = {z01.x, z01.y, z01.z, z01.w, z23.x, z23.y, z23.z, z23.w};
            if (tail) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int k0 = key0 + key + 2 * i;
                const uint32_t m = (k0 >= kv_end ? 0u : 0x0000ffffu) | (k0 + 1 >= kv_end ? 0u : 0xffff0000u);
                sc[i] &= m;
                zr[i] &= m;
              }
            }
#pragma unroll
            for (int rr = 0; rr < R; ++rr) {
              const uint2 nb = lds64(st + L::v_off(ch[rr], key));  // keys key .. key+15
              const uint32_t nw[4] = {nb.x, nb.x >> 16, nb.y, nb.y >> 16};
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t lo, hi;
                nibbles4_to_half2(nw[i], lo, hi);  // keys 4i, 4i+1 | 4i+2, 4i+3
                o[2 * i] = hfma2_u32(lo, sc[2 * i], zr[2 * i]);
                o[2 * i + 1] = hfma2_u32(hi, sc[2 * i + 1], zr[2 * i + 1]);
              }
              sts128(vrow + tc::sw128_chunk(ch[rr], key / 8, D), make_uint4(o[0], o[1], o[2], o[3]));
              sts128(vrow + tc::sw128_chunk(ch[rr], key / 8 + 1, D),
                     make_uint4(o[4], o[5], o[6], o[7]));
            }
          }
        } else {
          const int g = ch[0] / 32;
#pragma unroll
          for (int key = 0; key < C::kTile; key += 16) {  // 16 keys: one 16-byte load
            const uint4 s01 = lds128(st + L::vs_off(key, g));
            const uint4 s23 = lds128(st + L::vs_off(key + 8, g));
            uint32_t sc[8] = {s01.x, s01.y, s01.z, s01.w, s23.x, s23.y, s23.z, s23.w};
            if (tail) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int k0 = key0 + key + 2 * i;
                if (k0 >= kv_end) sc[i] &= 0xffff0000u;
                if (k0 + 1 >= kv_end) sc[i] &= 0x0000ffffu;
              }
            }
#pragma unroll
            for (int rr = 0; rr < R; ++rr) {
              const uint4 codes = lds128(st + L::v_off(ch[rr], key));
              uint32_t o[8];
              const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t lo, hi;
                codes4_to_half2(cw[i], lo, hi);
                o[2 * i] = hmul2_u32(lo, sc[2 * i]);
                o[2 * i + 1] = hmul2_u32(hi, sc[2 * i + 1]);
              }
              sts128(vrow + tc::sw128_chunk(ch[rr], key / 8, D), make_uint4(o[0], o[1], o[2], o[3]));
              sts128(vrow + tc::sw128_chunk(ch[rr], key / 8 + 1, D),
                     make_uint4(o[4], o[5], o[6], o[7]));
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarVFull + b));
          mbar_arrive(bar(kBarStEmpty + sb));
        }
      }
    }
  } else {
    // ============================================================ softmax
    const int hf = (warp - 6) >> 2;  // which 128-row half
    const int quarter = warp & 3;    // TMEM lanes this warp may access
    const int row = row0 + lane;
    const uint32_t t_lane = tmem + hf * C::kHalfCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool valid = row < n_rows;
    const float sl2 = a.scale_log2;
    // q row -> fp16 pairs in this lane's q columns (the QK MMA's A operand)
    {
      bool bad_q = false;
      cp_async_wait<0>();
      __syncwarp();
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb) {
        uint32_t qw[32];
#pragma unroll
        for (int c16 = 0; c16 < 8; ++c16) {
          const uint4 v = valid ? lds128(q_piece<D>(q_smem, lane, cb * 8 + c16)) : make_uint4(0u, 0u, 0u, 0u);
          qw[4 * c16 + 0] = pack_half2(bf16_lo(v.x), bf16_hi(v.x));
          qw[4 * c16 + 1] = pack_half2(bf16_lo(v.y), bf16_hi(v.y));
          qw[4 * c16 + 2] = pack_half2(bf16_lo(v.z), bf16_hi(v.z));
          qw[4 * c16 + 3] = pack_half2(bf16_lo(v.w), bf16_hi(v.w));
          bad_q |= half2_nonfinite(qw[4 * c16]) || half2_nonfinite(qw[4 * c16 + 1]) ||
                   half2_nonfinite(qw[4 * c16 + 2]) || half2_nonfinite(qw[4 * c16 + 3]);
        }
        tc::st32(t_lane + C::kQCol + cb * 32, qw);
      }
      // q values beyond the fp16 range (|q| >= 65520) would give inf scores
      if (__any_sync(0xffffffffu, bad_q) && lane == 0) flag_status(a.status, PA_DEV_BAD_Q);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQFull));
    }
    float m_used = -INFINITY;  // max the accumulator is scaled to (log2 units)
    float l = 0.0f;
    if (hf < halves) {
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        if (!mbar_wait(bar(kBarSFull + hf), j & 1)) { ok = false; break; }
        tc::fence_after();
        const int key0 = (t0 + j) * C::kTile;
        const bool need_mask = key0 + C::kTile > kv_end;  // the same for every row
        uint32_t sr[64];
        // S from TMEM; masked columns -> -inf, the rest pre-scaled (only on
        // the tile that holds the prefix's end)
        auto load_s = [&]() {
          tc::ld32(t_lane, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tc::ld32(t_lane + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tc::wait_loaded(*reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tc::wait_loaded(*reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          if (need_mask) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              sr[c] = __float_as_uint(key0 + c >= kv_end ? -INFINITY
                                                                         : __uint_as_float(sr[c]) * sl2);
          }
        };
        load_s();
        const float mul = need_mask ? 1.0f : sl2;
        // P = 2^(s * scale - m_used) as fp16 pairs and their fp32 sum; pairs
        // of columns go through the packed fp32 FMA and add
        uint32_t pw[32];
        float ts;
        auto exp_tile = [&]() {
          // no visible key yet (m_used = -inf): every column of this tile is
          // masked or the slow path below takes it, so any finite offset works
          const float neg_m = m_used == -INFINITY ? 0.0f : -m_used;
          const uint64_t mul2 = f32x2_pack(mul, mul), neg_m2 = f32x2_pack(neg_m, neg_m);
          uint64_t ls2[4] = {0, 0, 0, 0};  // +0.0f pairs
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float t0, t1;
            f32x2_unpack(f32x2_fma(f32x2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), mul2,
                                   neg_m2),
                         t0, t1);
            const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
            ls2[(c >> 1) & 3] = f32x2_add(ls2[(c >> 1) & 3], f32x2_pack(p0, p1));
            pw[c >> 1] = pack_half2(p0, p1);
          }
          float ls[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) f32x2_unpack(ls2[k], ls[2 * k], ls[2 * k + 1]);
          ts = ((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7]));
        };
        // The max the accumulator is scaled to moves only when this tile's
        // P would exceed C::kMaxTileSum (2^15, inside fp16): no row max is
        // taken on the common path.  A row with no max yet (m_used = -inf)
        // always takes the slow path, which sets it once a key is visible.
        exp_tile();
        const bool grow = !(ts <= C::kMaxTileSum) || m_used == -INFINITY;
        if (__any_sync(0xffffffffu, grow)) {
          float f = 1.0f;  // factor for what O and l hold
          load_s();        // S is still in TMEM (P not yet written)
          if (grow) {
            float e[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 64; ++c) e[c & 3] = fmaxf(e[c & 3], __uint_as_float(sr[c]) * mul);
            const float m_new = fmaxf(m_used, fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])));
            if (m_new > -INFINITY) {  // else nothing visible yet: P stays 0
              f = fast_exp2(m_used - m_new);  // 0 when the row had no max
              l *= f;
              m_used = m_new;
            }
          }
          exp_tile();
          if (j > 0) {
            // O holds tiles < j (PV(j - 1) completed before S(j) was
            // committed): scale it in TMEM
#pragma unroll 1
            for (int cb = 0; cb < D / 32; ++cb) {
              uint32_t orr[32];
              tc::ld32(t_lane + C::kOCol + cb * 32, orr);
              tc::wait_loaded(orr);
#pragma unroll
              for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * f);
              tc::st32(t_lane + C::kOCol + cb * 32, orr);
            }
            tc::wait_st();
          }
        }
        l += ts;
        tc::st32(t_lane, pw);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + hf));
      }
      // ---- epilogue: the row's triple
      if (ok && mbar_wait(bar(kBarPvDone + hf), 0)) {
        tc::fence_after();
        const int64_t r = static_cast<int64_t>(w.q0) * a.qpk + row, step = rows_total(sa) * 4;
        float *dst = acc_at<D>(sa, w.slot, h) + r * 4;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t orr[32];
          tc::ld32(t_lane + C::kOCol + cb * 32, orr);
          tc::wait_loaded(orr);
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4 *>(dst + (cb * 8 + i / 4) * step) =
                  make_uint4(orr[i], orr[i + 1], orr[i + 2], orr[i + 3]);
          }
        }
        if (valid)
          *reinterpret_cast<float2 *>(a.part_ml + (ml_at(sa, w.slot, h) + r) * 2) =
              make_float2(m_used, l);
      } else {
        ok = false;
      }
    }
  }
  if (!ok && lane == 0) flag_status(a.status, PA_DEV_TIMEOUT);

  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int BS, bool F8>
static cudaError_t launch_shared_tc_t(const SharedArgs &s, const CUtensorMap &tk,
                                      const CUtensorMap &tv, cudaStream_t stream) {
  using C = SharedTcCfg<D, BS, F8>;
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    return cudaFuncSetAttribute(shared_tc_kernel<D, BS, F8>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemOfSm);
  });
  if (e != cudaSuccess) return e;
  const int64_t gx = static_cast<int64_t>(s.n_pblocks) * s.ns_p * s.a.hk;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx));
  return launch_kernel(shared_tc_kernel<D, BS, F8>, grid, C::kWarps * 32, kSmemOfSm, stream, s,
                       tk, tv);
}

// Rows of one block, 0 where the kernel does not take the head size.
int shared_tc_rows(int d) { return d == 64 || d == 128 ? 256 : d == 256 ? 128 : 0; }

cudaError_t launch_shared_tc256(const SharedArgs &s, const CUtensorMap &tk, const CUtensorMap &tv, int bs,
                                bool f8v4, cudaStream_t stream);  // attn_shared_tc256.cu

cudaError_t launch_shared_tc(const SharedArgs &s, const CUtensorMap &tk, const CUtensorMap &tv,
                             int d, int bs, bool f8v4, cudaStream_t stream) {
#define PAQ8_TC_CASE(DD, BB)                                              \
  if (d == DD && bs == BB)                                                \
    return f8v4 ? launch_shared_tc_t<DD, BB, true>(s, tk, tv, stream)     \
                : launch_shared_tc_t<DD, BB, false>(s, tk, tv, stream);
  PAQ8_TC_CASE(64, 16)
  PAQ8_TC_CASE(64, 32)
  PAQ8_TC_CASE(128, 16)
  PAQ8_TC_CASE(128, 32)
  if (d == 256) return launch_shared_tc256(s, tk, tv, bs, f8v4, stream);
#undef PAQ8_TC_CASE
  return cudaErrorInvalidValue;
}

}  // namespace paq8
