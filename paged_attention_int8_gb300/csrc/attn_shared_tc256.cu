// Attention over a shared prefix on the 5th-generation tensor cores (tcgen05,
// TMEM): the prefix items of attn_shared.cuh for D = 256.
//
// One block = 128 rows (128 / qpk query tokens of one group x the qpk q heads
// of one kv head) x one key segment, in 64-key tiles.  The arithmetic is that
// of attn_shared_tc.cu; what D = 256 changes is the room: O takes 256 of TMEM's
// 512 columns and q 128, which leaves two 64-column S / P buffers for one
// 128-row half, and one tile's key operand (hi and lo parts, 32 KB each) is
// half of shared memory.  So instead of two halves the pipeline alternates the
// S buffers of one: QK(j + 1) runs while the softmax works on S(j), then PV(j).
//   tensor core, a tile: 2 x 16 MMAs of N = 64 and 4 of N = 256, 1536 cycles;
//   softmax, one row per thread, hidden behind QK(j + 1) and PV(j - 1);
//   shared memory: 34 KB staged, read and turned into 96 KB of operands that the
//   MMAs read once, 2060 cycles at 128 bytes each.
// A tile takes 2650 cycles: bound by shared memory and the conversions.
// Operand buffers: three 32 KB slots that hold the key parts hi(0), lo(0), hi(1),
// ... in turn, each freed when its own MMAs are done, and one value slot; pages
// are staged by TMA in rings of their own for keys (2) and for values (3).
// Warps: 5 and 18 producers, 1 MMA issuer; keys 0, 2, 3, 6, 14 - 17; values 4, 7, 12, 13;
// softmax 8 - 11 (one per TMEM lane quarter).  fp8 / 4-bit: keys are exact in one
// part.  What a converter can do before its slot is free it does (the keys' codes
// and half of the values in registers): waiting first took 3200 cycles a tile, with
// four key warps 4300.
#include <type_traits>

#include "attn_shared.cuh"
#include "tcgen05.cuh"

namespace paq8 {

namespace {

constexpr int kD = 256;

template <int BS, bool F8>
struct Tc256Cfg {
  static constexpr int kTile = 64;
  static constexpr int kStK = 2, kStV = 3;  // staging stages of the rings
  static constexpr int kWarps = 19;
  static constexpr int kKWarps = 8;
  static constexpr int kParts = F8 ? 1 : 2;  // key parts: hi, lo
  static constexpr int G = kD / 32;
  static constexpr int kPages = kTile / BS;
  // staged keys: codes [64][256] as two 128-byte halves, then scales [64][G]
  static constexpr int kKStage = kTile * kD + (F8 ? 0 : kTile * G * 2);
  // staged values: pages [256][BS] (nibbles: [256][BS / 2]), then scales (and zeros)
  static constexpr int kVCodes = F8 ? kTile * kD / 2 : kTile * kD;
  static constexpr int kVStage = kVCodes + (F8 ? 1024 : kTile * G * 2);
  static constexpr int kPartBytes = kTile * kD * 2;  // [D/64][64 keys][128 B]
  static constexpr int kVBytes = kD * kTile * 2;     // [256 rows][64 keys]
  static constexpr int kPartOff = 0;
  static constexpr int kVOff = 3 * kPartBytes;
  static constexpr int kStKOff = kVOff + kVBytes;
  static constexpr int kStVOff = kStKOff + kStK * kKStage;
  static constexpr int kBarOff = (kStVOff + kStV * kVStage + 1023) / 1024 * 1024;
  static constexpr int kSmem = kBarOff + 256 + 1024;
  static constexpr uint32_t kOCol = 0, kQCol = 256, kSCol = 384;
  static constexpr float kMaxTileSum = 32768.0f;  // bound on a tile's P sum (so on every P)
  static_assert(kSmem <= 232448 && kKStage % 1024 == 0 && kVStage % 1024 == 0, "shared memory");
};

// barriers (8 bytes each, from kBarOff)
enum : int {
  kStKFull = 0,    // [2] producer -> K dequant (tx bytes)
  kStKEmpty = 2,   // [2] K dequant -> producer (8 warps)
  kStVFull = 4,    // [3] producer -> V dequant
  kStVEmpty = 7,   // [3] V dequant -> producer (4 warps)
  kPartFull = 10,  // [3] K dequant -> MMA (8 warps)
  kPartEmpty = 13, // [3] commit after the part's MMAs -> K dequant
  kVFull = 16,     // V dequant -> MMA (4 warps)
  kPvDone = 17,    // commit after PV -> V dequant, softmax
  kSFull = 18,     // [2] commit after QK -> softmax
  kPFull = 20,     // [2] softmax (P in TMEM) -> MMA (4 warps)
  kQFull = 22,     // softmax (q in TMEM) -> MMA (4 warps)
  kAllDone = 23,   // commit after the last PV -> softmax (PvDone may be two phases off there)
  kIdle = 24,      // commit after the last MMA issued -> MMA issuer
  kBars = 25
};

template <int BS, bool F8>
// 19 warps, five on three of the SM sub-partitions: 96 registers at most
__global__ void __maxnreg__(96)
    shared_tc256_kernel(const __grid_constant__ SharedArgs sa, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v) {
  using C = Tc256Cfg<BS, F8>;
  constexpr int D = kD;
  constexpr int G = C::G;
  using L = std::conditional_t<F8, StageF8V4<D, BS, C::kTile>, StageLayout<D, BS, C::kTile>>;
  const AttnArgs &a = sa.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (smem_base - smem_u32(smem_raw));

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(sa.a.hk));

  if (threadIdx.x == 5 * 32) prefetch_tensormap(&tmap_k);
  if constexpr (!F8) {
    if (threadIdx.x == 18 * 32) prefetch_tensormap(&tmap_v);
  }
  wait_for_predecessor();
  launch_dependents();
  SharedWork w;
  if (!prefix_work(sa, static_cast<int>(blockIdx.x / static_cast<unsigned>(a.hk)), a.block_q, lane, w))
    return;
  const int n_rows = w.n_tok * a.qpk;
  // the softmax warps' 32 rows of q each, in flight during the set-up: they stand
  // in part slot 2 and the value slot until they are in TMEM
  const int row0 = (warp & 3) * 32;
  const uint32_t q_smem = smem_base + C::kPartOff + 2 * C::kPartBytes + row0 * (2 * D);
  if (warp >= 8 && warp < 12) copy_q_rows<D>(a, q_smem, w.q0, h, row0, n_rows, lane);
  const int kv_end = w.kv_end;  // kv_begin starts a tile
  const int t0 = w.kv_begin / C::kTile;
  const int nt = (kv_end + C::kTile - 1) / C::kTile - t0;

  const uint32_t bars = smem_base + C::kBarOff;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t tmem_slot = bars + 8 * kBars;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStK; ++i) {
      mbar_init(bar(kStKFull + i), 1);
      mbar_init(bar(kStKEmpty + i), C::kKWarps);
    }
    for (int i = 0; i < C::kStV; ++i) {
      mbar_init(bar(kStVFull + i), 1);
      mbar_init(bar(kStVEmpty + i), 4);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(kPartFull + i), C::kKWarps);
      mbar_init(bar(kPartEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kPFull + i), 4);
    }
    mbar_init(bar(kVFull), 4);
    mbar_init(bar(kPvDone), 1);
    mbar_init(bar(kQFull), 4);
    mbar_init(bar(kAllDone), 1);
    mbar_init(bar(kIdle), 1);
    fence_barrier_init();
  }
  if (warp == 1) tc::alloc(tmem_slot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + C::kBarOff + 8 * kBars);
  bool ok = true;

  if (warp == 5 || warp == 18) {
    // ============================================================ producers
    // One warp stages the keys, one the values: the values' ring is the shorter one
    // and follows PV, and one warp in order for both held the keys back to it.
    // Block-table entries are read 32 pages at a time, one per lane; pages at or
    // past the prefix's end are not staged.
    const bool keys = warp == 5;
    const int n_st = keys ? C::kStK : C::kStV;
    const int full0 = keys ? kStKFull : kStVFull, empty0 = keys ? kStKEmpty : kStVEmpty;
    const int n_pages = (kv_end + BS - 1) / BS;
    const int32_t *bt_row = a.block_table + static_cast<int64_t>(w.row) * a.bt_stride;
    int page_base = -(1 << 30), my_blk = -1;
    int st = 0, phase = 1;  // stage of the ring and the parity of its being empty
    int j = 0;
    for (; ok && j < nt; ++j) {
      if (j >= n_st) {
        int there = 1;
        if (lane == 0) there = mbar_wait(bar(empty0 + st), phase);
        if (!__shfl_sync(0xffffffffu, there, 0)) { ok = false; break; }
      }
      const int lp0 = (t0 + j) * C::kPages;
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
      // a lane per page and copy: keys two boxes and scales, values codes, scales, zeros
      const int my_page = lane >> 2, what = lane & 3;
      const int blk = __shfl_sync(0xffffffffu, my_blk, lp0 + min(my_page, C::kPages - 1) - page_base);
      const bool mine = my_page < C::kPages && blk >= 0;
      const int n_valid = __popc(__ballot_sync(0xffffffffu, mine && what == 0));
      constexpr uint32_t kVPage = F8 ? D * BS / 2 : D * BS;
      const uint32_t full = bar(full0 + st);
      if (lane == 0)
        mbar_arrive_expect_tx(full, n_valid * (keys ? BS * D + (F8 ? 0 : BS * G * 2)
                                                    : kVPage + (F8 ? 4 * BS : BS * G * 2)));
      __syncwarp();
      if (mine) {
        const int64_t page = static_cast<int64_t>(blk) * a.hk + h;
        if (keys) {
          const uint32_t sk = smem_base + C::kStKOff + st * C::kKStage;
          if (what < 2)
            tma_load_2d(sk + what * (C::kTile * 128) + my_page * (BS * 128), &tmap_k, what * 128,
                        static_cast<int32_t>(page * BS), full);
          if constexpr (!F8) {
            if (what == 2)
              bulk_load(sk + C::kTile * D + my_page * (BS * G * 2), a.k_scale + page * BS * G, BS * G * 2, full);
          }
        } else {
          const uint32_t sv = smem_base + C::kStVOff + st * C::kVStage;
          if constexpr (F8) {
            if (what == 0)
              bulk_load(sv + my_page * kVPage, reinterpret_cast<const uint8_t *>(a.v_cache) + page * kVPage,
                        kVPage, full);
            if (what == 1)
              bulk_load(sv + C::kVCodes + my_page * (BS * 2), a.v_scale + page * BS, BS * 2, full);
            if (what == 2)
              bulk_load(sv + C::kVCodes + C::kTile * 2 + my_page * (BS * 2), a.v_zero + page * BS, BS * 2, full);
          } else {
            if (what == 0)
              tma_load_2d(sv + my_page * kVPage, &tmap_v, 0, static_cast<int32_t>(page * D), full);
            if (what == 1)
              bulk_load(sv + C::kVCodes + my_page * (BS * G * 2), a.v_scale + page * BS * G, BS * G * 2, full);
          }
        }
      }
      if (++st == n_st) {
        st = 0;
        phase ^= 1;
      }
      __syncwarp();
    }
    // the block holds its shared memory until its copies have landed, whoever gave up
    for (int i = max(0, j - n_st); lane == 0 && i < j; ++i)
      ok &= mbar_wait(bar(full0 + i % n_st), (i / n_st) & 1);
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    // one elected lane (attn_shared_tc.cu)
    if (tc::elect_one()) {
      constexpr uint32_t id_qk = tc::idesc_f16(128, 64);
      constexpr uint32_t id_qk_neg = id_qk | (1u << 14);  // negate B: K_lo is stored as -lo
      constexpr uint32_t id_pv = tc::idesc_f16(128, D);
      const uint64_t part_desc = tc::desc_sw128(smem_base + C::kPartOff);
      const uint64_t v_desc = tc::desc_sw128(smem_base + C::kVOff);
      uint32_t slot = 0, phase = 0;  // of the next key part
      // S(j) = q K_hi(j)^T - q (-K_lo(j))^T into buffer j % 2, whose P(j - 2) is
      // consumed: PV(j - 2) was issued before, and MMAs execute in order
      auto issue_qk = [&](int j) -> bool {
        const uint32_t s_col = tmem + C::kSCol + (j & 1) * 64;
#pragma unroll 1
        for (int part = 0; part < C::kParts; ++part) {
          if (!mbar_wait(bar(kPartFull + slot), phase)) return false;
          tc::fence_after();
          const uint64_t desc = part_desc + slot * (C::kPartBytes >> 4);
          const uint32_t id = part ? id_qk_neg : id_qk;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc::mma_f16_ts(s_col, tmem + C::kQCol + ks * 8,
                           desc + (((ks >> 2) * (64 * 128) + (ks & 3) * 32) >> 4), id,
                           ks > 0 ? 1u : static_cast<uint32_t>(part));
          tc::commit(bar(kPartEmpty + slot));
          if (++slot == 3) {
            slot = 0;
            phase ^= 1;
          }
        }
        tc::commit(bar(kSFull + (j & 1)));
        return true;
      };
      ok = mbar_wait(bar(kQFull), 0);
      tc::fence_after();
      ok = ok && issue_qk(0);
#pragma unroll 1
      for (int j = 0; ok && j < nt; ++j) {
        if (j + 1 < nt && !issue_qk(j + 1)) { ok = false; break; }
        // O += P(j) V'(j)
        if (!mbar_wait(bar(kVFull), j & 1) || !mbar_wait(bar(kPFull + (j & 1)), (j >> 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after();
        const uint32_t p_col = tmem + C::kSCol + (j & 1) * 64;
#pragma unroll
        for (int ks = 0; ks < C::kTile / 16; ++ks)
          tc::mma_f16_ts(tmem + C::kOCol, p_col + ks * 8, v_desc + 2 * ks, id_pv,
                         (j > 0 || ks > 0) ? 1u : 0u);
        tc::commit(bar(kPvDone));
      }
      if (ok) tc::commit(bar(kAllDone));
      // the block holds its TMEM until its MMAs are done
      tc::commit(bar(kIdle));
      ok &= mbar_wait(bar(kIdle), 0);
    }
    ok = __all_sync(0xffffffffu, ok);
  } else if (warp == 0 || warp == 2 || warp == 3 || warp == 6 || (warp >= 14 && warp < 18)) {
    // ============================================================ K dequant
    // thread = one key row, 64 channels (two scale groups).  The codes are held in
    // registers: the hi part goes into a slot while the tensor core still reads both
    // parts of the tile before, the lo part into the next slot that it lets go.
    const int t = (warp >= 14 ? warp - 10 : warp == 6 ? 3 : warp == 0 ? 0 : warp - 1) * 32 + lane;
    const int r = t & 63;
    const int c0 = (t >> 6) * 64;
    uint32_t slot = 0, phase = 1;  // of the next part: the first round's slots are free
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      const int kb = j % C::kStK;
      if (j == 1 && !mbar_wait(bar(kQFull), 0)) { ok = false; break; }  // q is out of slot 2
      if (!mbar_wait(bar(kStKFull + kb), (j / C::kStK) & 1)) { ok = false; break; }
      const uint32_t st = smem_base + C::kStKOff + kb * C::kKStage;
      // keys at and past the prefix's end may hold stale bytes: converted as zeros
      const bool dead = (t0 + j) * C::kTile + r >= kv_end;
      const uint32_t scales = F8 || dead ? 0u : lds32(st + C::kTile * D + (r * G + c0 / 32) * 2);
      uint4 codes[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) codes[i] = lds128(st + L::k_off(r, c0 + 16 * i));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kStKEmpty + kb));
#pragma unroll 1
      for (int part = 0; part < C::kParts; ++part) {
        if (!mbar_wait(bar(kPartEmpty + slot), phase)) { ok = false; break; }
        const uint32_t dst = smem_base + C::kPartOff + slot * C::kPartBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + 16 * i;
          const uint32_t cw[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
          uint32_t o[8];
          if constexpr (F8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = dead ? 0u : e4m3x2_to_half2(cw[k]);
              o[2 * k + 1] = dead ? 0u : e4m3x2_to_half2(cw[k] >> 16);
            }
          } else {
            const uint32_t s2 = __byte_perm(scales, 0u, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t lo, hi;
              codes4_to_half2(cw[k], lo, hi);
              // hi part fp16(code * s); second part code * (-s) + hi = -lo, exact
              o[2 * k] = hmul2_u32(lo, s2);
              o[2 * k + 1] = hmul2_u32(hi, s2);
              if (part) {
                o[2 * k] = hfma2_u32(lo, s2 ^ 0x80008000u, o[2 * k]);
                o[2 * k + 1] = hfma2_u32(hi, s2 ^ 0x80008000u, o[2 * k + 1]);
              }
            }
          }
          sts128(dst + tc::sw128_chunk(r, c / 8, 64), make_uint4(o[0], o[1], o[2], o[3]));
          sts128(dst + tc::sw128_chunk(r, c / 8 + 1, 64), make_uint4(o[4], o[5], o[6], o[7]));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPartFull + slot));
        if (++slot == 3) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
    }
  } else if (warp == 4 || warp == 7 || warp == 12 || warp == 13) {
    // ============================================================ V dequant
    // thread = two channel rows of one scale group, all 64 keys.  The slot is single:
    // the first 32 keys are converted while the tensor core still reads the values of
    // the tile before, and wait in registers.
    const int t = (warp == 4 ? 0 : warp == 7 ? 1 : warp - 10) * 32 + lane;
    const int ch[2] = {(t >> 4) * 32 + (t & 15), (t >> 4) * 32 + (t & 15) + 16};
    const int g = t >> 4;
    const uint32_t vrow = smem_base + C::kVOff;
    int sb = 0, st_phase = 0;
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      if (!mbar_wait(bar(kStVFull + sb), st_phase)) { ok = false; break; }
      const uint32_t st = smem_base + C::kStVOff + sb * C::kVStage;
      const int key0 = (t0 + j) * C::kTile;
      const bool tail = key0 + C::kTile > kv_end;
      // 16 keys from `key` on of both rows, as fp16 pairs
      auto convert = [&](int key, uint32_t (&o)[2][8]) {
        uint32_t sc[8], zr[8];
        {
          // the 16 keys' scales (of this channel group; fp8 / 4-bit: of the key)
          const uint32_t at = F8 ? st + C::kVCodes + key * 2
                                 : st + C::kVCodes + ((key / BS) * (G * BS) + g * BS + key % BS) * 2;
          const uint4 s01 = lds128(at), s23 = lds128(at + 16);
          sc[0] = s01.x, sc[1] = s01.y, sc[2] = s01.z, sc[3] = s01.w;
          sc[4] = s23.x, sc[5] = s23.y, sc[6] = s23.z, sc[7] = s23.w;
          if constexpr (F8) {
            const uint4 z01 = lds128(at + C::kTile * 2), z23 = lds128(at + C::kTile * 2 + 16);
            zr[0] = z01.x, zr[1] = z01.y, zr[2] = z01.z, zr[3] = z01.w;
            zr[4] = z23.x, zr[5] = z23.y, zr[6] = z23.z, zr[7] = z23.w;
          }
        }
        if (tail) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int k0 = key0 + key + 2 * i;
            const uint32_t m = (k0 >= kv_end ? 0u : 0x0000ffffu) | (k0 + 1 >= kv_end ? 0u : 0xffff0000u);
            sc[i] &= m;
            if constexpr (F8) zr[i] &= m;
          }
        }
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          if constexpr (F8) {
            const uint2 nb = lds64(st + (key / BS) * (D * BS / 2) + ch[rr] * (BS / 2) + (key % BS) / 2);
            const uint32_t nw[4] = {nb.x, nb.x >> 16, nb.y, nb.y >> 16};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t lo, hi;
              nibbles4_to_half2(nw[i], lo, hi);
              o[rr][2 * i] = hfma2_u32(lo, sc[2 * i], zr[2 * i]);
              o[rr][2 * i + 1] = hfma2_u32(hi, sc[2 * i + 1], zr[2 * i + 1]);
            }
          } else {
            const uint4 codes = lds128(st + L::v_off(ch[rr], key) - L::kVOff);
            const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t lo, hi;
              codes4_to_half2(cw[i], lo, hi);
              o[rr][2 * i] = hmul2_u32(lo, sc[2 * i]);
              o[rr][2 * i + 1] = hmul2_u32(hi, sc[2 * i + 1]);
            }
          }
        }
      };
      auto put = [&](int key, const uint32_t (&o)[2][8]) {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          sts128(vrow + tc::sw128_chunk(ch[rr], key / 8, D), make_uint4(o[rr][0], o[rr][1], o[rr][2], o[rr][3]));
          sts128(vrow + tc::sw128_chunk(ch[rr], key / 8 + 1, D),
                 make_uint4(o[rr][4], o[rr][5], o[rr][6], o[rr][7]));
        }
      };
      uint32_t early[2][2][8];
      convert(0, early[0]);
      convert(16, early[1]);
      // the slot is free once q is in TMEM, then with each PV
      if (!mbar_wait(bar(j >= 1 ? kPvDone : kQFull), j >= 1 ? (j - 1) & 1 : 0)) { ok = false; break; }
      put(0, early[0]);
      put(16, early[1]);
#pragma unroll
      for (int key = 32; key < C::kTile; key += 16) {
        uint32_t o[2][8];
        convert(key, o);
        put(key, o);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kVFull));
        mbar_arrive(bar(kStVEmpty + sb));
      }
      if (++sb == C::kStV) {
        sb = 0;
        st_phase ^= 1;
      }
    }
  } else {
    // ============================================================ softmax
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const bool valid = row0 + lane < n_rows;
    const float sl2 = a.scale_log2;
    // q row -> fp16 pairs in this lane's q columns (the QK MMA's A operand)
    {
      bool bad_q = false;
      cp_async_wait<0>();
      __syncwarp();
#pragma unroll 1
      for (int cb = 0; cb < D / 64; ++cb) {
        uint32_t qw[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = valid ? lds128(q_piece<D>(q_smem, lane, cb * 8 + c)) : make_uint4(0u, 0u, 0u, 0u);
          qw[4 * c + 0] = pack_half2(bf16_lo(v.x), bf16_hi(v.x));
          qw[4 * c + 1] = pack_half2(bf16_lo(v.y), bf16_hi(v.y));
          qw[4 * c + 2] = pack_half2(bf16_lo(v.z), bf16_hi(v.z));
          qw[4 * c + 3] = pack_half2(bf16_lo(v.w), bf16_hi(v.w));
          bad_q |= half2_nonfinite(qw[4 * c]) || half2_nonfinite(qw[4 * c + 1]) ||
                   half2_nonfinite(qw[4 * c + 2]) || half2_nonfinite(qw[4 * c + 3]);
        }
        tc::st32(t_lane + C::kQCol + cb * 32, qw);
      }
      // q values beyond the fp16 range (|q| >= 65520) would give inf scores
      if (__any_sync(0xffffffffu, bad_q) && lane == 0) flag_status(a.status, PA_DEV_BAD_Q);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));
    }
    float m_used = -INFINITY;  // max the accumulator is scaled to (log2 units)
    float l = 0.0f;
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(kSFull + (j & 1)), (j >> 1) & 1))) { ok = false; break; }
      tc::fence_after();
      const uint32_t t_s = t_lane + C::kSCol + (j & 1) * 64;
      const int key0 = (t0 + j) * C::kTile;
      const bool need_mask = key0 + C::kTile > kv_end;  // the same for every row
      uint32_t sr[64];
      // S from TMEM; masked columns -> -inf, the rest pre-scaled (only on
      // the tile that holds the prefix's end)
      auto load_s = [&]() {
        tc::ld32(t_s, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tc::ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tc::wait_ld();
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
          // O holds tiles < j once PV(j - 1) is done (it may still run: S(j) was
          // issued before it): scale it in TMEM
          if (!__all_sync(0xffffffffu, mbar_wait(bar(kPvDone), (j - 1) & 1))) { ok = false; break; }
          tc::fence_after();
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t orr[32];
            tc::ld32(t_lane + C::kOCol + cb * 32, orr);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * f);
            tc::st32(t_lane + C::kOCol + cb * 32, orr);
          }
          tc::wait_st();
        }
      }
      l += ts;
      tc::st32(t_s, pw);
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPFull + (j & 1)));
    }
    // ---- epilogue: the row's triple
    if (ok && __all_sync(0xffffffffu, mbar_wait(bar(kAllDone), 0))) {
      tc::fence_after();
      const int64_t r = static_cast<int64_t>(w.q0) * a.qpk + row0 + lane, step = rows_total(sa) * 4;
      float *dst = acc_at<D>(sa, w.slot, h) + r * 4;
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t orr[32];
        tc::ld32(t_lane + C::kOCol + cb * 32, orr);
        tc::wait_ld();
        if (valid) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4 *>(dst + (cb * 8 + i / 4) * step) =
                make_uint4(orr[i], orr[i + 1], orr[i + 2], orr[i + 3]);
        }
      }
      if (valid)
        *reinterpret_cast<float2 *>(a.part_ml + (ml_at(sa, w.slot, h) + r) * 2) = make_float2(m_used, l);
    } else {
      ok = false;
    }
  }
  if (!ok && lane == 0) flag_status(a.status, PA_DEV_TIMEOUT);

  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int BS, bool F8>
cudaError_t launch_shared_tc256_t(const SharedArgs &s, const CUtensorMap &tk, const CUtensorMap &tv,
                                  cudaStream_t stream) {
  using C = Tc256Cfg<BS, F8>;
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    return cudaFuncSetAttribute(shared_tc256_kernel<BS, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t gx = static_cast<int64_t>(s.n_pblocks) * s.ns_p * s.a.hk;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_kernel(shared_tc256_kernel<BS, F8>, dim3(static_cast<unsigned>(gx)), C::kWarps * 32,
                       C::kSmem, stream, s, tk, tv);
}

}  // namespace

cudaError_t launch_shared_tc256(const SharedArgs &s, const CUtensorMap &tk, const CUtensorMap &tv, int bs,
                                bool f8v4, cudaStream_t stream) {
  if (bs == 16)
    return f8v4 ? launch_shared_tc256_t<16, true>(s, tk, tv, stream)
                : launch_shared_tc256_t<16, false>(s, tk, tv, stream);
  return f8v4 ? launch_shared_tc256_t<32, true>(s, tk, tv, stream)
              : launch_shared_tc256_t<32, false>(s, tk, tv, stream);
}

}  // namespace paq8
