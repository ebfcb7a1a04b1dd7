// Attention of a batch whose groups of sequences share a prefix: the row-tile
// kernel on warp MMAs, the join of the segments, and the dispatch.
// attn_shared.cuh states the decomposition.
//
// shared_mma_kernel: one item segment per block -- 64 / qpk query tokens x the
// qpk q heads of one kv head, up to 64 rows -- in the form of the generic
// attention kernel (attn_prefill.cu): warp 4 stages each 64-key tile's pages
// through a 4-deep mbarrier ring (16-byte cp.async copies); warps 0-3 take the
// rows in groups of 16 (R groups; the 4/R warps that share a group alternate
// tiles with private softmax states, merged at the end).  q8: QK^T on the
// exact integer codes (fp16) per 32-channel group, scaled by the group's fp16
// K scale in fp32; PV multiplies P (fp16) by V' = code * scale (fp16, one
// rounding).  fp8 / 4-bit: one QK accumulation of the exact keys, V' = idx *
// scale + zero in one fp16 FMA.  Sums, maxima and accumulators are fp32.
// A prefix of P keys costs ceil(rows / 64) reads of its pages (L2 serves all
// but the first), not one per sequence.
#include <algorithm>
#include <type_traits>

#include "attn_shared.cuh"

namespace paq8 {

cudaError_t launch_shared_rows(const SharedArgs &s, int d, int bs, bool f8v4, cudaStream_t stream);
cudaError_t launch_shared_tc(const SharedArgs &s, const CUtensorMap &tk, const CUtensorMap &tv,
                             int d, int bs, bool f8v4, cudaStream_t stream);
int shared_tc_rows(int d);

constexpr int kTile = kSegTile;
constexpr int kRowTile = 64;  // rows of one block of shared_mma_kernel

template <int D, int BS, bool F8>
struct SharedMmaCfg {
  using L = std::conditional_t<F8, StageF8V4<D, BS, kTile>, StageLayout<D, BS, kTile>>;
  static constexpr int G = D / 32;
  static constexpr int kQBytes = 4 * G * 2 * 32 * 16;  // fragment-ordered q, 4 row groups
  static constexpr int kQOff = kStages * L::kBytes;
  static constexpr int kBarOff = kQOff + kQBytes;
  static constexpr int kSmemBytes = kBarOff + 2 * kStages * 8 + 1024;  // + alignment slack
  // merge area (inside the stages) per partner warp: m0 m1 l0 l1 + O
  static constexpr int kMergeFields = 4 + 4 * 4 * G;
  static_assert(3 * kMergeFields * 32 * 4 <= kStages * L::kBytes, "merge area");
};

template <int D, int BS, bool F8>
__global__ void __launch_bounds__(kThreads) shared_mma_kernel(const __grid_constant__ SharedArgs s) {
  using C = SharedMmaCfg<D, BS, F8>;
  using L = typename C::L;
  constexpr int G = C::G;
  const AttnArgs &a = s.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (smem_base - smem_u32(smem_raw));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y;  // kv head
  if (s.first) wait_for_predecessor();
  launch_dependents();
  const LastBlockWaits at_end{blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1};

  // ---- which rows, which keys: prefix items first, segment-major
  SharedWork w;
  const int n_prefix = s.n_pblocks * s.ns_p;
  const int bx = static_cast<int>(blockIdx.x);
  if (bx < n_prefix) {
    if (!prefix_work(s, bx, a.block_q, lane, w)) return;
  } else {
    const int r = bx - n_prefix;
    if (!suffix_work(s, r % s.n_sblocks, r / s.n_sblocks, a.block_q, lane, w)) return;
  }
  const int kv_begin = w.kv_begin, kv_end = w.kv_end;
  const int n_rows = w.n_tok * a.qpk;
  const int tile_lo = kv_begin / kTile;
  const int n_iter = (kv_end + kTile - 1) / kTile - tile_lo;
  const int R = n_rows <= 16 ? 1 : (n_rows <= 32 ? 2 : 4);
  const int KG = kConsumerWarps / R;

  const uint32_t bar_full = smem_base + C::kBarOff;
  const uint32_t bar_empty = bar_full + kStages * 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full + 8 * i, 32);  // one arrival per producer lane
      mbar_init(bar_empty + 8 * i, R);  // a tile is consumed by the R warps of one key group
    }
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    if constexpr (F8)
      produce_f8v4<L, BS, kStages>(a, smem_base, bar_full, bar_empty, w.row, h, tile_lo, n_iter,
                                   kv_begin, kv_end, lane);
    else
      produce_tiles_lsu<L, BS>(a, smem_base, bar_full, bar_empty, w.row, h, tile_lo, n_iter,
                               kv_begin, kv_end, lane);
    return;
  }

  // ================================================================== consumers
  const int rg = warp % R;
  const int kg = warp / R;
  const int g = lane >> 2;
  const int t = lane & 3;
  const uint32_t q_frag = smem_base + C::kQOff;

  // q -> fp16 A fragments in MMA order: [row group][group][k-step][lane] x 16 B.
  // Channel order inside a k-step: cols 2t, 2t+1 <- 32gq + 8t + 4s + {0,1},
  // cols 2t+8, 2t+9 <- 32gq + 8t + 4s + {2,3}; K rows use the same order.
  if (warp < R) {
    bool bad_q = false;
#pragma unroll
    for (int gq = 0; gq < G; ++gq) {
      uint32_t f[2][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int idx = warp * 16 + g + 8 * half;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (idx < n_rows) {
          const int tq = idx / a.qpk;
          const int hh = h * a.qpk + idx % a.qpk;
          const uint16_t *src = a.q + (static_cast<int64_t>(w.q0 + tq) * a.hq + hh) * D +
                                gq * 32 + t * 8;
          v = *reinterpret_cast<const uint4 *>(src);
        }
        f[0][half] = pack_half2(bf16_lo(v.x), bf16_hi(v.x));
        f[0][2 + half] = pack_half2(bf16_lo(v.y), bf16_hi(v.y));
        f[1][half] = pack_half2(bf16_lo(v.z), bf16_hi(v.z));
        f[1][2 + half] = pack_half2(bf16_lo(v.w), bf16_hi(v.w));
        bad_q |= half2_nonfinite(f[0][half]) || half2_nonfinite(f[0][2 + half]) ||
                 half2_nonfinite(f[1][half]) || half2_nonfinite(f[1][2 + half]);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        sts128(q_frag + (((warp * G + gq) * 2 + s) * 32 + lane) * 16,
               make_uint4(f[s][0], f[s][1], f[s][2], f[s][3]));
    }
    // q values beyond the fp16 range (|q| >= 65520) would give inf scores
    if (__any_sync(0xffffffffu, bad_q) && lane == 0)
      flag_status(a.status, PA_DEV_BAD_Q);
  }
  named_barrier(1, kConsumerWarps * 32);

  // last visible keys of rows g and g + 8; padding rows copy the
  // block's last row so their arithmetic stays finite
  int lim[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int idx = rg * 16 + g + 8 * half;
    lim[half] = min(kv_end - 1, idx < n_rows ? w.limit0 + (idx / a.qpk) * w.limit_step : kv_end - 1);
  }
  int min_lim = min(lim[0], lim[1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, o));

  // key (within its 16-key block) of score column n of an even / odd n-tile
  const int kc0 = perm16(2 * t), kc1 = perm16(2 * t + 1);  // even n-tile, cols 2t, 2t+1
  const int kr_even = perm16(g), kr_odd = perm16(8 + g);    // K rows this lane loads

  float m_run[2] = {-INFINITY, -INFINITY};  // running max, log2 units
  float l_run[2] = {0.0f, 0.0f};            // this lane's share of the expsum
  float o_acc[4 * G][4];                    // n-tile (gq, j): channels 32gq + 8j + 2t + {0,1}
#pragma unroll
  for (int i = 0; i < 4 * G; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o_acc[i][e] = 0.0f;

  bool timed_out = false;
  for (int it = kg; it < n_iter; it += KG) {
    const int stage = it % kStages;
    if (!mbar_wait(bar_full + 8 * stage, (it / kStages) & 1, a.wait_limit_ns)) {
      timed_out = true;
      break;
    }
    const uint32_t st = smem_base + stage * L::kBytes;
    const int key0 = (tile_lo + it) * kTile;

    // ---------------- S = q k^T, exact codes, per-group scale
    float sc[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nt][e] = 0.0f;
#pragma unroll
    for (int gq = 0; gq < G; ++gq) {
      const uint4 qa0 = lds128(q_frag + (((rg * G + gq) * 2 + 0) * 32 + lane) * 16);
      const uint4 qa1 = lds128(q_frag + (((rg * G + gq) * 2 + 1) * 32 + lane) * 16);
#pragma unroll
      for (int nt = 0; nt < 8; ++nt) {
        const int kb16 = (nt >> 1) * 16;
        const uint2 kw = lds64(st + L::k_off(kb16 + ((nt & 1) ? kr_odd : kr_even), gq * 32 + t * 8));
        if constexpr (F8) {  // e4m3 bytes (0,1) -> k 2t, 2t+1; (2,3) -> k 2t+8, 2t+9
          mma_f16_16816(sc[nt], qa0.x, qa0.y, qa0.z, qa0.w, e4m3x2_to_half2(kw.x),
                        e4m3x2_to_half2(kw.x >> 16));
          mma_f16_16816(sc[nt], qa1.x, qa1.y, qa1.z, qa1.w, e4m3x2_to_half2(kw.y),
                        e4m3x2_to_half2(kw.y >> 16));
        } else {
          uint32_t b0, b1, b2, b3;
          codes4_to_half2(kw.x, b0, b1);
          codes4_to_half2(kw.y, b2, b3);
          float sg[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16_16816(sg, qa0.x, qa0.y, qa0.z, qa0.w, b0, b1);
          mma_f16_16816(sg, qa1.x, qa1.y, qa1.z, qa1.w, b2, b3);
          const int off = (nt & 1) ? 2 : 0;  // odd n-tiles hold keys 4t+2, 4t+3
          const float s0 = __half2float(__ushort_as_half(lds16(st + L::ks_off(kb16 + kc0 + off, gq))));
          const float s1 = __half2float(__ushort_as_half(lds16(st + L::ks_off(kb16 + kc1 + off, gq))));
          sc[nt][0] = fmaf(sg[0], s0, sc[nt][0]);
          sc[nt][1] = fmaf(sg[1], s1, sc[nt][1]);
          sc[nt][2] = fmaf(sg[2], s0, sc[nt][2]);
          sc[nt][3] = fmaf(sg[3], s1, sc[nt][3]);
        }
      }
    }

    // ---------------- mask, online softmax (log2 domain)
    const bool need_mask = key0 + kTile - 1 > min_lim || key0 < kv_begin;
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = sc[nt][e] * a.scale_log2;
        if (need_mask) {
          const int key = key0 + (nt >> 1) * 16 + ((e & 1) ? kc1 : kc0) + ((nt & 1) ? 2 : 0);
          if (key > lim[e >> 1] || key < kv_begin) v = -INFINITY;
        }
        sc[nt][e] = v;
        mx[e >> 1] = fmaxf(mx[e >> 1], v);
      }
    float alpha[2], mu[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      const float mn = fmaxf(m_run[r], mx[r]);
      mu[r] = mn == -INFINITY ? 0.0f : mn;
      alpha[r] = fast_exp2(m_run[r] - mu[r]);
      m_run[r] = mn;
      l_run[r] *= alpha[r];
    }
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = fast_exp2(sc[nt][e] - mu[e >> 1]);
        sc[nt][e] = p;
        l_run[e >> 1] += p;
      }
#pragma unroll
    for (int i = 0; i < 4 * G; ++i) {
      o_acc[i][0] *= alpha[0];
      o_acc[i][1] *= alpha[0];
      o_acc[i][2] *= alpha[1];
      o_acc[i][3] *= alpha[1];
    }

    // ---------------- O += P V', V' = code * scale in fp16 from channel-major pages
    const bool tail = key0 + kTile > kv_end || key0 < kv_begin;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t pa0 = pack_half2(sc[2 * kk][0], sc[2 * kk][1]);
      const uint32_t pa1 = pack_half2(sc[2 * kk][2], sc[2 * kk][3]);
      const uint32_t pa2 = pack_half2(sc[2 * kk + 1][0], sc[2 * kk + 1][1]);
      const uint32_t pa3 = pack_half2(sc[2 * kk + 1][2], sc[2 * kk + 1][3]);
      if constexpr (F8) {
        // the 4 keys 4t .. 4t+3 of this 16-key block: their scales and zeros
        // (zeroed outside [kv_begin, kv_end): stale bytes may sit there)
        uint2 vsc = lds64(st + L::vs_off(kk * 16 + 4 * t));
        uint2 vzr = lds64(st + L::vz_off(kk * 16 + 4 * t));
        if (tail) {
          const int k = key0 + kk * 16 + 4 * t;
          const auto in = [&](int x) { return x >= kv_begin && x < kv_end; };
          const uint32_t mx = (in(k) ? 0x0000ffffu : 0u) | (in(k + 1) ? 0xffff0000u : 0u);
          const uint32_t my = (in(k + 2) ? 0x0000ffffu : 0u) | (in(k + 3) ? 0xffff0000u : 0u);
          vsc.x &= mx;
          vzr.x &= mx;
          vsc.y &= my;
          vzr.y &= my;
        }
#pragma unroll
        for (int c8 = 0; c8 < D / 8; ++c8) {
          const uint32_t w = lds16(st + L::v_off(c8 * 8 + g, kk * 16 + 4 * t));
          uint32_t b0, b1;
          nibbles4_to_half2(w, b0, b1);  // keys 4t, 4t+1 | 4t+2, 4t+3
          mma_f16_16816(o_acc[c8], pa0, pa1, pa2, pa3, hfma2_u32(b0, vsc.x, vzr.x),
                        hfma2_u32(b1, vsc.y, vzr.y));
        }
      } else {
#pragma unroll
        for (int gq = 0; gq < G; ++gq) {
          const uint2 vsc = v_scales4<L>(st, kk * 16 + 4 * t, gq, tail, key0, kv_begin, kv_end);
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const uint32_t w = lds32(st + L::v_off(gq * 32 + jj * 8 + g, kk * 16 + 4 * t));
            uint32_t b0, b1;
            codes4_to_half2(w, b0, b1);  // keys 4t, 4t+1 -> k 2t, 2t+1; 4t+2, 4t+3 -> k 2t+8, 2t+9
            mma_f16_16816(o_acc[gq * 4 + jj], pa0, pa1, pa2, pa3, hmul2_u32(b0, vsc.x),
                          hmul2_u32(b1, vsc.y));
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_empty + 8 * stage);
  }
  if (timed_out && lane == 0) flag_status(a.status, PA_DEV_TIMEOUT);

  // row expsums: sum the 4 lanes of a row
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 1);
    l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 2);
  }

  // ---------------- merge the KG warps of a row group (field-major, no conflicts)
  if (KG > 1) {
    named_barrier(1, kConsumerWarps * 32);  // every stage consumed: reuse them
    float *mbuf = reinterpret_cast<float *>(smem);
    if (kg > 0) {
      float *dst = mbuf + (warp - R) * C::kMergeFields * 32 + lane;
      dst[0 * 32] = m_run[0];
      dst[1 * 32] = m_run[1];
      dst[2 * 32] = l_run[0];
      dst[3 * 32] = l_run[1];
#pragma unroll
      for (int i = 0; i < 4 * G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[(4 + i * 4 + e) * 32] = o_acc[i][e];
    }
    named_barrier(1, kConsumerWarps * 32);
    if (kg > 0) return;
    for (int k = 1; k < KG; ++k) {
      const float *src = mbuf + (rg + k * R - R) * C::kMergeFields * 32 + lane;
      float wa[2], wb[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mo = src[r * 32];
        const float lo = src[(2 + r) * 32];
        const float mn = fmaxf(m_run[r], mo);
        const float muv = mn == -INFINITY ? 0.0f : mn;
        wa[r] = fast_exp2(m_run[r] - muv);
        wb[r] = fast_exp2(mo - muv);
        m_run[r] = mn;
        l_run[r] = l_run[r] * wa[r] + lo * wb[r];
      }
#pragma unroll
      for (int i = 0; i < 4 * G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o_acc[i][e] = o_acc[i][e] * wa[e >> 1] + src[(4 + i * 4 + e) * 32] * wb[e >> 1];
    }
  }

  // ---------------- write this segment's triples
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int idx = rg * 16 + g + 8 * half;
    if (idx >= n_rows) continue;
    const int64_t r = static_cast<int64_t>(w.q0) * a.qpk + idx, step = rows_total(s) * 4;
    float *dst = acc_at<D>(s, w.slot, h) + (t >> 1) * step + r * 4 + (t & 1) * 2;
#pragma unroll
    for (int i = 0; i < 4 * G; ++i)  // channels 8i + 2t, + 1
      *reinterpret_cast<float2 *>(dst + 2 * i * step) =
          make_float2(o_acc[i][2 * half], o_acc[i][2 * half + 1]);
    if (t == 0)
      *reinterpret_cast<float2 *>(a.part_ml + (ml_at(s, w.slot, h) + r) * 2) =
          make_float2(m_run[half], l_run[half]);
  }
}

// The join: all segment triples of a row (query token x q head) and its sink
// merged to bf16 output and fp32 LSE.  One warp per 8 consecutive rows of a kv
// head and 16 channels: lane l reads 4 channels (l / 8) of row l % 8, so that
// eight lanes take a whole 128-byte line of a segment, and every segment's load
// is in flight at once (8 or 4 a batch); where there are more warps than fit at once,
// a warp takes several channel blocks in turn.  Bound by its reads (D + 2 floats a row and
// segment, L2 hits); with 32-byte pieces, two rows of all channels a warp, it
// took 15 us where it now takes 5 (64 requests, 21 segments).  Launched beside
// the last kernel: it looks up its rows' sequences and then waits.
template <int D, int kBatch>
__global__ void __launch_bounds__(256, kBatch == 8 ? 3 : 4)
    shared_join_kernel(const __grid_constant__ SharedArgs s, int cpw_log2) {
  constexpr int kCbLog2 = D == 64 ? 2 : D == 128 ? 3 : 4;  // D / 16 channel blocks of a row
  const AttnArgs &a = s.a;
  const LastBlockWaits at_end{blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1};
  const int lane = threadIdx.x & 31;
  // rows fit 32 bits: their output alone takes 128 bytes a row
  const uint32_t rows = static_cast<uint32_t>(rows_total(s));
  const uint32_t gw = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int slices_log2 = kCbLog2 - cpw_log2;
  if ((gw >> slices_log2) >= (rows + 7) / 8) return;
  const int cb0 = static_cast<int>(gw & ((1u << slices_log2) - 1u)) << cpw_log2;
  const int h = static_cast<int>(blockIdx.y);
  const uint32_t row = (gw >> slices_log2) * 8 + (lane & 7);
  const int piece = lane >> 3;  // 4 channels of the 16; segments piece + 4 j of a round

  // this lane's row: its token, q head, and how many segments hold its keys.  Few
  // groups are read by a lane each, beside the row's own entries: the blocks that
  // come last start when the kernel before has ended, and wait for each round.
  const bool few = s.num_groups < 32;
  int first = 0x7fffffff, len = 0;
  if (few && lane <= s.num_groups) {
    first = s.cu_groups[lane];
    if (lane < s.num_groups) len = s.prefix_lens[lane];
  }
  int n_p = 0, n_s = 0;
  const int tok = static_cast<int>(min(row, rows - 1) / static_cast<uint32_t>(a.qpk));
  const int hh = h * a.qpk + static_cast<int>(row % static_cast<uint32_t>(a.qpk));
  // a batch of single tokens: sequence = token; a search otherwise
  int seq = min(tok, a.num_seqs - 1);
  int c0 = a.cu_seqlens_q[seq], c1 = a.cu_seqlens_q[seq + 1], seq_len = a.seq_lens[seq];
  const int token = few && first >= 0 && first <= a.num_seqs ? a.cu_seqlens_q[first] : 0x7fffffff;
  if (c0 > tok || c1 <= tok) {
    seq = last_at_most(a.cu_seqlens_q, a.num_seqs, tok);
    c0 = a.cu_seqlens_q[seq], c1 = a.cu_seqlens_q[seq + 1], seq_len = a.seq_lens[seq];
  }
  // the row's group: its first sequence, that of the next, its prefix, its tokens
  int s0, s1, P, g0, g1;
  if (few) {
    int g = 0;
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
      const int v = __shfl_sync(0xffffffffu, first, (g + step) & 31);
      if (g + step < s.num_groups && v <= seq) g += step;
    }
    s0 = __shfl_sync(0xffffffffu, first, g), s1 = __shfl_sync(0xffffffffu, first, g + 1);
    P = __shfl_sync(0xffffffffu, len, g);
    g0 = __shfl_sync(0xffffffffu, token, g), g1 = __shfl_sync(0xffffffffu, token, g + 1);
  } else {
    const int g = last_at_most(s.cu_groups, s.num_groups, seq);
    s0 = s.cu_groups[g], s1 = s.cu_groups[g + 1], P = s.prefix_lens[g];
    g0 = group_token(s, g), g1 = group_token(s, g + 1);
  }
  const int ctx = seq_len - (c1 - c0);
  P = min(P, s.capacity);
  if (row < rows && c0 >= 0 && tok >= c0 && tok < c1) {  // else: a row no sequence owns
    if (c1 <= a.num_tokens && s0 <= seq && s1 > seq && rows_of(s, c1 - c0) <= s.max_rows && P >= 0 &&
        ctx >= P && g0 >= 0 && g0 <= tok && tok < g1 && g1 <= a.num_tokens) {
      n_p = shared_segments(0, P, s.seg_p, s.ns_p);
      n_s = shared_segments(P, min(ctx + tok - c0 + 1, s.capacity), s.seg_s, s.ns_s);
    } else {
      // its prefix or its suffix was not taken (bounds of its group out of the batch are
      // seen by the prefix items, its own entries by the suffix items): not written
      flag_status(a.status, PA_DEV_BAD_SEQ);
    }
  }
  const int n = n_s > 0 ? n_p + n_s : 0;  // 0: a row that is not written
  const int n_max = __reduce_max_sync(0xffffffffu, n);
  if (n_max == 0) return;
  const float sink = a.sinks && n > 0 ? sink_log2(a, hh) : -INFINITY;
  // segment k of the row: its slot k, past the prefix's the unused ones skipped
  const int64_t per_slot = static_cast<int64_t>(a.hk) * rows;  // (m, l) pairs; D floats of acc each
  const int64_t skip = (s.ns_p - n_p) * per_slot;
  const float *ml_row = a.part_ml + (ml_at(s, 0, h) + row) * 2;
  wait_for_predecessor();  // the triples
#pragma unroll 1
  for (int cb = cb0; cb < cb0 + (1 << cpw_log2); ++cb) {
    float M = sink;
    float total = sink > -INFINITY && piece == 0 ? 1.0f : 0.0f;  // this lane's share, scaled to M
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *acc_row = acc_at<D>(s, 0, h) + (static_cast<int64_t>(cb * 4 + piece) * rows + row) * 4;
    for (int k0 = 0; k0 < n_max; k0 += 16) {
      float4 x[kBatch];
      auto load = [&](int k1) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          x[i] = k1 + i < n ? *reinterpret_cast<const float4 *>(acc_row + (k1 + i) * (per_slot * D) +
                                                                (k1 + i < n_p ? 0 : skip * D))
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      };
      float2 ml[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + piece + 4 * j;
        ml[j] = k < n ? *reinterpret_cast<const float2 *>(ml_row + (k * per_slot + (k < n_p ? 0 : skip)) * 2)
                      : make_float2(-INFINITY, 0.0f);
      }
      load(k0);
      float m = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = fmaxf(M, fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16)));
      const float mu = m == -INFINITY ? 0.0f : m;
      const float f = fast_exp2(M - mu);
      M = m;
      float w[4];
      total *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = fast_exp2(ml[j].x - mu);
        total = fmaf(w[j], ml[j].y, total);
      }
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
#pragma unroll
      for (int b = 0; b < 16 / kBatch; ++b) {
        if (k0 + b * kBatch >= n_max) break;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int k = b * kBatch + i;
          const float wk = __shfl_sync(0xffffffffu, w[k >> 2], (k & 3) * 8 + (lane & 7));
          acc.x = fmaf(wk, x[i].x, acc.x);
          acc.y = fmaf(wk, x[i].y, acc.y);
          acc.z = fmaf(wk, x[i].z, acc.z);
          acc.w = fmaf(wk, x[i].w, acc.w);
        }
        if (b + 1 < 16 / kBatch) load(k0 + (b + 1) * kBatch);
      }
    }
    total += __shfl_xor_sync(0xffffffffu, total, 8);
    total += __shfl_xor_sync(0xffffffffu, total, 16);
    if (n > 0) {
      const float inv = 1.0f / total;
      const int64_t to = static_cast<int64_t>(tok) * a.hq + hh;
      *reinterpret_cast<uint2 *>(a.out + to * D + cb * 16 + piece * 4) =
          make_uint2(pack_bf162(acc.x * inv, acc.y * inv), pack_bf162(acc.z * inv, acc.w * inv));
      if (cb == 0 && piece == 0 && a.lse) a.lse[to] = (M + log2f(total)) * kLn2;
    }
  }
}

// ---------------------------------------------------------------------- host

// Whether the prefix items go to the tensor-core kernel: its blocks hold 256
// rows and convert a tile for them all, the warp-MMA kernel's hold 64.
static bool prefix_on_tc(int32_t num_tokens, int32_t num_groups, int32_t qpk, int32_t d) {
  return shared_tc_rows(d) > 0 &&
         static_cast<int64_t>(num_tokens) * qpk >= int64_t{32} * num_groups;
}

// a * b * c of sizes below 2^31, at most 2^40: no count of segments goes by more.
static int64_t blocks_of(int64_t a, int64_t b, int64_t c) {
  constexpr int64_t kMost = int64_t{1} << 40;
  const int64_t ab = a * b;
  return ab > kMost / c ? kMost : ab * c;
}

SharedSplits shared_splits(int32_t num_seqs, int32_t num_tokens, int32_t num_groups, int32_t hq,
                           int32_t hk, int32_t d, int32_t max_query_len, int32_t max_prefix_len,
                           int32_t max_suffix_len) {
  const int qpk = hq / hk;
  SharedSplits r;
  // suffixes: blocks of a segment (8 or 16 rows in the rows kernel, 64 in the row-tile
  // kernel), tiles of the longest.  Every sequence is taken for as long as the longest
  // query: one long query among many short ones leaves the prefix and the suffixes of
  // all too few segments (63 tokens and a query of 9 behind 8192 keys 142 us, 64
  // tokens 41).
  const int64_t most = static_cast<int64_t>(max_query_len) * qpk;
  const bool few = most <= kFewRows;
  const int64_t tile = few ? rows_per_pass(d, most) : kRowTile;
  const int64_t sunits = blocks_of(num_seqs, hk, (most + tile - 1) / tile);
  const int64_t stiles = (static_cast<int64_t>(max_suffix_len) + kTile - 1) / kTile;
  {
    // prefix: the count of segments that ends soonest, in units of a tile's time,
    // of a model fitted to 68 batches x 20 counts each (all D, both formats, 1 - 128
    // sequences, 1 - 5 groups): on average it was 2.8 % above the best count's time;
    // whole waves of the prefix's blocks by themselves were 8.4 % above it.  The kernels
    // have become faster since: 12 batches at D = 256 are now 5 % above their best on
    // average, 25 % at worst (8 requests of up to 1500 own keys behind 4096).
    //  - A block takes its tiles and 8 more (set-up, first loads, triples; row-tile
    //    kernel: 6).
    //  - The suffixes (half of the longest on average, and 5 tiles of set-up; a tile
    //    is 0.35 of a prefix tile, 3 in the row-tile kernel) run on the SMs that the
    //    prefix's blocks leave.  So a prefix of few, long blocks on half of the SMs
    //    beats one on all of them: 64 requests, 8192 keys, 8 segments 39 us, 19
    //    segments 50.
    //  - Several groups: their lengths differ, and waves overlap.
    //  - The join reads a triple a segment, 16 in flight at a time.
    const bool tc = prefix_on_tc(num_tokens, num_groups, qpk, d);
    const int rows = tc ? shared_tc_rows(d) : kRowTile;
    const int64_t block_q = std::max(1, rows / qpk);
    const int64_t units =
        blocks_of(std::max<int64_t>(num_groups, (num_tokens + block_q - 1) / block_q), hk, 1);
    const int64_t slots = tc || d == 256 ? 152 : 304;  // resident blocks
    const int64_t tiles = std::max(1, (max_prefix_len + kTile - 1) / kTile);
    const double join = static_cast<double>(num_tokens) * hq * (d + 2) * 8 / 2.2e6;
    const double suffix =
        (few ? 0.35 : 3.0) * static_cast<double>(sunits) * (0.5 * static_cast<double>(stiles) + 5.0);
    const double held = tc ? 1.0 : 0.5;  // share of an SM a prefix block takes
    double best = 0;
    r.prefix = 1;
    for (int n = 1; n <= 64 && n <= tiles; ++n) {
      const double blocks = static_cast<double>(units * n);
      const double waves = num_groups == 1 ? static_cast<double>((units * n + slots - 1) / slots)
                                           : std::max(1.0, 0.9 * blocks / static_cast<double>(slots));
      const double block = static_cast<double>((tiles + n - 1) / n) + (tc ? 8.0 : 6.0);
      const double cost =
          std::max(waves * block, (blocks * block * held + suffix) / static_cast<double>(slots)) +
          join * n + 1.5 * ((n + 15) / 16);
      if (n == 1 || cost < best) {
        best = cost;
        r.prefix = n;
      }
    }
  }
  {
    // suffix: ~1024 keys a segment (the decode kernel's measured best; 2048 where one
    // segment each fills the GPU, 128 requests of up to 2048 keys behind 32768: 218 us
    // against 228), more only while blocks are too few to fill the GPU: four of the
    // rows kernel to an SM, of 4 tiles at least; two at D = 256, where whole rounds of
    // them are taken, no part of one (32 requests behind 16384 keys, a segment each 43
    // us, two 46; 16 of 24 rows and up to 2048 keys behind 4096: two 26.5, three 23;
    // 64 of 16 rows and 2000 keys behind 8192: one 62, two 58); one of the row-tile
    // kernel, a tile at least (2 x 40 tokens of 4 rows behind 1284 keys of D = 256:
    // 7 segments 35 us, 3 45).
    const int64_t full = !few ? 152 : d == 256 ? 304 : 608;
    const int64_t cap = few ? (stiles + 3) / 4 : stiles + 1;
    const int64_t rounds = few && d == 256 ? full / sunits : (full + sunits - 1) / sunits;
    const int64_t keys = sunits >= full ? 2048 : 1024;
    int64_t n = std::max<int64_t>((static_cast<int64_t>(max_suffix_len) + keys - 1) / keys,
                                  std::min(rounds, cap));
    n = std::min(n, std::max<int64_t>(1, 8192 / sunits));
    r.suffix = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(n, 64)));
  }
  return r;
}

template <int D, int BS, bool F8>
static cudaError_t launch_shared_mma_t(const SharedArgs &s, cudaStream_t stream) {
  using C = SharedMmaCfg<D, BS, F8>;
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    return cudaFuncSetAttribute(shared_mma_kernel<D, BS, F8>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  const int64_t gx = static_cast<int64_t>(s.n_pblocks) * s.ns_p +
                     static_cast<int64_t>(s.n_sblocks) * s.ns_s;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(s.a.hk));
  return launch_kernel(shared_mma_kernel<D, BS, F8>, grid, kThreads, C::kSmemBytes, stream, s);
}

static cudaError_t launch_shared_mma(const SharedArgs &s, int d, int bs, bool f8v4,
                                     cudaStream_t stream) {
#define PAQ8_SHARED_CASE(DD, BB)                                          \
  if (d == DD && bs == BB)                                                \
    return f8v4 ? launch_shared_mma_t<DD, BB, true>(s, stream)            \
                : launch_shared_mma_t<DD, BB, false>(s, stream);
  PAQ8_SHARED_CASE(64, 16)
  PAQ8_SHARED_CASE(64, 32)
  PAQ8_SHARED_CASE(128, 16)
  PAQ8_SHARED_CASE(128, 32)
  PAQ8_SHARED_CASE(256, 16)
  PAQ8_SHARED_CASE(256, 32)
#undef PAQ8_SHARED_CASE
  return cudaErrorInvalidValue;
}

// 2-D byte map of page rows: `rows` rows of `row_bytes`, boxes of box_y rows of
// up to 128 bytes.
static bool encode_page_map(CUtensorMap *map, const void *base, int64_t rows, int row_bytes,
                            int box_y, CUtensorMapSwizzle swizzle) {
  typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const EncodeTiled fn = []() -> EncodeTiled {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(std::min(row_bytes, 128)),
                             static_cast<cuuint32_t>(box_y)};
  const cuuint32_t step[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_shared_prefix(const SharedLaunch &L, cudaStream_t stream) {
  SharedArgs s{};
  AttnArgs &a = s.a;
  a.q = static_cast<const uint16_t *>(L.q);
  a.cu_seqlens_q = L.cu;
  a.seq_lens = L.seq_lens;
  a.block_table = L.block_table;
  a.k_cache = static_cast<const int8_t *>(L.k_cache);
  a.v_cache = static_cast<const int8_t *>(L.v_cache);
  a.k_scale = static_cast<const uint16_t *>(L.k_scale);
  a.v_scale = static_cast<const uint16_t *>(L.v_scale);
  a.v_zero = static_cast<const uint16_t *>(L.v_zero);
  a.out = static_cast<uint16_t *>(L.out);
  a.lse = L.lse;
  a.status = reinterpret_cast<uint32_t *>(L.workspace);
  a.num_seqs = L.num_seqs;
  a.num_tokens = L.num_tokens;
  a.hq = L.hq;
  a.hk = L.hk;
  a.qpk = L.hq / L.hk;
  a.num_blocks = L.num_blocks;
  a.bt_stride = L.bt_stride;
  a.scale_log2 = L.softmax_scale * kLog2e;
  a.causal = 1;
  a.sinks = L.sinks;
  a.wait_limit_ns = kWaitLimitNs;
  const int64_t triples = static_cast<int64_t>(L.num_tokens) * L.hq *
                          (L.prefix_splits + L.suffix_splits);
  a.part_acc = reinterpret_cast<float *>(L.workspace + 256);
  a.part_ml = a.part_acc + triples * L.d;
  s.cu_groups = L.cu_groups;
  s.prefix_lens = L.prefix_lens;
  s.num_groups = L.num_groups;
  s.capacity = static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(L.bt_cols) * L.bs, 0x7fffffff - 4096));
  s.ns_p = L.prefix_splits;
  s.ns_s = L.suffix_splits;
  auto seg = [](int len, int ns) { return std::max(1, ((len + kTile - 1) / kTile + ns - 1) / ns); };
  s.seg_p = seg(L.max_prefix_len, s.ns_p);
  s.seg_s = seg(L.max_suffix_len + kTile, s.ns_s);  // a suffix may start inside a tile
  // Who takes what: the prefix goes to the tensor-core kernel or the row-tile
  // kernel (prefix_on_tc), a suffix of up to kFewRows rows to the rows kernel,
  // of more to the row-tile kernel.  Where that one takes the prefix and the
  // suffixes are little, it takes them all: a launch less (3.4 us of a call whose
  // host side is longer than its 8 - 12 us on the GPU).  On the GPU, one kernel
  // against two: 7.7 us and 8.3 (4 sequences, 37 own keys, 2 kv heads of 64), 11.6
  // and 12.7 (8 of 128), 16.8 and 22.7 (8 of 256); with 1000 own keys 11.1 and 9.8,
  // 26 and 15, 39 and 24.
  const bool tc = prefix_on_tc(L.num_tokens, L.num_groups, a.qpk, L.d);
  const int64_t little = L.d == 64 ? 256 : 64;  // (sequence, kv head, tile of keys)
  const bool one = !tc && static_cast<int64_t>(L.num_seqs) * L.hk *
                              ((static_cast<int64_t>(L.max_suffix_len) + kTile - 1) / kTile) <= little;
  const int64_t most = static_cast<int64_t>(L.max_query_len) * a.qpk;  // rows of a sequence
  const bool many = one || most > kFewRows;
  s.few_rows = one ? 0 : static_cast<int32_t>(std::min<int64_t>(most, kFewRows));
  s.max_rows = many ? 0x7fffffff : s.few_rows;
  cudaError_t e = cudaSuccess;
  if (tc) {
    CUtensorMap tk = {}, tv = {};
    const int64_t pages = static_cast<int64_t>(L.num_blocks) * L.hk;
    if (!encode_page_map(&tk, L.k_cache, pages * L.bs, L.d, L.bs,
                         L.d >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
        (!L.f8v4 && !encode_page_map(&tv, L.v_cache, pages * L.d, L.bs, L.d,
                                     L.bs == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                : CU_TENSOR_MAP_SWIZZLE_NONE)))
      return cudaErrorInvalidValue;
    SharedArgs p = s;
    p.a.block_q = shared_tc_rows(L.d) / a.qpk;
    p.n_pblocks = prefix_blocks(L.num_tokens, L.num_groups, p.a.block_q);
    if ((e = launch_shared_tc(p, tk, tv, L.d, L.bs, L.f8v4, stream)) != cudaSuccess) return e;
  }
  if (!tc || many) {
    a.block_q = std::max(1, kRowTile / a.qpk);
    s.n_pblocks = tc ? 0 : prefix_blocks(L.num_tokens, L.num_groups, a.block_q);
    s.n_sblocks = many ? L.num_tokens / a.block_q + L.num_seqs : 0;
    s.first = !tc;
    if ((e = launch_shared_mma(s, L.d, L.bs, L.f8v4, stream)) != cudaSuccess) return e;
  }
  if (!one && (e = launch_shared_rows(s, L.d, L.bs, L.f8v4, stream)) != cudaSuccess) return e;
  // All blocks resident at once, so that a row's look-ups are not repeated behind a
  // first wave: eight loads in flight a lane and three blocks an SM where each warp
  // can take one channel block so, else four loads, four blocks an SM, and several
  // channel blocks in turn (128 requests of 64 q heads 196 us against 199; the other
  // way round 32 requests of 256-channel heads 42.7 against 41.2)
  const int64_t groups = (static_cast<int64_t>(L.num_tokens) * a.qpk + 7) / 8;
  const int cb_log2 = L.d == 64 ? 2 : L.d == 128 ? 3 : 4;
  const bool eight = (groups << cb_log2) * L.hk <= 3 * 8 * 152;
  int cpw_log2 = 0;
  while (!eight && cpw_log2 < cb_log2 && (groups << (cb_log2 - cpw_log2)) * L.hk > 4 * 8 * 152) ++cpw_log2;
  const int64_t blocks = ((groups << (cb_log2 - cpw_log2)) + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(L.hk));
  switch (L.d) {
    case 64:
      return launch_kernel(eight ? shared_join_kernel<64, 8> : shared_join_kernel<64, 4>, grid, 256, 0, stream,
                           s, cpw_log2);
    case 128:
      return launch_kernel(eight ? shared_join_kernel<128, 8> : shared_join_kernel<128, 4>, grid, 256, 0,
                           stream, s, cpw_log2);
    case 256:
      return launch_kernel(eight ? shared_join_kernel<256, 8> : shared_join_kernel<256, 4>, grid, 256, 0,
                           stream, s, cpw_log2);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paq8
