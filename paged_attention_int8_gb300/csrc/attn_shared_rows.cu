// Attention over a shared prefix: the suffix of sequences with at most 32 query
// rows per kv head (query tokens x q heads: a decode token, a few draft tokens
// verified together), one key segment per block, in the swap-AB form
// of the decode kernel (attn_decode.cu): keys in the MMA's M dimension, rows in
// its N dimension,
//   S^T[16 keys x 8 rows] = K[16 x 16 ch] . Q^T[16 ch x 8],
//   O^T[16 ch x 8 rows] += V^T[16 ch x 16 keys] . P^T[16 keys x 8],
// NT tiles of 8 rows (1 or 2, by the bound of the query lengths) off every converted
// key and value: the conversions, not the MMAs, are most of a block's instructions.
// More rows than 8 NT take several passes.
// Each row has its own causal limit, taken on edge blocks only.  HBM bound:
// 2 (D + D / 16) bytes a key and kv head (q8), D + D / 2 + 4 (fp8 / 4-bit).
//
// Four warps share a segment's 16-key blocks round robin, each on its own: it
// copies its blocks with 16-byte cp.async into a private 3-stage ring and reads
// them back, so that no warp waits for another until the four softmax states
// are merged at the end (one fp32 triple per row); four blocks of 128 registers a
// thread hold an SM at D = 64, 128 and one row tile.
#include <type_traits>

#include "attn_shared.cuh"

namespace paq8 {

constexpr float kMaxP = 32768.0f;  // bound on P, inside fp16

// Four 8 x 16-byte matrices; lane l gives the address of row l % 8 of matrix l / 8 and
// gets bytes 4 (l % 4) .. + 3 of row l / 4 of each.
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr));
}

// The G fp16 K scales of one key row (contiguous) as floats.
template <int G>
__device__ __forceinline__ void load_key_scales(uint32_t addr, float (&f)[G]) {
  uint32_t w[G / 2];
  if constexpr (G == 2) {
    w[0] = lds32(addr);
  } else if constexpr (G == 4) {
    const uint2 v = lds64(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < G / 8; ++i) {
      const uint4 v = lds128(addr + 16 * i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < G / 2; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// One stage: a block of 16 keys.
//   K  [16][D] codes, rows of 128 bytes (D = 64: of 64, D = 256: two halves)
//   V  [D][16] codes (fp8 / 4-bit: [D][8], two keys a byte)
//   scales: K [16][G], V [G][16] fp16 (fp8 / 4-bit: scale [16], zero [16])
template <int D, bool F8>
struct RowsStage {
  static constexpr int G = D / 32;
  static constexpr int kVOff = 16 * D;
  static constexpr int kVBytes = F8 ? 8 * D : 16 * D;
  static constexpr int kKsOff = kVOff + kVBytes;        // fp8 / 4-bit: V scales
  static constexpr int kVsOff = kKsOff + (F8 ? 32 : 32 * G);  // fp8 / 4-bit: V zeros
  static constexpr int kBytes = (kVsOff + (F8 ? 32 : 32 * G) + 127) / 128 * 128;
  // Byte b of key row r.  A matrix of the MMA fragments' loads is one 16-byte piece
  // of the eight rows perm16(0 .. 7) (0, 1, 4, 5, 8, 9, 12, 13) or of those 2 on: the
  // pieces of a row are permuted so that these stand in different banks.
  __device__ static __forceinline__ uint32_t k_off(int r, int b) {
    if constexpr (D >= 128) {
      const int i = (r & 1) | ((r >> 2) << 1);
      const int off = r * 128 + (b & 127);
      return (b >> 7) * (16 * 128) + (off ^ ((((i & 3) << 1) | (i >> 2)) << 4));
    } else {
      const int off = r * 64 + b;
      return off ^ (((r >> 2) & 1) << 5) ^ (((r >> 3) & 1) << 4);
    }
  }
};

template <int D, int BS, bool F8, int NT>
struct SharedRowsCfg {
  using L = RowsStage<D, F8>;
  static constexpr int kWarps = 4;
  static constexpr int kSt = 3;
  static constexpr int kCm = D / 16;                    // 16-channel blocks of the output
  static constexpr int G = D / 32;
  // blocks per SM: as many as the registers hold without spills (48 requests of up to
  // 20 rows and 2000 keys, D = 128: three blocks 60 us, four with 144 bytes spilled 95)
  static constexpr int kMinBlocks = D == 256 ? 2 : (D == 128 && NT == 2) ? 3 : 4;
  static constexpr int kRing = kWarps * kSt * L::kBytes;
  static constexpr int kMerge = kWarps * 32 * NT * (4 + 4 * kCm) * 4;
  static constexpr int kSmem = (kRing > kMerge ? kRing : kMerge) + 1024;
};

// This lane's share of the copy of 16-key block `half` (of BS / 16) of page
// `page` (block id * hk + kv head) into the stage at `st`.
template <int D, int BS, bool F8>
__device__ __forceinline__ void copy_rows_block(const AttnArgs &a, uint32_t st, int64_t page, int half,
                                                int lane) {
  using L = RowsStage<D, F8>;
  constexpr int G = D / 32;
  const uint8_t *k = reinterpret_cast<const uint8_t *>(a.k_cache) + page * (BS * D) + half * (16 * D);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = lane + 32 * i;
    cp_async16(st + L::k_off(c / (D / 16), (c % (D / 16)) * 16), k + c * 16);
  }
  const uint8_t *v = reinterpret_cast<const uint8_t *>(a.v_cache);
  if constexpr (!F8) {
    v += page * (BS * D) + half * 16;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int c = lane + 32 * i;  // channel
      cp_async16(st + L::kVOff + c * 16, v + c * BS);
    }
    // 2 G pieces of K scales, then 2 G of V scales (G rows of BS)
    const uint8_t *ks = reinterpret_cast<const uint8_t *>(a.k_scale) + page * (BS * G * 2) + half * (32 * G);
    const uint8_t *vs = reinterpret_cast<const uint8_t *>(a.v_scale) + page * (BS * G * 2) + half * 32;
    if (lane < 4 * G) {
      const int c = lane < 2 * G ? lane : lane - 2 * G;
      cp_async16(st + (lane < 2 * G ? L::kKsOff : L::kVsOff) + c * 16,
                 lane < 2 * G ? ks + c * 16 : vs + (c >> 1) * (BS * 2) + (c & 1) * 16);
    }
  } else {
    v += page * (BS * D / 2) + half * 8;
    if constexpr (BS == 16) {
#pragma unroll
      for (int i = 0; i < (D / 2 + 31) / 32; ++i) {
        const int c = lane + 32 * i;  // two channels
        if (D / 2 >= 32 || c < D / 2) cp_async16(st + L::kVOff + c * 16, v + c * 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int c = lane + 32 * i;
        cp_async_8(st + L::kVOff + c * 8, v + c * (BS / 2));
      }
    }
    if (lane < 4) {
      const uint8_t *s = reinterpret_cast<const uint8_t *>(lane < 2 ? a.v_scale : a.v_zero);
      cp_async16(st + (lane < 2 ? L::kKsOff : L::kVsOff) + (lane & 1) * 16,
                 s + page * (BS * 2) + half * 32 + (lane & 1) * 16);
    }
  }
}

template <int D, int BS, bool F8, int NT>
__global__ void __launch_bounds__(128, SharedRowsCfg<D, BS, F8, NT>::kMinBlocks)
    shared_rows_kernel(const __grid_constant__ SharedArgs sa) {
  using Cfg = SharedRowsCfg<D, BS, F8, NT>;
  using L = typename Cfg::L;
  constexpr int G = Cfg::G;
  constexpr int kWarps = Cfg::kWarps;
  constexpr int kSt = Cfg::kSt;
  const AttnArgs &a = sa.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float *smem_f = reinterpret_cast<float *>(smem_raw + (smem_base - smem_u32(smem_raw)));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // segment-major order: every sequence's first segment launches before any
  // second one, so that the last wave holds the short last segments
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.hk));
  const int rest = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.hk));
  const int seq = rest % a.num_seqs;
  const int row0 = rest / a.num_seqs % sa.row_passes * (8 * NT);
  const int sigma = rest / a.num_seqs / sa.row_passes;

  launch_dependents();
  const LastBlockWaits at_end{blockIdx.x == gridDim.x - 1};
  // one round of loads before any of them is looked at
  const int q_start = a.cu_seqlens_q[seq], q_end = a.cu_seqlens_q[seq + 1];
  const int seq_len = a.seq_lens[seq];
  const int P = prefix_of(sa, seq, lane);
  const int q_len = q_end - q_start;
  const int all_rows = rows_of(sa, q_len);
  if (q_len <= 0) return;
  if (all_rows > sa.few_rows) {  // shared_mma_kernel's, where it runs
    if (all_rows > sa.max_rows && sigma == 0 && row0 == 0 && h == 0 && threadIdx.x == 0)
      flag_status(a.status, PA_DEV_BAD_SEQ);  // max_query_len was below a q_len
    return;
  }
  const int ctx = seq_len - q_len;
  if (q_start < 0 || q_start + q_len > a.num_tokens || P < 0 || ctx < P) {
    if (threadIdx.x == 0 && sigma == 0 && row0 == 0) flag_status(a.status, PA_DEV_BAD_SEQ);
    return;
  }
  const int n_rows = min(8 * NT, all_rows - row0);  // of this pass
  if (n_rows <= 0) return;
  SharedWork w;
  if (seq_len > sa.capacity && threadIdx.x == 0) flag_status(a.status, PA_DEV_BAD_BLOCK);
  if (!segment_keys(P, min(seq_len, sa.capacity), sa.seg_s, sa.ns_s, sigma, w)) return;
  const int kv_begin = w.kv_begin, kv_end = w.kv_end;
  // this warp's 16-key blocks: b0, b0 + 4, ...
  const int b0 = kv_begin / 16 + warp;
  const int n_blk = max(0, ((kv_end + 15) / 16 - b0 + kWarps - 1) / kWarps);
  const uint32_t ring = smem_base + warp * (kSt * L::kBytes);
  const int32_t *bt_row = a.block_table + static_cast<int64_t>(seq) * a.bt_stride;
  int held = -1;  // block id of this lane's block: number (i / 32) * 32 + lane of this warp's
  // block ids of the warp's blocks i .. i + 31; -1: a bad entry, flagged and not copied.  Its
  // keys are what stood in the stage before, and the rows that see them undefined.
  auto load_ids = [&](int i) {
    held = -1;
    if (i + lane < n_blk) {
      const int lp = static_cast<int>((static_cast<int64_t>(b0) + kWarps * (i + lane)) / (BS / 16));
      const int b = lp < a.bt_stride ? bt_row[lp] : -1;
      if (b >= 0 && b < a.num_blocks) held = b;
      else flag_status(a.status, PA_DEV_BAD_BLOCK);
    }
  };
  // block i's copy into its stage, one commit group per block
  auto issue = [&](int i) {
    if (i < n_blk) {
      if ((i & 31) == 0) load_ids(i);
      const int id = __shfl_sync(0xffffffffu, held, i & 31);
      if (id >= 0)
        copy_rows_block<D, BS, F8>(a, ring + (i % kSt) * L::kBytes, static_cast<int64_t>(id) * a.hk + h,
                                   BS == 32 ? (b0 + kWarps * i) & 1 : 0, lane);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kSt - 1; ++i) issue(i);

  const int g = lane >> 2;
  const int t = lane & 3;

  // Q^T as the B operand: of row tile nt, lane (g, t) holds row 8 nt + g, channels
  // 32gq + 16s + 4t + {0,1} (k = 2t, 2t+1) and + {2,3} (k = 2t+8, 2t+9) for k-step s.
  uint32_t qb[NT][G][2][2];
  bool bad_q = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const bool hv = 8 * nt + g < n_rows;
    const int row = row0 + (hv ? 8 * nt + g : 0);
    const uint16_t *src = a.q + (static_cast<int64_t>(q_start + row / a.qpk) * a.hq + h * a.qpk +
                                 row % a.qpk) * D + t * 4;
#pragma unroll
    for (int gq = 0; gq < G; ++gq) {
      uint2 v[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
      if (hv) {
        v[0] = *reinterpret_cast<const uint2 *>(src + gq * 32);
        v[1] = *reinterpret_cast<const uint2 *>(src + gq * 32 + 16);
      }
      qb[nt][gq][0][0] = pack_half2(bf16_lo(v[0].x), bf16_hi(v[0].x));
      qb[nt][gq][0][1] = pack_half2(bf16_lo(v[0].y), bf16_hi(v[0].y));
      qb[nt][gq][1][0] = pack_half2(bf16_lo(v[1].x), bf16_hi(v[1].x));
      qb[nt][gq][1][1] = pack_half2(bf16_lo(v[1].y), bf16_hi(v[1].y));
      bad_q |= half2_nonfinite(qb[nt][gq][0][0]) || half2_nonfinite(qb[nt][gq][0][1]) ||
               half2_nonfinite(qb[nt][gq][1][0]) || half2_nonfinite(qb[nt][gq][1][1]);
    }
  }
  // q values beyond the fp16 range (|q| >= 65520) would give inf scores
  if (__any_sync(0xffffffffu, bad_q) && warp == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_Q);
  const int r0 = perm16(g);      // key (within a 16-key block) of score row g
  const int r1 = perm16(g + 8);  // ... of score row g + 8
  // where this lane's rows of the K matrices stand in a stage: score rows 0 - 7 and
  // 8 - 15 of a group's first 16 channels, then of its others (group gq: ^ 32 gq in
  // each 128 bytes); of the V matrices: channels 8m .. 8m + 7, 16 keys each
  const uint32_t k_lane = L::k_off(perm16((lane & 7) + (lane & 8)), lane & 16);
  const uint32_t v_lane = L::kVOff + lane * 16;
  // last visible key of a row of this pass
  auto limit = [&](int row) {
    return min(kv_end - 1, ctx + (row0 + min(row, n_rows - 1)) / a.qpk);
  };
  const int all_end = min(kv_end, limit(0) + 1);  // the first key past those every row sees

  // rows 8 nt + 2t, + 1: the max O and l are scaled to (log2 units), the same with 0
  // for -inf, this lane's expsum
  float m_run[NT][2], mu[NT][2], l_run[NT][2];
  bool started[NT];  // both rows have a max
  float o[NT][Cfg::kCm][4];          // O^T: channels (g, g+8) x rows (2t, 2t+1)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m_run[nt][0] = m_run[nt][1] = -INFINITY;
    mu[nt][0] = mu[nt][1] = 0.0f;
    started[nt] = false;
    l_run[nt][0] = l_run[nt][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < Cfg::kCm; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
  }

#pragma unroll 1
  for (int i = 0; i < n_blk; ++i) {
    cp_async_wait<kSt - 2>();
    __syncwarp();  // block i has landed for every lane, block i - 1 is read by every lane
    issue(i + kSt - 1);
    const uint32_t st = ring + (i % kSt) * L::kBytes;
    const int key0 = (b0 + kWarps * i) * 16;
    // keys outside [kv_begin, kv_end) in this block: masked, V zeroed (stale
    // bytes may sit there); keys past a row's own limit masked.  Formed on edge
    // blocks only.
    const bool tail = key0 + 16 > all_end || key0 < kv_begin;
    uint2 vmask = make_uint2(0xffffffffu, 0xffffffffu);
    if (tail) {
      const auto in = [&](int k) { return k >= kv_begin && k < kv_end; };
      const int kv = key0 + 4 * t;
      vmask.x = (in(kv) ? 0x0000ffffu : 0u) | (in(kv + 1) ? 0xffff0000u : 0u);
      vmask.y = (in(kv + 2) ? 0x0000ffffu : 0u) | (in(kv + 3) ? 0xffff0000u : 0u);
    }

    // ---------------- S^T = K Q^T: q8 with exact codes, scaled per group; fp8
    // keys exact in one accumulation
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
    if constexpr (F8) {
#pragma unroll
      for (int gq = 0; gq < G; ++gq) {
        uint32_t c[4];  // k-step 0: rows g, g + 8; k-step 1
        ldmatrix4(st + ((k_lane + (gq >> 2) * (16 * 128)) ^ ((gq & 3) * 32)), c);
        // bytes (0,1) -> k 2t, 2t+1; (2,3) -> k 2t+8, 2t+9, as codes4_to_half2
        const uint32_t a00 = e4m3x2_to_half2(c[0]), a02 = e4m3x2_to_half2(c[0] >> 16);
        const uint32_t a01 = e4m3x2_to_half2(c[1]), a03 = e4m3x2_to_half2(c[1] >> 16);
        const uint32_t a10 = e4m3x2_to_half2(c[2]), a12 = e4m3x2_to_half2(c[2] >> 16);
        const uint32_t a11 = e4m3x2_to_half2(c[3]), a13 = e4m3x2_to_half2(c[3] >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(s[nt], a00, a01, a02, a03, qb[nt][gq][0][0], qb[nt][gq][0][1]);
          mma_f16_16816(s[nt], a10, a11, a12, a13, qb[nt][gq][1][0], qb[nt][gq][1][1]);
        }
      }
    } else {
      float ks0[G], ks1[G];
      load_key_scales<G>(st + L::kKsOff + r0 * G * 2, ks0);
      load_key_scales<G>(st + L::kKsOff + r1 * G * 2, ks1);
#pragma unroll
      for (int gq = 0; gq < G; ++gq) {
        uint32_t c[4];
        ldmatrix4(st + ((k_lane + (gq >> 2) * (16 * 128)) ^ ((gq & 3) * 32)), c);
        uint32_t a00, a02, a01, a03, a10, a12, a11, a13;
        codes4_to_half2(c[0], a00, a02);  // row g, k-step 0: (k 2t,2t+1), (k 2t+8,2t+9)
        codes4_to_half2(c[1], a01, a03);  // row g+8
        codes4_to_half2(c[2], a10, a12);  // k-step 1
        codes4_to_half2(c[3], a11, a13);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float sg[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16_16816(sg, a00, a01, a02, a03, qb[nt][gq][0][0], qb[nt][gq][0][1]);
          mma_f16_16816(sg, a10, a11, a12, a13, qb[nt][gq][1][0], qb[nt][gq][1][1]);
          s[nt][0] = fmaf(sg[0], ks0[gq], s[nt][0]);
          s[nt][1] = fmaf(sg[1], ks0[gq], s[nt][1]);
          s[nt][2] = fmaf(sg[2], ks1[gq], s[nt][2]);
          s[nt][3] = fmaf(sg[3], ks1[gq], s[nt][3]);
        }
      }
    }

    // ---------------- mask the edges, online softmax over keys (rows of S^T)
    uint32_t pb[NT][2];
    const float mul = tail ? 1.0f : a.scale_log2;  // an edge block's scores are scaled as they are masked
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (tail) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = key0 + (e < 2 ? r0 : r1);
          s[nt][e] = k < kv_begin || k > limit(8 * nt + 2 * t + (e & 1)) ? -INFINITY
                                                                         : s[nt][e] * a.scale_log2;
        }
      }
      // P = 2^(s scale - m).  m is the largest score of the row's first block with a
      // visible key; it moves, and O and l with it, only when a P would pass 2^15
      // (inside fp16): no row maximum is taken on the common path.
      float p[4];
      auto exps = [&]() {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = fast_exp2(fmaf(s[nt][e], mul, -mu[nt][e & 1]));
      };
      exps();
      const bool fits = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])) <= kMaxP;
      if (!__all_sync(0xffffffffu, fits && started[nt])) {
        float mx[2], alpha[2];
        started[nt] = true;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[c] = fmaxf(s[nt][c] * mul, s[nt][2 + c] * mul);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
          const float mn = fmaxf(m_run[nt][c], mx[c]);
          started[nt] &= mn > -INFINITY;
          mu[nt][c] = mn == -INFINITY ? 0.0f : mn;
          alpha[c] = fast_exp2(m_run[nt][c] - mu[nt][c]);
          m_run[nt][c] = mn;
          l_run[nt][c] *= alpha[c];
        }
#pragma unroll
        for (int i = 0; i < Cfg::kCm; ++i) {
          o[nt][i][0] *= alpha[0];
          o[nt][i][1] *= alpha[1];
          o[nt][i][2] *= alpha[0];
          o[nt][i][3] *= alpha[1];
        }
        exps();
      }
      pb[nt][0] = movmatrix_trans(pack_half2(p[0], p[1]));  // keys 0..7 -> k 2t, 2t+1
      pb[nt][1] = movmatrix_trans(pack_half2(p[2], p[3]));  // keys 8..15 -> k 2t+8, 2t+9
      l_run[nt][0] += p[0] + p[2];
      l_run[nt][1] += p[1] + p[3];
    }

    // ---------------- O^T += V'^T P^T, V' = code * scale (fp8 / 4-bit: idx * scale
    // + zero) in fp16
    if constexpr (F8) {
      uint2 vsc = lds64(st + L::kKsOff + 8 * t);
      uint2 vzr = lds64(st + L::kVsOff + 8 * t);
      vsc.x &= vmask.x;
      vsc.y &= vmask.y;
      vzr.x &= vmask.x;
      vzr.y &= vmask.y;
#pragma unroll
      for (int cm = 0; cm < Cfg::kCm; ++cm) {
        const uint32_t w0 = lds16(st + L::kVOff + (cm * 16 + g) * 8 + 2 * t);
        const uint32_t w1 = lds16(st + L::kVOff + (cm * 16 + g + 8) * 8 + 2 * t);
        uint32_t a0, a2, a1, a3;
        nibbles4_to_half2(w0, a0, a2);  // channel g: keys 4t, 4t+1 | 4t+2, 4t+3
        nibbles4_to_half2(w1, a1, a3);  // channel g + 8
        a0 = hfma2_u32(a0, vsc.x, vzr.x);
        a2 = hfma2_u32(a2, vsc.y, vzr.y);
        a1 = hfma2_u32(a1, vsc.x, vzr.x);
        a3 = hfma2_u32(a3, vsc.y, vzr.y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16_16816(o[nt][cm], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    } else {
#pragma unroll
      for (int gv = 0; gv < G; ++gv) {
        uint2 vsc = lds64(st + L::kVsOff + (gv * 16 + 4 * t) * 2);
        vsc.x &= vmask.x;
        vsc.y &= vmask.y;
        uint32_t c[4];  // the group's 32 channels, 8 a matrix: keys 4t .. 4t + 3 of channel g
        ldmatrix4(st + v_lane + gv * (32 * 16), c);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int cm = gv * 2 + half;
          uint32_t a0, a2, a1, a3;
          codes4_to_half2(c[2 * half], a0, a2);      // channel g: keys 4t..4t+1 | 4t+2..4t+3
          codes4_to_half2(c[2 * half + 1], a1, a3);  // channel g + 8
          a0 = hmul2_u32(a0, vsc.x);
          a2 = hmul2_u32(a2, vsc.y);
          a1 = hmul2_u32(a1, vsc.x);
          a3 = hmul2_u32(a3, vsc.y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16_16816(o[nt][cm], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      }
    }
  }

  // expsum of each row: sum over the 8 lanes that share t
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        l_run[nt][c] += __shfl_xor_sync(0xffffffffu, l_run[nt][c], off);

  // ---------------- merge the 4 warps through shared memory (field-major), each
  // warp taking a quarter of the channels of every row, and write the triples
  constexpr int kFields = 4 + 4 * Cfg::kCm;
  constexpr int kMine = Cfg::kCm / kWarps;  // 16-channel blocks a warp merges
  cp_async_wait<0>();
  __syncthreads();  // every block consumed: reuse the rings
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float *dst = smem_f + (warp * NT + nt) * kFields * 32 + lane;
    dst[0] = m_run[nt][0];
    dst[32] = m_run[nt][1];
    dst[64] = l_run[nt][0];
    dst[96] = l_run[nt][1];
#pragma unroll
    for (int i = 0; i < Cfg::kCm; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(4 + i * 4 + e) * 32] = o[nt][i][e];
  }
  __syncthreads();
  const int64_t step = rows_total(sa) * 4;
#pragma unroll 1
  for (int nt = 0; nt < NT && 8 * nt < n_rows; ++nt) {
    const float *src = smem_f + nt * kFields * 32 + lane;
    constexpr int kNext = NT * kFields * 32;  // the next warp's
    float m[2], l[2], wt[kWarps][2], sum[kMine][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[c] = fmaxf(fmaxf(src[c * 32], src[kNext + c * 32]),
                   fmaxf(src[2 * kNext + c * 32], src[3 * kNext + c * 32]));
      const float mu = m[c] == -INFINITY ? 0.0f : m[c];
      l[c] = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        wt[k][c] = fast_exp2(src[k * kNext + c * 32] - mu);
        l[c] = fmaf(wt[k][c], src[k * kNext + (2 + c) * 32], l[c]);
      }
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sum[i][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
          sum[i][e] = fmaf(wt[k][e & 1], src[k * kNext + (4 + (warp * kMine + i) * 4 + e) * 32], sum[i][e]);
      }
    // lane (g, t) holds channels cm*16 + g (+8) of rows 8 nt + 2t, + 1
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * nt + 2 * t + c;
      if (row >= n_rows) continue;
      const int64_t r = static_cast<int64_t>(q_start) * a.qpk + row0 + row;
      float *dst = acc_at<D>(sa, sa.ns_p + sigma, h) + (warp * kMine * 4 + (g >> 2)) * step + r * 4 + (g & 3);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        dst[(i * 4) * step] = sum[i][c];
        dst[(i * 4 + 2) * step] = sum[i][2 + c];
      }
      if (warp == 0 && g == 0)
        *reinterpret_cast<float2 *>(a.part_ml + (ml_at(sa, sa.ns_p + sigma, h) + r) * 2) =
            make_float2(m[c], l[c]);
    }
  }
}

template <int D, int BS, bool F8, int NT>
static cudaError_t launch_shared_rows_t(const SharedArgs &s, cudaStream_t stream) {
  using Cfg = SharedRowsCfg<D, BS, F8, NT>;
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    cudaError_t r = cudaFuncSetAttribute(shared_rows_kernel<D, BS, F8, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    // all of the SM's shared memory, for four blocks
    return r != cudaSuccess ? r
                            : cudaFuncSetAttribute(shared_rows_kernel<D, BS, F8, NT>,
                                                   cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  if (e != cudaSuccess) return e;
  SharedArgs p = s;
  p.row_passes = (s.few_rows + 8 * NT - 1) / (8 * NT);
  const int64_t grid = static_cast<int64_t>(s.a.num_seqs) * s.ns_s * s.a.hk * p.row_passes;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_kernel(shared_rows_kernel<D, BS, F8, NT>, dim3(static_cast<unsigned>(grid)), 128,
                       Cfg::kSmem, stream, p);
}

template <int D, int BS>
static cudaError_t launch_shared_rows_d(const SharedArgs &s, bool f8v4, cudaStream_t stream) {
  if (rows_per_pass(D, s.few_rows) == 8)
    return f8v4 ? launch_shared_rows_t<D, BS, true, 1>(s, stream)
                : launch_shared_rows_t<D, BS, false, 1>(s, stream);
  if constexpr (D != 256)
    return f8v4 ? launch_shared_rows_t<D, BS, true, 2>(s, stream)
                : launch_shared_rows_t<D, BS, false, 2>(s, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_shared_rows(const SharedArgs &s, int d, int bs, bool f8v4, cudaStream_t stream) {
#define PAQ8_SHARED_CASE(DD, BB) \
  if (d == DD && bs == BB) return launch_shared_rows_d<DD, BB>(s, f8v4, stream);
  PAQ8_SHARED_CASE(64, 16)
  PAQ8_SHARED_CASE(64, 32)
  PAQ8_SHARED_CASE(128, 16)
  PAQ8_SHARED_CASE(128, 32)
  PAQ8_SHARED_CASE(256, 16)
  PAQ8_SHARED_CASE(256, 32)
#undef PAQ8_SHARED_CASE
  return cudaErrorInvalidValue;
}

}  // namespace paq8
