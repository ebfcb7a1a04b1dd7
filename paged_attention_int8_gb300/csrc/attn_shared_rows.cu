// Attention over a shared prefix: the suffix of sequences with at most 8 query
// rows per kv head (query tokens x q heads; a decode token of up to 8 heads, a
// few draft tokens of fewer), one key segment per block, in the swap-AB form
// of the decode kernel (attn_decode.cu): keys in the MMA's M dimension, rows in
// its N dimension,
//   S^T[16 keys x 8 rows] = K[16 x 16 ch] . Q^T[16 ch x 8],
//   O^T[16 ch x 8 rows] += V^T[16 ch x 16 keys] . P^T[16 keys x 8].
// Each row has its own causal limit, taken on edge blocks only.  HBM bound:
// 2 (D + D / 16) bytes a key and kv head (q8), D + D / 2 + 4 (fp8 / 4-bit).
//
// Four warps share a segment's 16-key blocks round robin, each on its own: it
// copies its blocks with 16-byte cp.async into a private 3-stage ring and reads
// them back, so that no warp waits for another until the four softmax states
// are merged at the end (one fp32 triple per row).  No producer warp, because
// four warps of at most 128 registers fit beside a block of the tensor-core
// kernel (its 16 warps leave 4096 registers of each SM sub-partition, one warp's;
// a fifth warp would double up on one): the prefix, bound by the tensor core, and
// the suffixes, bound by HBM, then share every SM from the start.
#include <type_traits>

#include "attn_shared.cuh"

namespace paq8 {

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
  // Byte b of key row r.  A lane of the MMA fragment (g, t) reads 8 bytes at 8t
  // of key perm16(g): the 16-byte pieces of a row are permuted so that the four
  // rows of a phase (0, 1, 4, 5 or 8, 9, 12, 13; 2 more for the second half)
  // stand in different banks.
  __device__ static __forceinline__ uint32_t k_off(int r, int b) {
    if constexpr (D >= 128) {
      const int i = (r & 1) | ((r >> 2) << 1);
      const int off = r * 128 + (b & 127);
      return (b >> 7) * (16 * 128) + (off ^ ((((i & 3) << 1) | (i >> 2)) << 4));
    } else {
      const int off = r * 64 + b;
      return off ^ (((r >> 2) & 1) << 5);
    }
  }
};

template <int D, int BS, bool F8>
struct SharedRowsCfg {
  using L = RowsStage<D, F8>;
  static constexpr int kWarps = 4;
  static constexpr int kSt = 3;
  static constexpr int kCm = D / 16;                    // 16-channel blocks of the output
  static constexpr int G = D / 32;
  static constexpr int kMinBlocks = D == 256 ? 2 : 4;   // blocks per SM
  static constexpr int kRing = kWarps * kSt * L::kBytes;
  static constexpr int kMerge = (kWarps - 1) * 32 * (4 + 4 * kCm) * 4;
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

template <int D, int BS, bool F8>
__global__ void __launch_bounds__(128, SharedRowsCfg<D, BS, F8>::kMinBlocks)
    shared_rows_kernel(const __grid_constant__ SharedArgs sa) {
  using Cfg = SharedRowsCfg<D, BS, F8>;
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
  const int sigma = rest / a.num_seqs;

  launch_dependents();
  const LastBlockWaits at_end{blockIdx.x == gridDim.x - 1};
  const int q_start = a.cu_seqlens_q[seq];
  const int q_len = a.cu_seqlens_q[seq + 1] - q_start;
  const int n_rows = rows_of(sa, q_len);
  if (q_len <= 0) return;
  if (n_rows > kFewRows) {  // shared_mma_kernel's, where it runs
    if (n_rows > sa.max_rows && sigma == 0 && h == 0 && threadIdx.x == 0)
      flag_status(a.status, PA_DEV_BAD_SEQ);  // max_query_len was below a q_len
    return;
  }
  const int seq_len = a.seq_lens[seq];
  const int ctx = seq_len - q_len;
  const int P = prefix_of(sa, seq, lane);
  if (q_start < 0 || q_start + q_len > a.num_tokens || P < 0 || ctx < P) {
    if (threadIdx.x == 0 && sigma == 0) flag_status(a.status, PA_DEV_BAD_SEQ);
    return;
  }
  SharedWork w;
  if (!segment_keys(P, seq_len, sa.seg_s, sa.ns_s, sigma, w)) return;
  const int kv_begin = w.kv_begin, kv_end = w.kv_end;
  // this warp's 16-key blocks: b0, b0 + 4, ...
  const int b0 = kv_begin / 16 + warp;
  const int n_blk = max(0, ((kv_end + 15) / 16 - b0 + kWarps - 1) / kWarps);
  const uint32_t ring = smem_base + warp * (kSt * L::kBytes);
  const int32_t *bt_row = a.block_table + static_cast<int64_t>(seq) * a.bt_stride;
  int held = -1;  // block id of this lane's block: number (i / 32) * 32 + lane of this warp's
  // block ids of the warp's blocks i .. i + 31 (-1: a bad entry, flagged and masked by no copy)
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

  // Q^T as the B operand: lane (g, t) holds row g, channels 32gq + 8t + 4s +
  // {0,1} (k = 2t, 2t+1) and + {2,3} (k = 2t+8, 2t+9) for k-step s.
  uint32_t qb[G][2][2];
  {
    const int row = g < n_rows ? g : 0;
    const bool hv = g < n_rows;
    const uint16_t *src = a.q + (static_cast<int64_t>(q_start + row / a.qpk) * a.hq + h * a.qpk +
                                 row % a.qpk) * D + t * 8;
    bool bad_q = false;
#pragma unroll
    for (int gq = 0; gq < G; ++gq) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (hv) v = *reinterpret_cast<const uint4 *>(src + gq * 32);
      qb[gq][0][0] = pack_half2(bf16_lo(v.x), bf16_hi(v.x));
      qb[gq][0][1] = pack_half2(bf16_lo(v.y), bf16_hi(v.y));
      qb[gq][1][0] = pack_half2(bf16_lo(v.z), bf16_hi(v.z));
      qb[gq][1][1] = pack_half2(bf16_lo(v.w), bf16_hi(v.w));
      bad_q |= half2_nonfinite(qb[gq][0][0]) || half2_nonfinite(qb[gq][0][1]) ||
               half2_nonfinite(qb[gq][1][0]) || half2_nonfinite(qb[gq][1][1]);
    }
    // q values beyond the fp16 range (|q| >= 65520) would give inf scores
    if (__any_sync(0xffffffffu, bad_q) && warp == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_Q);
  }
  const int r0 = perm16(g);      // key (within a 16-key block) of score row g
  const int r1 = perm16(g + 8);  // ... of score row g + 8
  // last visible keys of this lane's two rows, and the first key past the
  // block that every row sees
  const int lim0 = min(kv_end - 1, ctx + min(2 * t, n_rows - 1) / a.qpk);
  const int lim1 = min(kv_end - 1, ctx + min(2 * t + 1, n_rows - 1) / a.qpk);
  const int all_end = min(kv_end, ctx + 1);

  float m_run[2] = {-INFINITY, -INFINITY};  // rows 2t, 2t+1 (log2 units)
  float l_run[2] = {0.0f, 0.0f};            // this lane's share of the expsum
  float o[Cfg::kCm][4];                     // O^T: channels (g, g+8) x rows (2t, 2t+1)
#pragma unroll
  for (int i = 0; i < Cfg::kCm; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

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
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    {
      const int k0 = r0, k1 = r1;
      if constexpr (F8) {
#pragma unroll
        for (int gq = 0; gq < G; ++gq) {
          const uint2 c0 = lds64(st + L::k_off(k0, gq * 32 + t * 8));
          const uint2 c1 = lds64(st + L::k_off(k1, gq * 32 + t * 8));
          // bytes (0,1) -> k 2t, 2t+1; (2,3) -> k 2t+8, 2t+9, as codes4_to_half2
          const uint32_t a00 = e4m3x2_to_half2(c0.x), a02 = e4m3x2_to_half2(c0.x >> 16);
          const uint32_t a01 = e4m3x2_to_half2(c1.x), a03 = e4m3x2_to_half2(c1.x >> 16);
          const uint32_t a10 = e4m3x2_to_half2(c0.y), a12 = e4m3x2_to_half2(c0.y >> 16);
          const uint32_t a11 = e4m3x2_to_half2(c1.y), a13 = e4m3x2_to_half2(c1.y >> 16);
          mma_f16_16816(s, a00, a01, a02, a03, qb[gq][0][0], qb[gq][0][1]);
          mma_f16_16816(s, a10, a11, a12, a13, qb[gq][1][0], qb[gq][1][1]);
        }
      } else {
        float ks0[G], ks1[G];
        load_key_scales<G>(st + L::kKsOff + k0 * G * 2, ks0);
        load_key_scales<G>(st + L::kKsOff + k1 * G * 2, ks1);
#pragma unroll
        for (int gq = 0; gq < G; ++gq) {
          const uint2 c0 = lds64(st + L::k_off(k0, gq * 32 + t * 8));
          const uint2 c1 = lds64(st + L::k_off(k1, gq * 32 + t * 8));
          uint32_t a00, a02, a01, a03, a10, a12, a11, a13;
          codes4_to_half2(c0.x, a00, a02);  // row g, k-step 0: (k 2t,2t+1), (k 2t+8,2t+9)
          codes4_to_half2(c1.x, a01, a03);  // row g+8
          codes4_to_half2(c0.y, a10, a12);  // k-step 1
          codes4_to_half2(c1.y, a11, a13);
          float sg[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16_16816(sg, a00, a01, a02, a03, qb[gq][0][0], qb[gq][0][1]);
          mma_f16_16816(sg, a10, a11, a12, a13, qb[gq][1][0], qb[gq][1][1]);
          s[0] = fmaf(sg[0], ks0[gq], s[0]);
          s[1] = fmaf(sg[1], ks0[gq], s[1]);
          s[2] = fmaf(sg[2], ks1[gq], s[2]);
          s[3] = fmaf(sg[3], ks1[gq], s[3]);
        }
      }
    }

    // ---------------- mask the tail, online softmax over keys (rows)
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = s[e] * a.scale_log2;
      if (tail) {
        const int k = key0 + (e < 2 ? r0 : r1);
        if (k < kv_begin || k > ((e & 1) ? lim1 : lim0)) v = -INFINITY;
      }
      s[e] = v;
      mx[e & 1] = fmaxf(mx[e & 1], v);
    }
    float alpha[2], mu[2];
    bool grew = false;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], off));
      const float mn = fmaxf(m_run[c], mx[c]);
      grew |= mn != m_run[c];
      mu[c] = mn == -INFINITY ? 0.0f : mn;
      alpha[c] = fast_exp2(m_run[c] - mu[c]);
      m_run[c] = mn;
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = fast_exp2(s[e] - mu[e & 1]);
    const uint32_t pb0 = movmatrix_trans(pack_half2(p[0], p[1]));  // keys 0..7 -> k 2t, 2t+1
    const uint32_t pb1 = movmatrix_trans(pack_half2(p[2], p[3]));  // keys 8..15 -> k 2t+8, 2t+9
    // rescale only when some row's running max moved (alpha == 1 otherwise)
    if (__any_sync(0xffffffffu, grew)) {
      l_run[0] *= alpha[0];
      l_run[1] *= alpha[1];
#pragma unroll
      for (int i = 0; i < Cfg::kCm; ++i) {
        o[i][0] *= alpha[0];
        o[i][1] *= alpha[1];
        o[i][2] *= alpha[0];
        o[i][3] *= alpha[1];
      }
    }
    l_run[0] += p[0] + p[2];
    l_run[1] += p[1] + p[3];

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
        mma_f16_16816(o[cm], a0, a1, a2, a3, pb0, pb1);
      }
    } else {
#pragma unroll
      for (int gv = 0; gv < G; ++gv) {
        uint2 vsc = lds64(st + L::kVsOff + (gv * 16 + 4 * t) * 2);
        vsc.x &= vmask.x;
        vsc.y &= vmask.y;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int cm = gv * 2 + half;
          const uint32_t w0 = lds32(st + L::kVOff + (cm * 16 + g) * 16 + 4 * t);
          const uint32_t w1 = lds32(st + L::kVOff + (cm * 16 + g + 8) * 16 + 4 * t);
          uint32_t a0, a2, a1, a3;
          codes4_to_half2(w0, a0, a2);  // channel g: keys 4t..4t+1 | 4t+2..4t+3
          codes4_to_half2(w1, a1, a3);  // channel g + 8
          a0 = hmul2_u32(a0, vsc.x);
          a2 = hmul2_u32(a2, vsc.y);
          a1 = hmul2_u32(a1, vsc.x);
          a3 = hmul2_u32(a3, vsc.y);
          mma_f16_16816(o[cm], a0, a1, a2, a3, pb0, pb1);
        }
      }
    }
  }

  // expsum of each row: sum over the 8 lanes that share t
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l_run[c] += __shfl_xor_sync(0xffffffffu, l_run[c], off);

  // ---------------- merge the 4 warps (field-major through shared memory)
  constexpr int kFields = 4 + 4 * Cfg::kCm;
  cp_async_wait<0>();
  __syncthreads();  // every block consumed: reuse the rings
  if (warp > 0) {
    float *dst = smem_f + (warp - 1) * kFields * 32 + lane;
    dst[0] = m_run[0];
    dst[32] = m_run[1];
    dst[64] = l_run[0];
    dst[96] = l_run[1];
#pragma unroll
    for (int i = 0; i < Cfg::kCm; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(4 + i * 4 + e) * 32] = o[i][e];
  }
  __syncthreads();
  if (warp > 0) return;
#pragma unroll 1
  for (int k = 0; k < kWarps - 1; ++k) {
    const float *src = smem_f + k * kFields * 32 + lane;
    float wa[2], wb[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float mo = src[c * 32];
      const float mn = fmaxf(m_run[c], mo);
      const float muv = mn == -INFINITY ? 0.0f : mn;
      wa[c] = fast_exp2(m_run[c] - muv);
      wb[c] = fast_exp2(mo - muv);
      m_run[c] = mn;
      l_run[c] = l_run[c] * wa[c] + src[(2 + c) * 32] * wb[c];
    }
#pragma unroll
    for (int i = 0; i < Cfg::kCm; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[i][e] = o[i][e] * wa[e & 1] + src[(4 + i * 4 + e) * 32] * wb[e & 1];
  }

  // ---------------- write the triples: lane (g, t) holds channels cm*16 + g (+8)
  // of rows 2t, 2t+1
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int row = 2 * t + c;
    if (row >= n_rows) continue;
    const int64_t r = static_cast<int64_t>(q_start) * a.qpk + row, step = rows_total(sa) * 4;
    float *dst = acc_at<D>(sa, sa.ns_p + sigma, h) + (g >> 2) * step + r * 4 + (g & 3);
#pragma unroll
    for (int cm = 0; cm < Cfg::kCm; ++cm) {
      dst[(cm * 4) * step] = o[cm][c];
      dst[(cm * 4 + 2) * step] = o[cm][2 + c];
    }
    if (g == 0)
      *reinterpret_cast<float2 *>(a.part_ml + (ml_at(sa, sa.ns_p + sigma, h) + r) * 2) =
          make_float2(m_run[c], l_run[c]);
  }
}

template <int D, int BS, bool F8>
static cudaError_t launch_shared_rows_t(const SharedArgs &s, cudaStream_t stream) {
  using Cfg = SharedRowsCfg<D, BS, F8>;
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    cudaError_t r = cudaFuncSetAttribute(shared_rows_kernel<D, BS, F8>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    // the tensor-core kernel's carveout, so that blocks of both are resident together
    return r != cudaSuccess ? r
                            : cudaFuncSetAttribute(shared_rows_kernel<D, BS, F8>,
                                                   cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  });
  if (e != cudaSuccess) return e;
  const int64_t grid = static_cast<int64_t>(s.a.num_seqs) * s.ns_s * s.a.hk;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_kernel(shared_rows_kernel<D, BS, F8>, dim3(static_cast<unsigned>(grid)), 128,
                       Cfg::kSmem, stream, true, s);
}

cudaError_t launch_shared_rows(const SharedArgs &s, int d, int bs, bool f8v4, cudaStream_t stream) {
#define PAQ8_SHARED_CASE(DD, BB)                                           \
  if (d == DD && bs == BB)                                                 \
    return f8v4 ? launch_shared_rows_t<DD, BB, true>(s, stream)            \
                : launch_shared_rows_t<DD, BB, false>(s, stream);
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
