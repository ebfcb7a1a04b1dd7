// Attention over a shared prefix: the suffix of sequences with at most 8 query
// rows per kv head (query tokens x q heads; a decode token of up to 8 heads, a
// few draft tokens of fewer), one key segment per block, in the swap-AB form
// of the decode kernel (attn_decode.cu): keys in the MMA's M dimension, rows in
// its N dimension,
//   S^T[16 keys x 8 rows] = K[16 x 16 ch] . Q^T[16 ch x 8],
//   O^T[16 ch x 8 rows] += V^T[16 ch x 16 keys] . P^T[16 keys x 8],
// four consumer warps on the 16-key blocks of each 64-key tile (32-key tiles
// at D = 256, pairs of warps on alternate tiles) with private softmax states
// merged at the end, one producer warp copying pages with 16-byte cp.async
// into a 3-stage ring (4 at D = 256). Each row has its own causal limit, taken
// on edge tiles only. HBM bound: 2 (D + D / 16) bytes a key and kv head (q8),
// D + D / 2 + 4 (fp8 / 4-bit); each block leaves one fp32 triple per row.
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

template <int D, int BS, bool F8>
struct SharedRowsCfg {
  static constexpr int kTile = D == 256 ? 32 : 64;
  using L = std::conditional_t<F8, StageF8V4<D, BS, kTile>, StageLayout<D, BS, kTile>>;
  static constexpr int kMt = kTile / 16;   // 16-key blocks per tile
  static constexpr int kWpt = kMt < kConsumerWarps ? kMt : kConsumerWarps;  // warps per tile
  static constexpr int kKg = kConsumerWarps / kWpt;  // tile groups (alternate tiles)
  static constexpr int kCm = D / 16;       // 16-channel blocks of the output
  static constexpr int G = D / 32;
  static constexpr int kSt = D == 256 ? 4 : 3;          // ring stages
  static constexpr int kMinBlocks = D == 256 ? 2 : 4;   // blocks per SM
  static constexpr int kSmem = kSt * L::kBytes + 2 * kSt * 8 + 1024;
};

template <int D, int BS, bool F8>
__global__ void __launch_bounds__(kThreads, SharedRowsCfg<D, BS, F8>::kMinBlocks)
    shared_rows_kernel(const __grid_constant__ SharedArgs sa) {
  using Cfg = SharedRowsCfg<D, BS, F8>;
  using L = typename Cfg::L;
  constexpr int G = Cfg::G;
  constexpr int kTile = Cfg::kTile;
  constexpr int kWpt = Cfg::kWpt;
  constexpr int kKg = Cfg::kKg;
  constexpr int kStages = Cfg::kSt;
  static_assert(kStages % kKg == 0, "a stage always feeds the same tile group");
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
  const int tile_lo = kv_begin / kTile;
  const int n_iter = (kv_end + kTile - 1) / kTile - tile_lo;

  constexpr int kMergeBytes = 3 * 32 * (4 + 4 * Cfg::kCm) * 4;
  constexpr int kRingBytes = kStages * L::kBytes;
  static_assert(kMergeBytes <= kRingBytes, "merge area fits in the ring");
  const uint32_t bar_full = smem_base + kRingBytes;
  const uint32_t bar_empty = bar_full + kStages * 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full + 8 * i, 32);    // one arrival per producer lane
      mbar_init(bar_empty + 8 * i, kWpt);  // every warp of the tile group reads it
    }
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    if constexpr (F8)
      produce_f8v4<L, BS, kStages>(a, smem_base, bar_full, bar_empty, seq, h, tile_lo, n_iter,
                                   kv_begin, kv_end, lane);
    else
      produce_tiles_lsu<L, BS, kStages>(a, smem_base, bar_full, bar_empty, seq, h, tile_lo,
                                        n_iter, kv_begin, kv_end, lane);
    return;
  }

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

  // Warp w takes the 16-key block mt = w % kWpt of every tile of its tile
  // group (w / kWpt): all warps read every stage, so the whole ring is in
  // flight for each of them.
  const int my_mt = warp % kWpt;
  const int kg = warp / kWpt;
  bool timed_out = false;
  for (int it = kg; it < n_iter; it += kKg) {
    const int stage = it % kStages;
    if (!mbar_wait(bar_full + 8 * stage, (it / kStages) & 1, a.wait_limit_ns)) {
      timed_out = true;
      break;
    }
    const uint32_t st = smem_base + stage * L::kBytes;
    const int key0 = (tile_lo + it) * kTile + my_mt * 16;  // first key of this warp's block
    // keys outside [kv_begin, kv_end) in this block: masked, V zeroed (stale
    // bytes may sit there); keys past a row's own limit masked.  Formed on edge
    // tiles only.
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
      const int k0 = my_mt * 16 + r0, k1 = my_mt * 16 + r1;
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
        load_key_scales<G>(st + L::ks_off(k0, 0), ks0);
        load_key_scales<G>(st + L::ks_off(k1, 0), ks1);
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
      uint2 vsc = lds64(st + L::vs_off(my_mt * 16 + 4 * t));
      uint2 vzr = lds64(st + L::vz_off(my_mt * 16 + 4 * t));
      vsc.x &= vmask.x;
      vsc.y &= vmask.y;
      vzr.x &= vmask.x;
      vzr.y &= vmask.y;
#pragma unroll
      for (int cm = 0; cm < Cfg::kCm; ++cm) {
        const uint32_t w0 = lds16(st + L::v_off(cm * 16 + g, my_mt * 16 + 4 * t));
        const uint32_t w1 = lds16(st + L::v_off(cm * 16 + g + 8, my_mt * 16 + 4 * t));
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
        uint2 vsc = lds64(st + L::vs_off(my_mt * 16 + 4 * t, gv));
        vsc.x &= vmask.x;
        vsc.y &= vmask.y;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int cm = gv * 2 + half;
          const uint32_t w0 = lds32(st + L::v_off(cm * 16 + g, my_mt * 16 + 4 * t));
          const uint32_t w1 = lds32(st + L::v_off(cm * 16 + g + 8, my_mt * 16 + 4 * t));
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
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_empty + 8 * stage);
  }
  if (timed_out && lane == 0) flag_status(a.status, PA_DEV_TIMEOUT);

  // expsum of each row: sum over the 8 lanes that share t
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l_run[c] += __shfl_xor_sync(0xffffffffu, l_run[c], off);

  // ---------------- merge the 4 warps (field-major through shared memory)
  constexpr int kFields = 4 + 4 * Cfg::kCm;
  named_barrier(1, kConsumerWarps * 32);  // every stage consumed: reuse the ring
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
  named_barrier(1, kConsumerWarps * 32);
  if (warp > 0) return;
#pragma unroll 1
  for (int k = 0; k < kConsumerWarps - 1; ++k) {
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
    return cudaFuncSetAttribute(shared_rows_kernel<D, BS, F8>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t grid = static_cast<int64_t>(s.a.num_seqs) * s.ns_s * s.a.hk;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_kernel(shared_rows_kernel<D, BS, F8>, dim3(static_cast<unsigned>(grid)), kThreads,
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
