// Attention over the 4-bit cache (q4.cuh): for query row i of a sequence (a token and a
// q head), over its visible keys j,
//   s_j = scale * q . k_j,  out = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - m),
//   lse = m + ln sum_j p_j,   with k_j, v_j = code * scale + zero per 32 channels.
//
// Bound by HBM for single tokens: 5/4 D bytes a (key, kv head).  Everything is read
// once by warps whose lanes hold the codes of their MMA fragments, and no code is
// turned into a number by arithmetic: a nibble masked out of its word is, as fp16, the
// subnormal code * 2^-24 (or 16 code * 2^-24 for the upper nibble of a byte), exact in
// the tensor cores, and the powers of two leave in fp32.
//   Scores  S^T[16 keys x 8 rows] = K[16 x 16 ch] Q^T[16 ch x 8 rows], keys in the
//     MMA's M dimension.  Per group s_g sum q c is scaled in fp32; the zeros' part
//     sum_g z_g (sum q)_g is one more MMA over the groups, with the q sums as two fp16
//     parts (22 bits; q is a row's, formed once).  No rounding but q's to fp16, in a power of
//     two of a block's largest (query_scale).
//   Output  O^T[16 ch x 8 rows] += V^T P^T, where the key's scale goes into P: per
//     group P_g = fp16(p s_g), so that the codes again enter as they are; the zeros'
//     part is one more MMA (groups in M).  p and p s_g are rounded to fp16 (2^-11).
// The maximum that p is taken against moves only when a score passes it by 2^2: one
// vote a block of keys instead of a reduction.  p is lifted by 2^10, so that small
// weights of small scales stay out of fp16's subnormals (p s_g is normal from 6e-8
// on); with s_g of 16 and more, ranges above 240, the product can leave fp16, whose
// infinity then stands in the sums: such a warp goes over its keys again without the
// lift (p s_g is at most 4 s_g), and where that is too much, from s_g 16376 on, a third
// time with p at most 1.
//
// A thread block takes 8 NB rows (tokens x the q heads of a kv head) and a segment of
// the keys; its four warps work on their own 16-key blocks, each with its own ring of
// asynchronous copies, and join their sums at the end.  Segments leave fp32 triples
// that q4_join_kernel merges.  Long queries go to attn_q4_tc.cu (on_tc below).
#include <algorithm>
#include <utility>

#include "attn_common.cuh"
#include "attn_q4.cuh"
#include "launch.h"
#include "programmatic.cuh"
#include "q4.cuh"
#include "q4.h"
#include "segments.cuh"

namespace paq8 {

namespace {

using namespace q4;

constexpr int kWarps = 4;
constexpr float kMargin = 2.0f;  // log2 of the largest p over that of the maximum
constexpr float kLift = 10.0f;   // log2 of p at the maximum

// Ring depth by the bytes of a 16-key block (20 D): what keeps about 100 KB an SM in flight.
constexpr int ring_stages(int d) { return d == 256 ? 4 : 6; }
template <int D>
struct Q4Cfg {
  static constexpr int G = D / 32;
  static constexpr int kRow = D / 2;                 // bytes of a row's codes
  static constexpr int kKs = 16 * kRow;              // K scales [16][G], zeros [16][G]
  static constexpr int kV = kKs + 16 * G * 4;        // V codes
  static constexpr int kVs = kV + 16 * kRow;         // V scales [G][16], zeros [G][16]
  static constexpr int kBlock = kVs + 16 * G * 4;    // 20 D bytes
  static constexpr int kStages = ring_stages(D);
};

// D = A B, m16n8k16, fp16 inputs, fp32 accumulators, no addend.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ float half_lo(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}
__device__ __forceinline__ float half_hi(uint32_t w) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16)));
}

__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// N 32-bit words from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds32(addr);
  } else if constexpr (N == 2) {
    const uint2 v = lds64(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = lds128(addr + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  }
}

// Where 16-byte chunk c of key r's codes lies in a staged block.  K rows stand in
// the order of the score MMA's rows, V rows in the order in which the four lanes of
// a channel row read them, so that the rows of one load are neighbours; chunks of
// wider rows are exchanged so that the lanes of one phase meet no bank twice.
template <int D>
__device__ __forceinline__ uint32_t k_place(int r, int c) {
  const int row = (r >> 2) * 2 + (r & 1) + ((r >> 1) & 1) * 8;  // inverse of perm16
  return row * (D / 2) + ((D == 256 ? c ^ (row & 1) : c) * 16);
}
template <int D>
__device__ __forceinline__ uint32_t v_place(int r, int c) {
  const int t = r >> 2, i = r & 3;
  const int x = D == 256 ? 2 * t : D == 128 ? (t >> 1) * 2 : 0;
  return (i * 4 + t) * (D / 2) + (c ^ x) * 16;
}

// Thread blocks an SM: what the registers allow, and the rings (of the 228 KB of an SM's shared
// memory, of which a block takes 1 KB more than its own): two at D 256.
constexpr int resident_blocks(int d, bool wide) {
  const int by_registers = wide ? 2 : d == 64 ? 5 : 3;
  const int by_rings = 228 * 1024 / (kWarps * ring_stages(d) * 20 * d + 1024);
  return by_registers < by_rings ? by_registers : by_rings;
}
// Two blocks of keys at a time where that pays: the chain from a block's scores to its products
// is long, and a second one fills its gaps (D 128, 32 sequences x 6000 keys, 3 x 4 rows: 39 us, 50
// with one at three thread blocks an SM).  At D 64 the registers of 16 rows are better spent
// otherwise (64 x 4096 keys, 16 q heads a kv head: 23 us, 27 with two); at D 256 one block of keys
// takes 232 of 255.
constexpr int keys_blocks(int d, bool wide) { return d == 128 || (d == 64 && !wide) ? 2 : 1; }

template <int D, int BS, int NB>
__global__ void __launch_bounds__(kWarps * 32, resident_blocks(D, NB == 2)) attn_q4_kernel(const __grid_constant__ Q4Args a) {
  using C = Q4Cfg<D>;
  constexpr int G = C::G;
  constexpr int KB = keys_blocks(D, NB == 2);  // blocks of keys in work together
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  wait_for_predecessor();
  launch_dependents();  // the join waits for all of this grid
  const int item = blockIdx.x, h = blockIdx.y, sigma = blockIdx.z;
  // r / qpk of a row r < 128 of the block
  const auto token_of = [&](int r) { return (r * a.qpk_inverse) >> 16; };

  // ---- which rows, which keys
  int seq = item, tok0 = 0;
  if (a.p.max_query_len > 1) {
    seq = find_seq(a.p.cu, a.p.num_seqs, a.block_tokens, item, lane);
    const int c0 = a.p.cu[seq];
    tok0 = (item - ((a.block_tokens == 1 ? c0 : c0 / a.block_tokens + seq))) * a.block_tokens;
  }
  const int q0 = a.p.cu[seq];
  const int q_len = a.p.cu[seq + 1] - q0;
  const int seq_len = a.p.seq_lens[seq];
  if (tok0 < 0 || tok0 >= q_len || !valid_sequence(a, q0, q_len, seq_len)) {
    if (threadIdx.x == 0) flag_bad_sequences(a, item, h, sigma);
    return;
  }
  const KeyRange range = key_range(a, seq_len, q_len, tok0);
  if (seq_len > int64_t{a.p.table_columns} * BS && sigma == 0 && threadIdx.x == 0)
    flag_status(a.status, PA_DEV_BAD_BLOCK);
  if (sigma > 0 && a.seg_start[sigma] >= range.blocks) return;  // (as segments() counts)
  const int n_rows = min(a.block_tokens, q_len - tok0) * a.qpk;
  const int seg0 = range.first + a.seg_start[sigma];
  const int seg1 = sigma == a.num_splits - 1 ? range.first + range.blocks
                                             : min(range.first + range.blocks, range.first + a.seg_start[sigma + 1]);

  // ---- q as the B operand: lane (g, t) holds row 8 nb + g
  //   group gr, step e: channels 32 gr + 8 t + 2 e' of the nibbles that step e's words
  //   hold: step 0 nibbles (0, 4 | 1, 5), step 1 nibbles (2, 6 | 3, 7); the second pair
  //   of each meets codes of weight 16 and is divided by it
  uint32_t qb[NB][G][2][2];
  uint32_t qs[NB][2];  // sums over groups 2t, 2t + 1 of row g: fp16 high and low parts
  int lim[NB][2], lo[NB][2];  // visible keys of rows 8 nb + 2t, + 1
  int min_lim = 0x7fffffff, max_lo = 0;
  bool bad_q = false;
  uint4 raw[NB][G];
  float largest = 0.0f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int row = nb * 8 + g;
    const bool real = row < n_rows;
    const int tr = real ? token_of(row) : 0;
    const uint16_t *src = a.p.q + (static_cast<int64_t>(q0 + tok0 + tr) * a.p.hq + h * a.qpk +
                                   (real ? row - tr * a.qpk : 0)) * D;
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      raw[nb][gr] = make_uint4(0u, 0u, 0u, 0u);
      if (real) raw[nb][gr] = *reinterpret_cast<const uint4 *>(src + gr * 32 + t * 8);
    }
  }

  // ---- this warp's copies: block b of the segment for b % 4 == warp
  const uint32_t ring = smem_u32(smem_raw) + warp * (C::kStages * C::kBlock);
  const int n_mine = (seg1 - seg0 - warp + kWarps - 1) / kWarps;  // may be <= 0
  constexpr int kPer = 16 * C::kRow / 16 / 32;    // code chunks a lane, of K and of V
  constexpr int kScChunks = 16 * G * 2 / 16;      // of one plane of scales or zeros
  constexpr int kScPer = (4 * kScChunks + 31) / 32;
  constexpr int kPlane = BS * G * 2;              // bytes of a page's plane
  constexpr int kRowChunks = C::kRow / 16;
  const int32_t *table = a.p.block_table + static_cast<int64_t>(seq) * a.p.table_stride;
  // this lane's chunks: where they stand in a page, and where they go in a stage
  const uint8_t *k_src = a.p.k_cache + static_cast<int64_t>(h) * BS * C::kRow + lane * 16;
  const uint8_t *v_src = a.p.v_cache + static_cast<int64_t>(h) * BS * C::kRow + lane * 16;
  const int64_t code_page = static_cast<int64_t>(a.p.hk) * BS * C::kRow;
  const int64_t scale_page = static_cast<int64_t>(a.p.hk) * 2 * kPlane;
  uint32_t k_dst[kPer], v_dst[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int c = k * 32 + lane;
    k_dst[k] = k_place<D>(c / kRowChunks, c % kRowChunks);
    v_dst[k] = C::kV + v_place<D>(c / kRowChunks, c % kRowChunks);
  }
  const uint8_t *sc_src[kScPer];  // planes: K scales, K zeros, V scales, V zeros
  uint32_t sc_dst[kScPer], sc_half[kScPer];  // sc_half: to the page's second 16 keys
#pragma unroll
  for (int k = 0; k < kScPer; ++k) {
    const int c = k * 32 + lane, plane = (c / kScChunks) & 1, x = c % kScChunks;
    const bool keys = c < 2 * kScChunks;
    sc_src[k] = reinterpret_cast<const uint8_t *>(keys ? a.p.k_scale : a.p.v_scale) +
                static_cast<int64_t>(h) * 2 * kPlane + plane * kPlane +
                (keys ? x * 16 : (x >> 1) * (BS * 2) + (x & 1) * 16);
    sc_dst[k] = keys ? C::kKs + c * 16 : C::kVs + (c - 2 * kScChunks) * 16;
    sc_half[k] = keys ? 16 * G * 2 : 32;
  }
  int entries = -1;  // page of this warp's block (32 i + lane), refilled every 32 blocks
  auto refill = [&](int i) {
    const int b = seg0 + warp + (i + lane) * kWarps;
    entries = -1;
    if (i + lane < n_mine) {
      const int e = table[b * 16 / BS];
      if (e >= 0 && e < a.p.num_blocks) entries = e;
      else flag_status(a.status, PA_DEV_BAD_BLOCK);
    }
  };
  uint32_t live = 0;  // bit s: stage s holds a block of a valid page
  auto issue = [&](int i) {  // copies of this warp's i-th block
    if ((i & 31) == 0 && i < n_mine) refill(i);
    const int e = __shfl_sync(0xffffffffu, entries, i & 31);
    const int stage = i % C::kStages;
    live &= ~(1u << stage);
    if (i < n_mine && e >= 0) {
      live |= 1u << stage;
      const uint32_t st = ring + stage * C::kBlock;
      const int second = BS == 32 ? (seg0 + warp + i * kWarps) & 1 : 0;  // half of the page
      const int64_t code = e * code_page + second * (16 * C::kRow), scale = e * scale_page;
#pragma unroll
      for (int k = 0; k < kPer; ++k) cp_async_16(st + k_dst[k], k_src + code + k * 512);
#pragma unroll
      for (int k = 0; k < kPer; ++k) cp_async_16(st + v_dst[k], v_src + code + k * 512);
#pragma unroll
      for (int k = 0; k < kScPer; ++k)
        if (4 * kScChunks % 32 == 0 || k * 32 + lane < 4 * kScChunks)
          cp_async_16(st + sc_dst[k], sc_src[k] + scale + second * sc_half[k]);
    }
    cp_async_commit();
  };
  // the first copies go out while q is on its way
#pragma unroll
  for (int i = 0; i < C::kStages - KB; ++i) issue(i);

#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int gr = 0; gr < G; ++gr) largest = fmaxf(largest, largest_of(raw[nb][gr]));
  const QueryScale by = query_scale(warp_largest(largest), a.scale_log2);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float sums[G];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      const uint4 v = raw[nb][gr];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]) * by.up;
        x[2 * i + 1] = bf16_hi(w[i]) * by.up;
        bad_q |= half2_nonfinite(pack_half2(x[2 * i], x[2 * i + 1]));
      }
      qb[nb][gr][0][0] = pack_half2(x[0], x[4]);
      qb[nb][gr][0][1] = pack_half2(x[1] * 0.0625f, x[5] * 0.0625f);
      qb[nb][gr][1][0] = pack_half2(x[2], x[6]);
      qb[nb][gr][1][1] = pack_half2(x[3] * 0.0625f, x[7] * 0.0625f);
      sums[gr] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    }
    float mine[2] = {0.0f, 0.0f};
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      sums[gr] += __shfl_xor_sync(0xffffffffu, sums[gr], 1);
      sums[gr] += __shfl_xor_sync(0xffffffffu, sums[gr], 2);
      // over 32, so that 32 values of the fp16 range stay inside it
      if (gr >> 1 == t) mine[gr & 1] = sums[gr] * 0.03125f;
    }
    const float hi0 = __half2float(__float2half_rn(mine[0])), hi1 = __half2float(__float2half_rn(mine[1]));
    qs[nb][0] = pack_half2(hi0, hi1);
    qs[nb][1] = pack_half2(mine[0] - hi0, mine[1] - hi1);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = nb * 8 + 2 * t + c;
      // rows past the last take its keys, so that their arithmetic stays finite
      const int i = tok0 + token_of(r < n_rows ? r : n_rows - 1);
      lim[nb][c] = a.p.causal ? seq_len - q_len + i : seq_len - 1;
      lo[nb][c] = a.p.window > 0 ? max(0, lim[nb][c] - a.p.window + 1) : 0;
      min_lim = min(min_lim, lim[nb][c]);
      max_lo = max(max_lo, lo[nb][c]);
    }
  }
  if (__any_sync(0xffffffffu, bad_q) && warp == 0 && lane == 0 && sigma == 0)
    flag_status(a.status, PA_DEV_BAD_Q);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, o));
    max_lo = max(max_lo, __shfl_xor_sync(0xffffffffu, max_lo, o));
  }

  float m_used[NB][2], l[NB][2];  // rows 2t, 2t + 1 (log2 units; l: this lane's share)
  float o[NB][G][2][4], oz[NB][4];
  const float c1 = by.codes, c2 = by.zeros;
  float m_safe[NB][2];  // m_used, 0 before the first key
  const int key_r0 = perm16(g), key_r1 = perm16(g + 8);
  // (m_used: the maximum less the lift, which p, l and o are taken against)
  float lift = kLift;
again:
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m_safe[nb][c] = 0.0f;
      m_used[nb][c] = -INFINITY;
      l[nb][c] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      oz[nb][e] = 0.0f;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) o[nb][gr][0][e] = o[nb][gr][1][e] = 0.0f;
    }
  }
  bool started = false;

  for (int i = 0; i < n_mine; i += KB) {
    cp_async_wait<C::kStages - 2 * KB>();
    __syncwarp();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) issue(i + kb + C::kStages - KB);  // where the last blocks stood
    uint32_t st[KB];
    int key0[KB];
    bool dead[KB];  // no block, or no such page: its keys are left out
    bool edge = false;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const int stage = (i + kb) % C::kStages;
      st[kb] = ring + stage * C::kBlock;
      key0[kb] = (seg0 + warp + (i + kb) * kWarps) * 16;
      dead[kb] = !((live >> stage) & 1u);
      edge = edge || dead[kb] || key0[kb] + 15 > min_lim || key0[kb] < max_lo;
    }
    if (KB == 1 && dead[0]) continue;

    // ---- scores
    float s[KB][NB][4];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t w0[G], w1[G];  // codes of key rows g and g + 8, one word a group
      if constexpr (D == 256) {
        const int x = g & 1;  // rows g and g + 8: the same parity
        const uint32_t r0 = st[kb] + g * C::kRow + t * 32, r1 = r0 + 8 * C::kRow;
        const uint4 a0 = lds128(r0 + x * 16), a1 = lds128(r0 + (x ^ 1) * 16);
        const uint4 b0 = lds128(r1 + x * 16), b1 = lds128(r1 + (x ^ 1) * 16);
        w0[0] = a0.x; w0[1] = a0.y; w0[2] = a0.z; w0[3] = a0.w;
        w0[4] = a1.x; w0[5] = a1.y; w0[6] = a1.z; w0[7] = a1.w;
        w1[0] = b0.x; w1[1] = b0.y; w1[2] = b0.z; w1[3] = b0.w;
        w1[4] = b1.x; w1[5] = b1.y; w1[6] = b1.z; w1[7] = b1.w;
      } else {
        lds_words(st[kb] + g * C::kRow + t * (G * 4), w0);
        lds_words(st[kb] + (g + 8) * C::kRow + t * (G * 4), w1);
      }
      uint32_t sw0[G / 2], sw1[G / 2];  // scales of the two keys, two groups a word
      lds_words(st[kb] + C::kKs + key_r0 * (G * 2), sw0);
      lds_words(st[kb] + C::kKs + key_r1 * (G * 2), sw1);
      const bool has = 2 * t < G;
      const uint32_t zk = st[kb] + C::kKs + 16 * G * 2 + (has ? 4 * t : 0);
      uint32_t z0 = lds32(zk + key_r0 * (G * 2)), z1 = lds32(zk + key_r1 * (G * 2));
      if (!has) z0 = z1 = 0u;
      float acc[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nb][e] = 0.0f;
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const uint32_t lo4 = 0x000f000fu, hi4 = 0x00f000f0u;
        const uint32_t u0 = w0[gr] >> 8, u1 = w1[gr] >> 8;
        const float s0 = gr & 1 ? half_hi(sw0[gr >> 1]) : half_lo(sw0[gr >> 1]);
        const float s1 = gr & 1 ? half_hi(sw1[gr >> 1]) : half_lo(sw1[gr >> 1]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float part[4];
          mma_first(part, w0[gr] & lo4, w1[gr] & lo4, w0[gr] & hi4, w1[gr] & hi4, qb[nb][gr][0][0],
                    qb[nb][gr][0][1]);
          mma_f16_16816(part, u0 & lo4, u1 & lo4, u0 & hi4, u1 & hi4, qb[nb][gr][1][0],
                        qb[nb][gr][1][1]);
          acc[nb][0] = fmaf(s0, part[0], acc[nb][0]);
          acc[nb][1] = fmaf(s0, part[1], acc[nb][1]);
          acc[nb][2] = fmaf(s1, part[2], acc[nb][2]);
          acc[nb][3] = fmaf(s1, part[3], acc[nb][3]);
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float zp[4];
        mma_first(zp, z0, z1, z0, z1, qs[nb][0], qs[nb][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)  // scores less m_safe, log2 units
          s[kb][nb][e] = fmaf(acc[nb][e], c1, fmaf(zp[e], c2, -m_safe[nb][e & 1]));
      }
    }
    if (edge) {
      // keys that a row does not see (and stale ones: whatever stands there)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0[kb] + (e < 2 ? key_r0 : key_r1);
            if (dead[kb] || key > lim[nb][e & 1] || key < lo[nb][e & 1]) s[kb][nb][e] = -INFINITY;
          }
      // keys that no row sees may hold anything: zeros for their values' scales and zeros
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int key = key0[kb] + (lane & 15);
        if (dead[kb] || key >= range.end || key < range.begin) {
#pragma unroll
          for (int k = 0; k < 16 * G * 2 / 32; ++k)
            sts16(st[kb] + C::kVs + (2 * k + (lane >> 4)) * 32 + (lane & 15) * 2, 0);
        }
      }
      __syncwarp();
    }

    // ---- softmax against m_used, which moves only when a score passes it by kMargin
    float top = s[0][0][0];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; e += 2) top = fmax3(top, s[kb][nb][e], s[kb][nb][e + 1]);
    // (before a row's first key any score moves it: it stands at -inf)
    if (__any_sync(0xffffffffu, top > (started ? kMargin + lift : -INFINITY))) {
      bool all = true;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(s[0][nb][c], s[0][nb][2 + c]);
#pragma unroll
          for (int kb = 1; kb < KB; ++kb) mx = fmax3(mx, s[kb][nb][c], s[kb][nb][2 + c]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float mn = fmaxf(m_used[nb][c], mx + m_safe[nb][c] - lift);
          if (mn > -INFINITY) {
            const float d = m_safe[nb][c] - mn, f = fast_exp2(m_used[nb][c] - mn);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
              s[kb][nb][c] += d;
              s[kb][nb][2 + c] += d;
            }
            m_used[nb][c] = m_safe[nb][c] = mn;
            l[nb][c] *= f;
            oz[nb][c] *= f;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              o[nb][gr][0][c] *= f;
              o[nb][gr][0][2 + c] *= f;
              o[nb][gr][1][c] *= f;
              o[nb][gr][1][2 + c] *= f;
            }
          } else {
            all = false;
          }
        }
      started = __all_sync(0xffffffffu, all);  // every row of the warp has a maximum
    }

    // ---- output: keys 4t .. 4t + 3 of each block
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t pb[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = fast_exp2(s[kb][nb][e]);
        l[nb][0] += p[0] + p[2];
        l[nb][1] += p[1] + p[3];
        pb[nb][0] = movmatrix_trans(pack_half2(p[0], p[1]));
        pb[nb][1] = movmatrix_trans(pack_half2(p[2], p[3]));
      }
      {
        uint2 z = lds64(st[kb] + C::kVs + (G + (g < G ? g : 0)) * 32 + t * 8);
        if (g >= G) z = make_uint2(0u, 0u);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          mma_f16_16816(oz[nb], z.x, 0u, z.y, 0u, pb[nb][0], pb[nb][1]);
      }
      constexpr int W = G / 2;  // words of a lane's codes of one key: 16 bits a group
      uint32_t vw[4][W];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = D == 256 ? 2 * t : D == 128 ? (t >> 1) * 2 : 0;
        const int byte = g * (G * 2);
        lds_words(st[kb] + C::kV + (k * 4 + t) * C::kRow + (((byte >> 4) ^ x) << 4) + (byte & 15), vw[k]);
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const uint2 sc = lds64(st[kb] + C::kVs + gr * 32 + t * 8);
        const uint32_t sel = gr & 1 ? 0x7632u : 0x5410u;
        const uint32_t x01 = __byte_perm(vw[0][gr >> 1], vw[1][gr >> 1], sel);
        const uint32_t x23 = __byte_perm(vw[2][gr >> 1], vw[3][gr >> 1], sel);
        const uint32_t lo4 = 0x000f000fu, hi4 = 0x00f000f0u;
        const uint32_t y01 = x01 >> 8, y23 = x23 >> 8;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t p0 = hmul2_u32(pb[nb][0], sc.x), p1 = hmul2_u32(pb[nb][1], sc.y);
          mma_f16_16816(o[nb][gr][0], x01 & lo4, y01 & lo4, x23 & lo4, y23 & lo4, p0, p1);
          mma_f16_16816(o[nb][gr][1], x01 & hi4, y01 & hi4, x23 & hi4, y23 & hi4, p0, p1);
        }
      }
    }
  }
  cp_async_wait<0>();
  if (lift > -kMargin) {
    float nan = 0.0f;  // NaN where a sum is infinite, or NaN
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int gr = 0; gr < G; ++gr)
#pragma unroll
        for (int e = 0; e < 4; ++e) nan = fmaf(o[nb][gr][0][e], 0.0f, fmaf(o[nb][gr][1][e], 0.0f, nan));
    if (__any_sync(0xffffffffu, nan != nan)) {
      lift = lift > 0.0f ? 0.0f : -kMargin;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < C::kStages - KB; ++i) issue(i);
      goto again;
    }
  }

  // ---- O^T of this warp as numbers: channels 32 gr + 4 g + i of rows 2t, 2t + 1
  // (nibble i: o[gr][i & 1][(i & 2) + row]), the zeros' part from the lane of its group
  float out[NB][2][G][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float z = __shfl_sync(0xffffffffu, oz[nb][c], gr * 4 + t);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          out[nb][c][gr][i] = fmaf(o[nb][gr][i & 1][(i & 2) + c], i & 1 ? 0x1p20f : 0x1p24f, z);
      }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], off);

  // ---- the four warps' sums joined by warp 0 (the rings are no longer read)
  constexpr int kFields = NB * (4 + 8 * G);
  float *area = reinterpret_cast<float *>(smem_raw);
  __syncthreads();
  if (warp > 0) {
    float *dst = area + (warp - 1) * kFields * 32 + lane;
    int f = 0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        dst[32 * f++] = m_used[nb][c];
        dst[32 * f++] = l[nb][c];
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[32 * f++] = out[nb][c][gr][i];
      }
  }
  __syncthreads();
  if (warp > 0) {
    if (threadIdx.x == 32 && a.p.max_query_len > 1) flag_bad_sequences(a, item, h, sigma);
    return;
  }
#pragma unroll 1
  for (int k = 0; k < kWarps - 1; ++k) {
    const float *src = area + k * kFields * 32 + lane;
    int f = 0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float mo = src[32 * f++];
        const float mn = fmaxf(m_used[nb][c], mo);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        const float wa = fast_exp2(m_used[nb][c] - mu), wb = fast_exp2(mo - mu);
        m_used[nb][c] = mn;
        l[nb][c] = l[nb][c] * wa + src[32 * f++] * wb;
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
          for (int i = 0; i < 4; ++i) out[nb][c][gr][i] = out[nb][c][gr][i] * wa + src[32 * f++] * wb;
      }
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = nb * 8 + 2 * t + c;
      if (row >= n_rows) continue;
      const int tr = token_of(row);
      const int head = h * a.qpk + row - tr * a.qpk;
      const int64_t at = static_cast<int64_t>(q0 + tok0 + tr) * a.p.hq + head;
      float m = m_used[nb][c], sum = l[nb][c];
      if (a.num_splits > 1) {
        const int64_t prow = at * a.num_splits + sigma;
        if (g == 0) a.part_ml[prow] = make_float2(m, sum);
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
          *reinterpret_cast<float4 *>(a.part_acc + prow * D + gr * 32 + g * 4) =
              make_float4(out[nb][c][gr][0], out[nb][c][gr][1], out[nb][c][gr][2], out[nb][c][gr][3]);
        continue;
      }
      float w = 1.0f;
      if (a.p.sinks) {
        const float sk = a.p.sinks[head] * kLog2e;
        const float mn = fmaxf(m, sk);
        if (mn > -INFINITY) {
          w = fast_exp2(m - mn);
          sum = sum * w + fast_exp2(sk - mn);
          m = mn;
        }
      }
      const float inv = sum == 0.0f ? 0.0f : w / sum;  // a row that sees no key: 0 (a NaN stays one)
      uint16_t *dst = a.p.out + at * D + g * 4;
#pragma unroll
      for (int gr = 0; gr < G; ++gr)
        *reinterpret_cast<uint2 *>(dst + gr * 32) =
            make_uint2(pack_bf162(out[nb][c][gr][0] * inv, out[nb][c][gr][1] * inv),
                       pack_bf162(out[nb][c][gr][2] * inv, out[nb][c][gr][3] * inv));
      if (g == 0 && a.p.lse) a.p.lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
}

// Joins the triples of a row (token, q head), one warp a row.
template <int D>
__global__ void __launch_bounds__(128) q4_join_kernel(const __grid_constant__ Q4Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (at >= static_cast<int64_t>(a.p.num_tokens) * a.p.hq) return wait_for_predecessor();
  // The row's sequence and its segments, while the kernel before still runs: what this
  // reads was there before that kernel let this one start.
  const int tok = static_cast<int>(at / a.p.hq);
  const int head = static_cast<int>(at % a.p.hq);
  const int seq = find_seq(a.p.cu, a.p.num_seqs, 1, tok, lane);
  const int q0 = a.p.cu[seq], q_len = a.p.cu[seq + 1] - q0, seq_len = a.p.seq_lens[seq];
  const bool owned = tok >= q0 && tok - q0 < q_len && valid_sequence(a, q0, q_len, seq_len);
  const int tok0 = owned ? (tok - q0) / a.block_tokens * a.block_tokens : 0;
  const int n = owned ? segments(a, key_range(a, seq_len, q_len, tok0).blocks) : 0;
  const float sink = a.p.sinks ? a.p.sinks[head] * kLog2e : -INFINITY;
  const int64_t prow = at * a.num_splits;
  wait_for_predecessor();
  if (owned)
    join_row<D>(a.part_acc + prow * D, a.part_ml + prow, n, sink, a.p.out + at * D,
                a.p.lse ? a.p.lse + at : nullptr, lane);
}

template <int D, int BS, int NB>
cudaError_t launch_rows(const Q4Args &a, cudaStream_t stream) {
  using C = Q4Cfg<D>;
  constexpr int kRing = kWarps * C::kStages * C::kBlock;
  constexpr int kMerge = (kWarps - 1) * 32 * NB * (4 + 8 * C::G) * 4;
  constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    return cudaFuncSetAttribute(attn_q4_kernel<D, BS, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.num_items), static_cast<unsigned>(a.p.hk),
                  static_cast<unsigned>(a.num_splits));
  return launch_kernel(attn_q4_kernel<D, BS, NB>, grid, kWarps * 32, kSmem, stream, a);
}

template <int D>
cudaError_t launch_join(const Q4Args &a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.p.num_tokens) * a.p.hq;
  return launch_kernel(q4_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, stream, a);
}

template <int D>
cudaError_t launch_d(const Q4Args &a, cudaStream_t stream) {
  const bool wide = a.block_tokens * a.qpk > 8;
  const bool big = a.p.bs == 32;
  cudaError_t e = wide ? (big ? launch_rows<D, 32, 2>(a, stream) : launch_rows<D, 16, 2>(a, stream))
                       : (big ? launch_rows<D, 32, 1>(a, stream) : launch_rows<D, 16, 1>(a, stream));
  return e != cudaSuccess || a.num_splits == 1 ? e : launch_join<D>(a, stream);
}

}  // namespace

namespace {
// Long queries go to the tcgen05 kernel (attn_q4_tc.cu), which turns a key's codes into
// operands once per 64 rows: from more than 64 rows a sequence and kv head on it is ahead at D 128
// (16 sequences x 4096 keys: 32 rows 44 us here, 55 there, 64 rows 61 and 54, 128 rows 97 and 77, 1200
// rows 695 and 509; 4 x 8192: 56 rows 36 and 42, 112 rows 45 and 40, 2100 rows 470 and 258).
bool on_tc(int32_t qpk, int32_t max_query_len, int32_t d) {
  return d == 128 && max_query_len > 1 && int64_t{max_query_len} * qpk > 64;
}
}  // namespace

// Rows a block.  16 rows read each key once for twice the rows, 8 leave more blocks an SM: at D
// 64 and 256 a sequence of few rows is faster in eights (16 sequences x 4096 keys, D 256, 3
// tokens x 4 heads: 50 us, 58 in sixteens; 8 x 4096, D 64, 8 x 4: 21 and 27), one of many in
// sixteens (D 256, 40 tokens x 7 heads: 146 and 166).  At D 128 sixteens hold two blocks of keys
// in work as eights do, and neither wins by more than a tenth.
int32_t q4_block_tokens(int32_t qpk, int32_t max_query_len, int32_t d) {
  if (max_query_len <= 1) return 1;
  if (on_tc(qpk, max_query_len, d)) return kTcRows / qpk;
  const bool eights = d != 128 && int64_t{max_query_len} * qpk <= 64;
  return std::max(1, (eights ? 8 : 16) / qpk);
}

namespace {
// Blocks of rows of a call (at most, by the hint of its longest query), and how many stand on
// the GPU at once.
std::pair<int64_t, int64_t> blocks_and_places(int32_t num_seqs, int32_t num_tokens, int32_t hq, int32_t hk,
                                              int32_t d, int32_t max_query_len) {
  const int32_t tokens = q4_block_tokens(hq / hk, max_query_len, d);
  const int64_t items = std::min<int64_t>({num_tokens, num_tokens / tokens + num_seqs,
                                           (int64_t{max_query_len} + tokens - 1) / tokens * num_seqs});
  const int resident = on_tc(hq / hk, max_query_len, d) ? 1 : resident_blocks(d, tokens * (hq / hk) > 8);
  return {std::max<int64_t>(1, items * hk), int64_t{152} * resident};
}
}  // namespace

// Key segments.  Blocks that do not fill the GPU's places (three quarters of what is
// resident) are split until about three times as many stand in line, in segments of at least
// 512 keys (256 where very few stand); where that limit leaves fewer than 2.5 rounds, one
// full round: 1 x 131072 keys (8 kv heads, D 128, caches cold) takes 379 us in 2 segments, 60 in
// 16, 54 in 57 (456 blocks on 456 places), 65 in 64.  Eights at D 256 stand two an SM: 4.5 times the
// places in line, 512 keys at least (1 x 131072 keys 84 us in 38 segments, 304 blocks on 304 places,
// and 103 in 57; 24 x up to 32768 keys 210 us in 8 segments, 231 in 5; 1 x 8192 keys 18 us in 16
// segments, 22 in 32; 8 x 8192 would be 36 us in 7, 41 as it is).  Blocks that fill it are split at 2048 keys,
// so that the last of long sequences do not run alone: 64 x up to 8192 keys 87 us in 4 segments,
// 105 in one; 128 x up to 2048 keys 56 us in one, 62 in 4 (the join is another launch and trip
// to memory).
// Where segments stand in line, those that start first are the longest (n - i parts of n (n + 1) /
// 2 each), so that the last ones to run are short: 64 x up to 8192 keys 93 us in equal
// segments, 87 so; 48 x 5 tokens x 8 heads on up to 6001 keys 127 and 117; 16 x up to 32768 keys 105
// and 97; 6 x up to 131072 keys at D 256, five drawings of lengths, 1268 and 1133 together.
int32_t q4_auto_splits(int32_t num_seqs, int32_t num_tokens, int32_t hq, int32_t hk, int32_t d,
                       int32_t max_query_len, int32_t max_seq_len) {
  const auto [blocks, places] = blocks_and_places(num_seqs, num_tokens, hq, hk, d, max_query_len);
  const int64_t keys = std::max<int64_t>(1, max_seq_len);
  int64_t ns = (keys + 2047) / 2048;
  if (4 * blocks < 3 * places) {
    const bool eights = d == 256 && q4_block_tokens(hq / hk, max_query_len, d) * (hq / hk) <= 8;
    const int64_t line = eights ? 9 * places / 2 : 3 * places;
    const int64_t least = 8 * blocks < places && !eights ? 256 : 512;
    ns = std::min<int64_t>({(line + blocks - 1) / blocks, keys / least, kMaxSegments});
    if (ns * blocks > places && 2 * ns * blocks < 5 * places) ns = places / blocks;
  } else {
    ns = std::min(ns, (16 * places + blocks - 1) / blocks);
  }
  return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(ns, kMaxSegments)));
}

cudaError_t launch_attention_q4(const AttnQ4 &p, cudaStream_t stream) {
  Q4Args a;
  a.p = p;
  a.status = reinterpret_cast<uint32_t *>(p.workspace);
  a.num_splits = p.num_splits;
  a.part_acc = reinterpret_cast<float *>(p.workspace + 256);
  a.part_ml = reinterpret_cast<float2 *>(a.part_acc + static_cast<int64_t>(p.num_tokens) * p.hq *
                                                          p.num_splits * p.d);
  a.qpk = p.hq / p.hk;
  a.qpk_inverse = 65536 / a.qpk + 1;
  a.block_tokens = q4_block_tokens(a.qpk, p.max_query_len, p.d);
  a.num_items = p.max_query_len <= 1 ? p.num_seqs
                : a.block_tokens == 1 ? p.num_tokens
                                      : p.num_tokens / a.block_tokens + p.num_seqs;
  a.scale_log2 = p.softmax_scale * kLog2e;
  int blocks = (p.max_seq_len + 15) / 16;
  if (p.window > 0 && p.window < p.max_seq_len) blocks = std::min(blocks, (p.window + a.block_tokens + 15) / 16 + 1);
  const auto [row_blocks, places] = blocks_and_places(p.num_seqs, p.num_tokens, p.hq, p.hk, p.d, p.max_query_len);
  const bool falling = p.num_splits * row_blocks > places;
  const int64_t n = p.num_splits;
  for (int64_t i = 0; i < n; ++i)
    a.seg_start[i] = static_cast<int32_t>(
        falling ? blocks * i * (2 * n + 1 - i) / (n * (n + 1)) : i * std::max<int64_t>(1, (blocks + n - 1) / n));
  if (on_tc(a.qpk, p.max_query_len, p.d)) {
    for (int64_t i = 0; i < n; ++i) a.seg_start[i] = (a.seg_start[i] + 7) / 8 * 8;  // whole tiles of 128 keys
    const cudaError_t e = launch_attention_tc(a, stream);
    return e != cudaSuccess || a.num_splits == 1 ? e : launch_join<128>(a, stream);
  }
  switch (p.d) {
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    case 256: return launch_d<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paq8
