// Attention over the 4-bit cache for blocks of many query rows (D 128): up to 64 rows (tokens x
// the q heads of a kv head) against 128-key tiles on tcgen05, keys in the M dimension.
//
//   S_g^T[128 keys x 64 rows] = C_g[128 x 32 ch] Q_g^T      codes of group g, as fp16
//   S^T = sum_g s_g S_g^T + Z[128 x 16] (sums of q)^T       each key's scales in its own thread
//   O^T[128 ch x 64 rows] += V'^T[128 ch x 128 keys] P^T    V' = fp16(code * scale + zero)
//
// A key's row of S belongs to one thread (a TMEM lane), so its group scales are scalars of that
// thread and the codes enter the product exactly: masked out of their words they are the
// fp16 subnormals code * 2^-24.  The zeros' part is one MMA more over the groups, q's sums in two
// fp16 parts.  P^T (64 rows a key: 128 bytes) and the rows of V' (channels contiguous) are
// written to shared memory as they are formed: both are operands whose M or N dimension is the
// contiguous one.
// The mma.sync kernel turns every key's codes into operands once per 16 rows; this one once
// per 64, and leaves the products to the tensor core.  Measured: 1 sequence x 32768 keys, 8 kv
// heads, one segment, 1.65 us a 128-key tile (3100 cycles) on each of 8 SMs: the softmax warps' chain
// (the five accumulators 700 cycles, the maximum 190, the vote 400, P 540, waits 700), then the
// 17 MMAs (60 cycles each at N = 64).  With four softmax warps and the codes in shared memory 1.85.
// 16 sequences x 4096 keys x 300 tokens x 4 heads: 509 us (mma.sync 695).
//
// V' is rounded to fp16 (2^-11 of a value; past 65504 infinite); P to fp16.
//
// Softmax: sums along a row run over threads.  Every row's maximum (less the lift of 2^10, which
// keeps small p out of fp16's subnormals) stands in shared memory; a vote of the four warps
// decides whether one moves, by 2^4 at least, and only then are column maxima formed
// (exchanges that halve the columns) and O^T in TMEM rescaled.
//
// Warps: 0 - 7 softmax (a TMEM quarter and half the rows each), 8 - 11 codes of keys to operands
// (in TMEM: a key is a lane), 12 - 15 those of values (a key a thread, two tiles' codes on
// their way in registers), 16 issues the MMAs.
#include "attn_common.cuh"
#include "attn_q4.cuh"
#include "launch.h"
#include "programmatic.cuh"
#include "q4.cuh"
#include "tcgen05.cuh"

namespace paq8 {
namespace q4 {

namespace {

constexpr int kD = 128;
constexpr int kG = 4;
constexpr int kN = kTcRows;
constexpr int kKeys = 128;
constexpr int kHalf = kN / 2;  // rows of a softmax thread
constexpr int kSoftmaxWarps = 8, kThreads = (kSoftmaxWarps + 8 + 4) * 32;
constexpr float kLift = 10.0f;   // log2 of p at the maximum
constexpr float kMargin = 4.0f;  // log2 of the largest p over that

// shared memory
constexpr int kZBytes = kKeys * 128;     // zeros: 32 bytes of each 128-byte row
constexpr int kVBytes = kKeys * kD * 2;  // two chunks of 64 channels
constexpr int kPBytes = kKeys * 128;
constexpr int kZOff = 0;                        // [2]
constexpr int kVOff = kZOff + 2 * kZBytes;      // [2]
constexpr int kPOff = kVOff + 2 * kVBytes;      // [2]
constexpr int kQOff = kPOff + 2 * kPBytes;      // two chunks of 64 rows
constexpr int kQsOff = kQOff + kN * kD * 2;     // sums of q
constexpr int kScOff = kQsOff + kN * 128;       // [4][128] scales of a key's groups, fp16
constexpr int kDeadOff = kScOff + 4 * kKeys * 8;  // [4][4] keys without a page, a bit each
constexpr int kRowOff = kDeadOff + 64;          // m, shift, factor: fp32 [3][64]
constexpr int kPartOff = kRowOff + 3 * kN * 4;  // column maxima and sums of the four warps
constexpr int kBarOff = kPartOff + 4 * kN * 4;
constexpr int kSmem = kBarOff + 256 + 1024;
static_assert(kSmem <= 232448, "shared memory");

// barriers
constexpr int kBarK = 0;       // [2] codes and zeros of a tile -> MMA
constexpr int kBarKFree = 2;   // [2] commit of QK -> codes
constexpr int kBarV = 4;       // [2] values of a tile -> MMA
constexpr int kBarPv = 6;      // [2] commit of PV -> values, P, rescale, epilogue
constexpr int kBarS = 8;       // commit of QK -> softmax
constexpr int kBarSFree = 9;   // S was read -> MMA
constexpr int kBarP = 10;      // [2] P of a tile -> MMA
constexpr int kBarSc = 12;     // [4] scales of a tile -> softmax
constexpr int kBarQ = 16;      // q -> MMA
constexpr int kBarDrain = 17;
constexpr int kNumBars = 18;

// TMEM columns
constexpr uint32_t kSCol = 0;               // S_g at 64 g, the zeros' part at 256
constexpr uint32_t kOCol = (kG + 1) * kN;
constexpr uint32_t kKCol = kOCol + kN;      // [2] codes of a tile, two channels a column
static_assert(kKCol + 2 * (kD / 2) <= 512, "TMEM");

// A and B fp16; a_m, b_n: the operand's M (N) dimension is the contiguous one.
__host__ __device__ constexpr uint32_t idesc(int n, bool a_m, bool b_n) {
  return tc::idesc_f16(128, n) | (a_m ? 1u << 15 : 0u) | (b_n ? 1u << 16 : 0u);
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The softmax warps' own barrier, and their vote.
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void sts_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ void sts_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_u64(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// Combines 32 columns over the 32 lanes of a warp (max or sum): lane l ends with column l in
// x[0].  Each exchange halves the columns that a lane still holds.
template <bool SUM>
__device__ __forceinline__ void reduce_columns(float (&x)[kHalf], int lane) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < off; ++i) {
      const float send = upper ? x[i] : x[i + off];
      const float keep = upper ? x[i + off] : x[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, off);
      x[i] = SUM ? keep + got : fmaxf(keep, got);
    }
  }
}

// 16 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <int BS>
__global__ void __launch_bounds__(kThreads, 1) attn_q4_tc_kernel(const __grid_constant__ Q4Args a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem + kBarOff;
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  const uint32_t tmem_slot = bars + 8 * kNumBars;

  wait_for_predecessor();
  launch_dependents();  // the join waits for all of this grid
  // ---- which rows, which keys (all warps alike)
  const int item = blockIdx.x, h = blockIdx.y, sigma = blockIdx.z;
  const int seq = find_seq(a.p.cu, a.p.num_seqs, a.block_tokens, item, lane);
  const int q0 = a.p.cu[seq];
  const int q_len = a.p.cu[seq + 1] - q0;
  const int seq_len = a.p.seq_lens[seq];
  const int tok0 = (item - ((a.block_tokens == 1 ? q0 : q0 / a.block_tokens + seq))) * a.block_tokens;
  if (tok0 < 0 || tok0 >= q_len || !valid_sequence(a, q0, q_len, seq_len)) {
    if (threadIdx.x == 0) flag_bad_sequences(a, item, h, sigma);
    return;
  }
  const KeyRange range = key_range(a, seq_len, q_len, tok0);
  if (seq_len > int64_t{a.p.table_columns} * BS && sigma == 0 && threadIdx.x == 0)
    flag_status(a.status, PA_DEV_BAD_BLOCK);
  if (sigma > 0 && a.seg_start[sigma] >= range.blocks) return;  // (as segments() counts)
  const int n_tok = min(a.block_tokens, q_len - tok0);
  const int n_rows = n_tok * a.qpk;
  const int seg0 = range.first + a.seg_start[sigma];
  const int seg1 = sigma == a.num_splits - 1 ? range.first + range.blocks
                                             : min(range.first + range.blocks, range.first + a.seg_start[sigma + 1]);
  // keys of this segment; a key past them is left out as one without a page
  const int begin = max(range.begin, seg0 * 16), end = min(range.end, seg1 * 16);
  const int nt = end > begin ? (end - seg0 * 16 + kKeys - 1) / kKeys : 0;
  const int first_lim = a.p.causal ? seq_len - q_len + tok0 : seq_len - 1;  // last key of token 0

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBarK + s), 4);
      mbar_init(bar(kBarKFree + s), 1);
      mbar_init(bar(kBarV + s), 4);
      mbar_init(bar(kBarPv + s), 1);
      mbar_init(bar(kBarP + s), kSoftmaxWarps);
    }
    for (int s = 0; s < 4; ++s) mbar_init(bar(kBarSc + s), 4);
    mbar_init(bar(kBarS), 1);
    mbar_init(bar(kBarSFree), kSoftmaxWarps);
    mbar_init(bar(kBarQ), kSoftmaxWarps);
    mbar_init(bar(kBarDrain), 1);
    fence_barrier_init();
  }
  constexpr int kMmaWarp = kSoftmaxWarps + 8;
  if (warp == kMmaWarp) tc::alloc(tmem_slot, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot) : "memory");
  bool ok = true;

  if (warp < kSoftmaxWarps) {
    // ============================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int tid = threadIdx.x;
    const int quarter = warp & 3, r_first = (warp >> 2) * kHalf;  // TMEM lanes (keys), first row
    const int t = quarter * 32 + lane;                            // key of the tile
    auto wait = [&](int b, uint32_t parity) {  // (the warps stay together: no barrier is left out)
      if (ok && !__all_sync(0xffffffffu, mbar_test(bar(b), parity)))
        ok = __all_sync(0xffffffffu, mbar_wait(bar(b), parity));
    };
    QueryScale by;
    // ---- q: a row's group a thread, octets as the codes' words have them: 0, 4, 1, 5, 2, 6, 3, 7
    {
      const int row = tid & 63, g = tid >> 6;
      const bool real = row < n_rows;
      const int tr = real ? (row * a.qpk_inverse) >> 16 : 0;
      const uint16_t *src = a.p.q + (static_cast<int64_t>(q0 + tok0 + tr) * a.p.hq + h * a.qpk +
                                     (real ? row - tr * a.qpk : 0)) * kD + g * 32;
      uint4 v[4];
      float largest = 0.0f;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        v[o] = make_uint4(0u, 0u, 0u, 0u);
        if (real) v[o] = *reinterpret_cast<const uint4 *>(src + o * 8);
      }
#pragma unroll
      for (int o = 0; o < 4; ++o) largest = fmaxf(largest, largest_of(v[o]));
      largest = warp_largest(largest);
      if (lane == 0) sts_f32(smem + kPartOff + warp * 4, largest);
      softmax_sync();
      largest = warp_largest(lds_f32(smem + kPartOff + (lane % kSoftmaxWarps) * 4));
      by = query_scale(largest, a.scale_log2);
      bool bad_q = false;
      float sum = 0.0f;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const uint32_t w[4] = {v[o].x, v[o].y, v[o].z, v[o].w};
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = bf16_lo(w[i]) * by.up;
          x[2 * i + 1] = bf16_hi(w[i]) * by.up;
          bad_q |= half2_nonfinite(pack_half2(x[2 * i], x[2 * i + 1]));
        }
        sts128(smem + kQOff + tc::sw128_chunk(row, g * 4 + o, kN),
               make_uint4(pack_half2(x[0], x[4]), pack_half2(x[1], x[5]), pack_half2(x[2], x[6]),
                          pack_half2(x[3], x[7])));
        sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
      }
      // over 32, so that 32 values of the fp16 range stay inside it
      sum *= 0.03125f;
      const float hi = __half2float(__float2half_rn(sum));
      const uint32_t at = smem + kQsOff + tc::sw128_chunk(row, 0, kN) + g * 2;
      sts_u16(at, static_cast<uint16_t>(pack_half2(hi, 0.0f)));
      sts_u16(at + 8, static_cast<uint16_t>(pack_half2(sum - hi, 0.0f)));
      if (g == 0) sts128(smem + kQsOff + tc::sw128_chunk(row, 1, kN), make_uint4(0u, 0u, 0u, 0u));
      if (__any_sync(0xffffffffu, bad_q) && lane == 0 && sigma == 0) flag_status(a.status, PA_DEV_BAD_Q);
      if (tid < kN) sts_f32(smem + kRowOff + tid * 4, 0.0f);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQ));
    }
    softmax_sync();

    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + r_first;
    const float c1 = by.codes, c2 = by.zeros;
    uint64_t l2[kHalf / 2];
#pragma unroll
    for (int i = 0; i < kHalf / 2; ++i) l2[i] = 0;
    // row tid (tid < 64): its maximum less the lift, -inf before its first key
    float m_row = -INFINITY;
    bool started = false;
    const int last_lim = a.p.causal ? first_lim + n_tok - 1 : first_lim;
    const int max_lo = a.p.window > 0 ? max(0, last_lim - a.p.window + 1) : 0;
    const uint32_t m_at = smem + kRowOff, m_mine = m_at + r_first * 4;
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      wait(kBarSc + (j & 3), (j >> 2) & 1);
      uint32_t dead_bits;
      uint2 sw;
      asm volatile("ld.shared.u32 %0, [%1];"
                   : "=r"(dead_bits)
                   : "r"(smem + kDeadOff + (j & 3) * 16 + quarter * 4)
                   : "memory");
      sw = lds64(smem + kScOff + (j & 3) * (kKeys * 8) + t * 8);
      float sc[kG];
      sc[0] = __half2float(__ushort_as_half(static_cast<uint16_t>(sw.x))) * c1;
      sc[1] = __half2float(__ushort_as_half(static_cast<uint16_t>(sw.x >> 16))) * c1;
      sc[2] = __half2float(__ushort_as_half(static_cast<uint16_t>(sw.y))) * c1;
      sc[3] = __half2float(__ushort_as_half(static_cast<uint16_t>(sw.y >> 16))) * c1;
      uint64_t sc2[kG];
#pragma unroll
      for (int g = 0; g < kG; ++g) sc2[g] = f32x2_pack(sc[g], sc[g]);
      const uint64_t z2 = f32x2_pack(c2, c2), minus1 = f32x2_pack(-1.0f, -1.0f);
      wait(kBarS, j & 1);
      tc::fence_after();
      uint64_t x2[kHalf / 2];  // scores less m, log2 units
      {
        uint32_t r0[32], r1[32];
        tc::ld32(t_lane + kSCol + 4 * kN, r0);
        tc::ld32(t_lane + kSCol + 0 * kN, r1);
#pragma unroll
        for (int i = 0; i < kHalf / 4; ++i) {
          const uint4 m = lds128(m_mine + i * 16);
          x2[2 * i] = f32x2_mul(f32x2_pack(__uint_as_float(m.x), __uint_as_float(m.y)), minus1);
          x2[2 * i + 1] = f32x2_mul(f32x2_pack(__uint_as_float(m.z), __uint_as_float(m.w)), minus1);
        }
        auto add = [&](const uint32_t(&r)[32], uint64_t f) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x2[i] = f32x2_fma(f32x2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), f, x2[i]);
        };
        tc::wait_loaded(r0);
        tc::wait_loaded(r1);
        add(r0, z2);
        add(r1, sc2[0]);
        tc::ld32(t_lane + kSCol + 1 * kN, r0);
        tc::ld32(t_lane + kSCol + 2 * kN, r1);
        tc::wait_loaded(r0);
        tc::wait_loaded(r1);
        add(r0, sc2[1]);
        add(r1, sc2[2]);
        tc::ld32(t_lane + kSCol + 3 * kN, r0);
        tc::wait_loaded(r0);
        add(r0, sc2[3]);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarSFree));
      float x[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) f32x2_unpack(x2[i], x[2 * i], x[2 * i + 1]);
      const int key0 = seg0 * 16 + j * kKeys, key = key0 + t;
      if (dead_bits != 0u || key0 + kKeys - 1 > first_lim || key0 < max_lo) {
        const bool dead = (dead_bits >> lane) & 1u;
        const int tok_last = a.p.causal ? key - first_lim : (key <= first_lim ? 0 : 0x7fffffff);
        // visible to tokens i with lim = first_lim + i >= key and lim - window < key
        const int tok_end = a.p.window > 0 ? static_cast<int>(min(static_cast<int64_t>(key) - first_lim + a.p.window,
                                                                  int64_t{0x7fffffff}))
                                           : 0x7fffffff;
#pragma unroll
        for (int r = 0; r < kHalf; ++r) {
          const int i = (min(r_first + r, n_rows - 1) * a.qpk_inverse) >> 16;
          if (dead || i < tok_last || i >= tok_end) x[r] = -INFINITY;
        }
      }
      float top4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top4[i] = fmaxf(x[i * (kHalf / 4)], x[i * (kHalf / 4) + 1]);
#pragma unroll
        for (int r = 2; r < kHalf / 4; r += 2)
          top4[i] = fmax3(top4[i], x[i * (kHalf / 4) + r], x[i * (kHalf / 4) + r + 1]);
      }
      const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
      if (softmax_any(top > (started ? kLift + kMargin : -INFINITY))) {
        float most[kHalf];
#pragma unroll
        for (int r = 0; r < kHalf; ++r) most[r] = x[r];
        reduce_columns<false>(most, lane);
        sts_f32(smem + kPartOff + (quarter * kN + r_first + lane) * 4, most[0]);
        softmax_sync();
        bool has = true;
        if (tid < kN) {
          float mx = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) mx = fmaxf(mx, lds_f32(smem + kPartOff + (w * kN + tid) * 4));
          const float safe = m_row == -INFINITY ? 0.0f : m_row;
          const float mn = fmaxf(m_row, mx + safe - kLift);
          const float f = mn == -INFINITY ? 1.0f : fast_exp2(m_row - mn);
          const float safe_n = mn == -INFINITY ? 0.0f : mn;
          sts_f32(m_at + tid * 4, safe_n);
          sts_f32(m_at + (kN + tid) * 4, safe - safe_n);
          sts_f32(m_at + (2 * kN + tid) * 4, f);
          m_row = mn;
          has = mn > -INFINITY;
        }
        started = !softmax_any(!has);  // (and the rows' values stand)
#pragma unroll
        for (int r = 0; r < kHalf; r += 4) {
          const uint4 d = lds128(m_mine + (kN + r) * 4), f = lds128(m_mine + (2 * kN + r) * 4);
          x[r] += __uint_as_float(d.x);
          x[r + 1] += __uint_as_float(d.y);
          x[r + 2] += __uint_as_float(d.z);
          x[r + 3] += __uint_as_float(d.w);
          l2[r / 2] = f32x2_mul(l2[r / 2], f32x2_pack(__uint_as_float(f.x), __uint_as_float(f.y)));
          l2[r / 2 + 1] = f32x2_mul(l2[r / 2 + 1], f32x2_pack(__uint_as_float(f.z), __uint_as_float(f.w)));
        }
        if (j > 0) {
          wait(kBarPv + ((j - 1) & 1), ((j - 1) >> 1) & 1);
          tc::fence_after();
          uint32_t o[32];
          tc::ld32(t_lane + kOCol, o);
          tc::wait_loaded(o);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            o[c] = __float_as_uint(__uint_as_float(o[c]) * lds_f32(m_mine + (2 * kN + c) * 4));
          tc::st32(t_lane + kOCol, o);
          tc::wait_st();
          tc::fence_before();
        }
      }
      // ---- P^T: this key's row, half of its 64 (PV(j - 2), the buffer's last reader, was issued
      // before QK(j), and S(j) is complete when all before it is)
      const uint32_t p_at = smem + kPOff + (j & 1) * kPBytes + t * 128;
#pragma unroll
      for (int c = 0; c < kHalf / 8; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p0 = fast_exp2(x[8 * c + 2 * i]), p1 = fast_exp2(x[8 * c + 2 * i + 1]);
          l2[4 * c + i] = f32x2_add(l2[4 * c + i], f32x2_pack(p0, p1));
          w[i] = pack_half2(p0, p1);
        }
        sts128(p_at + (((r_first / 8 + c) ^ (t & 7)) * 16), make_uint4(w[0], w[1], w[2], w[3]));
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarP + (j & 1)));
    }

    // ---- epilogue: the rows' sums, then O^T
    {
      float sums[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) f32x2_unpack(l2[i], sums[2 * i], sums[2 * i + 1]);
      reduce_columns<true>(sums, lane);
      sts_f32(smem + kPartOff + (quarter * kN + r_first + lane) * 4, sums[0]);
    }
    softmax_sync();
    if (nt > 0) wait(kBarPv + ((nt - 1) & 1), ((nt - 1) >> 1) & 1);
    tc::fence_after();
    if (tid < kN) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) sum += lds_f32(smem + kPartOff + (w * kN + tid) * 4);
      float inv = 0.0f;
      if (tid < n_rows && ok) {
        const int tr = (tid * a.qpk_inverse) >> 16;
        const int head = h * a.qpk + tid - tr * a.qpk;
        const int64_t at = static_cast<int64_t>(q0 + tok0 + tr) * a.p.hq + head;
        if (a.num_splits > 1) {
          a.part_ml[at * a.num_splits + sigma] = make_float2(m_row, sum);
        } else {
          float w = 1.0f, m = m_row;
          if (a.p.sinks) {
            const float sk = a.p.sinks[head] * kLog2e;
            const float mn = fmaxf(m, sk);
            if (mn > -INFINITY) {
              w = fast_exp2(m - mn);
              sum = sum * w + fast_exp2(sk - mn);
              m = mn;
            }
          }
          inv = sum == 0.0f ? 0.0f : w / sum;  // a row that sees no key: 0 (a NaN stays one)
          if (a.p.lse) a.p.lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
        }
      }
      sts_f32(m_at + tid * 4, inv);
    }
    softmax_sync();
    // channel of this TMEM lane
    const int ch = 64 * (quarter >> 1) + 16 * (quarter & 1) + 32 * (lane & 1) + 4 * (lane >> 3) + ((lane >> 1) & 3);
    uint32_t o[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) o[c] = 0u;
    if (nt > 0) {
      tc::ld32(t_lane + kOCol, o);
      tc::wait_loaded(o);
    }
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const int row = r_first + c;
      if (row >= n_rows || !ok) break;
      const int tr = (row * a.qpk_inverse) >> 16;
      const int64_t at = static_cast<int64_t>(q0 + tok0 + tr) * a.p.hq + h * a.qpk + row - tr * a.qpk;
      const float v = __uint_as_float(o[c]);
      if (a.num_splits > 1)
        a.part_acc[(at * a.num_splits + sigma) * kD + ch] = v;
      else
        a.p.out[at * kD + ch] = static_cast<uint16_t>(pack_bf162(v * lds_f32(m_at + row * 4), 0.0f));
    }
  } else if (warp < kMmaWarp) {
    // ============================================================ codes to operands
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const bool values = warp >= kSoftmaxWarps + 4;
    const int t = threadIdx.x & 127;  // key of the tile
    constexpr int kRow = kD / 2;
    constexpr int kPlane = BS * kG * 2;  // bytes of a page's plane of scales or zeros
    const int32_t *table = a.p.block_table + static_cast<int64_t>(seq) * a.p.table_stride;
    const int64_t code_page = static_cast<int64_t>(a.p.hk) * BS * kRow;
    const int64_t scale_page = static_cast<int64_t>(a.p.hk) * 2 * kPlane;
    const uint8_t *codes = (values ? a.p.v_cache : a.p.k_cache) + static_cast<int64_t>(h) * BS * kRow;
    const uint8_t *scales = reinterpret_cast<const uint8_t *>(values ? a.p.v_scale : a.p.k_scale) +
                            static_cast<int64_t>(h) * 2 * kPlane;
    auto wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(b), parity)) != 0; };
    const int off = (seg0 * 16 + t) % BS;  // (a tile is whole pages)
    // the table's entry for this thread's key of tile j, -1 where the key is not wanted (looked
    // at a tile later: nothing here waits for it)
    auto wanted = [&](int j) {
      const int key = seg0 * 16 + j * kKeys + t;
      return key >= begin && key < end;
    };
    auto entry = [&](int j) { return wanted(j) ? table[(seg0 * 16 + j * kKeys + t) / BS] : -1; };
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    // two tiles in registers: codes, scales and zeros (keys: two groups a word)
    uint4 c[2][4];
    uint32_t sc[2][kG], z[2][kG];
    bool live[2];
    auto load = [&](int b, int j, int entry_of) {
      live[b] = entry_of >= 0 && entry_of < a.p.num_blocks;
      if (!live[b]) {
        if (wanted(j)) flag_status(a.status, PA_DEV_BAD_BLOCK);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[b][i] = zero4;
#pragma unroll
        for (int g = 0; g < kG; ++g) sc[b][g] = z[b][g] = 0u;
        return;
      }
      const uint4 *src = reinterpret_cast<const uint4 *>(codes + entry_of * code_page + off * kRow);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[b][i] = src[i];
      const uint8_t *s = scales + entry_of * scale_page;
      if (!values) {
        const uint2 x = *reinterpret_cast<const uint2 *>(s + off * (kG * 2));
        const uint2 y = *reinterpret_cast<const uint2 *>(s + kPlane + off * (kG * 2));
        sc[b][0] = x.x;
        sc[b][1] = x.y;
        z[b][0] = y.x;
        z[b][1] = y.y;
      } else {
        const uint16_t *v = reinterpret_cast<const uint16_t *>(s) + off;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          sc[b][g] = v[g * BS];
          z[b][g] = v[(kG + g) * BS];
        }
      }
    };
    {
      const int e0 = nt > 0 ? entry(0) : -1, e1 = nt > 1 ? entry(1) : -1;
      load(0, 0, e0);
      load(1, 1, e1);
    }
    int next = nt > 2 ? entry(2) : -1;
    const uint32_t row = smem + t * 128;
    const uint32_t swz = t & 7;
#pragma unroll 1
    for (int j0 = 0; ok && j0 < nt; j0 += 2) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int j = j0 + b;
        if (j >= nt) break;
        const int after = j + 3 < nt ? entry(j + 3) : -1;
        if (j >= 2 && !wait((values ? kBarPv : kBarKFree) + b, ((j - 2) >> 1) & 1)) { ok = false; break; }
        const uint32_t *w = reinterpret_cast<const uint32_t *>(c[b]);
        if (!values) {
          // word 4 u + group: octet u of the group, this key's lane of TMEM
          tc::fence_after();
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            uint32_t k[16];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) k[4 * u + i] = (w[u * kG + g] >> (4 * i)) & 0x000f000fu;
            st16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kKCol + b * (kD / 2) + g * 16, k);
          }
          const uint32_t zr = row + kZOff + b * kZBytes;
          sts128(zr + ((0 ^ swz) * 16), make_uint4(z[b][0], z[b][1], z[b][0], z[b][1]));
          sts128(zr + ((1 ^ swz) * 16), zero4);
          const uint32_t dead = __ballot_sync(0xffffffffu, !live[b]);
          sts_u64(smem + kScOff + (j & 3) * (kKeys * 8) + t * 8, make_uint2(sc[b][0], sc[b][1]));
          if (lane == 0) sts_u32(smem + kDeadOff + (j & 3) * 16 + (warp & 3) * 4, dead);
          tc::wait_st();
          tc::fence_before();
        } else {
          // the codes of word 2 u + gp (four channels of groups 2 gp and 2 gp + 1) are the
          // 16-byte piece 8 gp + u
          const uint32_t at = row + kVOff + b * kVBytes;
          const uint32_t magic = 0x64006400u;  // 1024 in fp16, and 1024 + code below
          const uint32_t minus = 0xe400e400u;  // -1024
          const uint32_t sixteenth = 0x2c002c00u, minus64 = 0xd400d400u;
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {
            const uint32_t s2 = sc[b][2 * gp] | sc[b][2 * gp + 1] << 16, z2 = z[b][2 * gp] | z[b][2 * gp + 1] << 16;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const uint32_t x = w[u * 2 + gp], y = x >> 8;
              const uint32_t c0 = hadd2((x & 0x000f000fu) | magic, minus);
              const uint32_t c1 = hfma2((x & 0x00f000f0u) | magic, sixteenth, minus64);
              const uint32_t c2 = hadd2((y & 0x000f000fu) | magic, minus);
              const uint32_t c3 = hfma2((y & 0x00f000f0u) | magic, sixteenth, minus64);
              sts128(at + gp * (kKeys * 128) + ((u ^ swz) * 16),
                     make_uint4(hfma2(c0, s2, z2), hfma2(c1, s2, z2), hfma2(c2, s2, z2), hfma2(c3, s2, z2)));
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar((values ? kBarV : kBarK) + b));
          if (!values) mbar_arrive(bar(kBarSc + (j & 3)));
        }
        load(b, j + 2, next);
        next = after;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == kMmaWarp) {
      // ========================================================== MMA issue
      if (tc::elect_one()) {
        constexpr uint32_t id_qk = idesc(kN, false, false), id_pv = idesc(kN, true, true);
        const uint64_t q_desc = tc::desc_sw128(smem + kQOff), qs_desc = tc::desc_sw128(smem + kQsOff);
        const uint64_t z_desc = tc::desc_sw128(smem + kZOff);
        const uint64_t v_desc = tc::desc_mn_major(smem + kVOff, kKeys * 128);
        const uint64_t p_desc = tc::desc_mn_major(smem + kPOff, kPBytes);
        auto wait = [&](int i, uint32_t parity) {
          return mbar_test(bar(i), parity) || (ok = mbar_wait(bar(i), parity));
        };
        if (nt > 0) wait(kBarQ, 0);
#pragma unroll 1
        for (int j = 0; ok && j <= nt; ++j) {
          if (j < nt) {
            const int b = j & 1;
            if (!wait(kBarK + b, (j >> 1) & 1)) break;
            if (j > 0 && !wait(kBarSFree, (j - 1) & 1)) break;
            tc::fence_after();
            const uint32_t k_tmem = tmem + kKCol + b * (kD / 2);
#pragma unroll
            for (int g = 0; g < kG; ++g)
#pragma unroll
              for (int s = 0; s < 2; ++s) {  // 16 channels
                const int step = (g & 1) * 2 + s;
                tc::mma_f16_ts(tmem + kSCol + g * kN, k_tmem + (g * 2 + s) * 8,
                               q_desc + (g >> 1) * (kN * 128 >> 4) + 2 * step, id_qk, s);
              }
            tc::mma_f16(tmem + kSCol + kG * kN, z_desc + b * (kZBytes >> 4), qs_desc, id_qk, 0u);
            tc::commit(bar(kBarKFree + b));
            tc::commit(bar(kBarS));
          }
          if (j > 0) {
            const int i = j - 1, b = i & 1;
            if (!wait(kBarV + b, (i >> 1) & 1) || !wait(kBarP + b, (i >> 1) & 1)) break;
            tc::fence_after();
            const uint64_t vd = v_desc + b * (kVBytes >> 4), pd = p_desc + b * (kPBytes >> 4);
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              tc::mma_f16(tmem + kOCol, vd + s * 128, pd + s * 128, id_pv, (i > 0 || s > 0) ? 1u : 0u);
            tc::commit(bar(kBarPv + b));
          }
        }
        // no block gives up its shared memory and TMEM before its own MMAs have ended
        tc::commit(bar(kBarDrain));
        mbar_wait(bar(kBarDrain), 0);
      }
      __syncwarp();
    } else if (warp == kMmaWarp + 1 && lane == 0) {
      flag_bad_sequences(a, item, h, sigma);
    }
  }
  if (!ok) flag_status(a.status, PA_DEV_TIMEOUT);

  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

template <int BS>
cudaError_t launch(const Q4Args &a, cudaStream_t stream) {
  static DeviceOnce configured;
  const cudaError_t e = configured.get(nullptr, [](int, int *) {
    const cudaError_t r = registers_cover(reinterpret_cast<const void *>(attn_q4_tc_kernel<BS>), kThreads,
                                          256 * 144 + 256 * 80 + 128 * 32);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(attn_q4_tc_kernel<BS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.num_items), static_cast<unsigned>(a.p.hk),
                  static_cast<unsigned>(a.num_splits));
  return launch_kernel(attn_q4_tc_kernel<BS>, grid, kThreads, kSmem, stream, a);
}

}  // namespace

cudaError_t launch_attention_tc(const Q4Args &a, cudaStream_t stream) {
  return a.p.bs == 32 ? launch<32>(a, stream) : launch<16>(a, stream);
}

}  // namespace q4
}  // namespace paq8
