// kv_store in the 4-bit format (q4.cuh).  Per (token, kv head, 32 channels) of K and V:
//   lo, hi = min, max;  s = max((hi - lo) * fp32(1 / 15), 1e-8)           (fp32)
//   code = clamp(round_half_away((x - lo) / s), 0, 15)   (the IEEE fp32 quotient)
//   scale = fp16(s), zero = fp16(lo), to nearest even.
//
// Bound by HBM: 4 D bytes read and D + D / 4 written a (token, kv head); in practice by its
// latencies (55 % of the issue slots, 39 % of HBM: loads, arithmetic and small writes one
// behind another at half the warps of an SM).  Packed fp32, one reciprocal of 23 bits a half group.  A
// thread takes 16 channels (two 16-byte loads), two neighbouring lanes a group (one
// exchange for its extremes); its codes are two words of a K row or four halves of a V row.
// Several pieces a thread keep their loads in flight together.
// Measured on 17,296 tokens (8 kv heads, D 128): 23.8 us; with 8 channels a thread 29.5, with a
// whole group a thread 26 to 29; with 8 channels and the scales of 8 to 32 tokens gathered in
// shared memory and written side by side 36 to 38.
#include "launch.h"
#include "programmatic.cuh"
#include "q4.cuh"
#include "q4.h"
#include "q8_quant.cuh"

namespace paq8 {

constexpr int kStoreThreads = 256;
constexpr int kStorePieces = 2;  // 32-byte pieces a thread, of K or of V

// The codes of 8 values (pairs x) in a group with minimum lo and step s (rs = 1 / s),
// channel i at nibble i.  c = the integer next to v / s, in the low bits of one fused
// multiply-add of 1.5 * 2^23, exact unless v / s lies within 2^-15 of a tie, which
// tie_code_bits decides (rs need only be good to 2^-22: v * rs is then within 2^-18 of v /
// s); 0 <= v <= RN(hi - lo), so 0 <= v * rs < 15.0001 and no clamp is needed.  Two values an instruction (packed fp32, each rounded as by itself).
__device__ __forceinline__ uint32_t q4_codes(const uint64_t *x, float lo, float s, float rs) {
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23 = 0x4b400000
  constexpr float kFar = 0.5f - 0x1p-15f;
  const uint64_t nlo2 = f32x2_pack(-lo, -lo), rs2 = f32x2_pack(rs, rs);
  const uint64_t shift2 = f32x2_pack(kShift, kShift), minus1 = f32x2_pack(-1.0f, -1.0f);
  float v[8], t[8], d[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v2 = f32x2_add(x[i], nlo2);
    const uint64_t t2 = f32x2_fma(v2, rs2, shift2);
    const uint64_t d2 = f32x2_fma(v2, rs2, f32x2_fma(t2, minus1, shift2));  // v * rs - c
    f32x2_unpack(v2, v[2 * i], v[2 * i + 1]);
    f32x2_unpack(t2, t[2 * i], t[2 * i + 1]);
    f32x2_unpack(d2, d[2 * i], d[2 * i + 1]);
  }
  float far = fmax3(fabsf(d[0]), fabsf(d[1]), fabsf(d[2]));
  far = fmax3(far, fabsf(d[3]), fabsf(d[4]));
  far = fmax3(far, fabsf(d[5]), fmaxf(fabsf(d[6]), fabsf(d[7])));
  if (far >= kFar) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(d[i]) >= kFar) {
        const uint32_t bits =
            tie_code_bits(v[i], s, __fadd_rn(copysignf(0.5f, d[i]), __fsub_rn(t[i], kShift)));
        t[i] = __uint_as_float((bits & 0xfu) | 0x4b400000u);
      }
  }
  // sum of the words' bits << 4 i, less that of 0x4b400000 << 4 i (mod 2^32)
  uint32_t word = __float_as_uint(t[7]);
#pragma unroll
  for (int i = 6; i >= 0; --i) word = word * 16u + __float_as_uint(t[i]);
  return word - (0x4b400000u + 0xb4000000u + 0x40000000u);
}

// The least of the arguments, NaN where one of them is (fminf passes it over).
__device__ __forceinline__ float fmin_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float fmin3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int D>
__global__ void __launch_bounds__(kStoreThreads)
    kv_store_q4_kernel(const __grid_constant__ KvStoreQ4 p, const FastDiv per_token,
                       const uint32_t pieces, const int bs_log2) {
  constexpr int G = D / 32;
  constexpr int kPer = D / 16;  // pieces of a row
  wait_for_predecessor();
  const bool values = blockIdx.y != 0;
  const uint16_t *src = values ? p.value : p.key;
  const int64_t stride = values ? p.value_stride : p.key_stride;
  const int64_t num_slots = static_cast<int64_t>(p.num_blocks) << bs_log2;
  const uint32_t first = blockIdx.x * (kStoreThreads * kStorePieces) + threadIdx.x;
  uint4 raw[kStorePieces][2];
  int64_t slot[kStorePieces];
  uint32_t inner[kStorePieces];  // piece within the token
#pragma unroll
  for (int k = 0; k < kStorePieces; ++k) {
    const uint32_t i = first + k * kStoreThreads;
    slot[k] = -1;
    raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
    inner[k] = 0;
    if (i < pieces) {
      const uint32_t token = per_token.div(i);
      inner[k] = i - token * per_token.d;
      slot[k] = p.slot_mapping[token];
      const uint4 *at = reinterpret_cast<const uint4 *>(src + token * stride + inner[k] * 16);
      raw[k][0] = at[0];
      raw[k][1] = at[1];
    }
  }
#pragma unroll
  for (int k = 0; k < kStorePieces; ++k) {
    uint64_t x[8];
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w[4] = {raw[k][half].x, raw[k][half].y, raw[k][half].z, raw[k][half].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
        lo = fmin3_nan(lo, a, b);  // a NaN becomes its group's zero, and its scale
        hi = fmax3(hi, a, b);
        x[4 * half + i] = f32x2_pack(a, b);
      }
    }
    lo = fmin_nan(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
    if (slot[k] < 0) continue;  // the same for the two lanes of a group
    if (slot[k] >= num_slots) {
      if (inner[k] == 0 && !values) flag_status(p.status, PA_DEV_BAD_SLOT);
      continue;
    }
    float s = __fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f);
    s = s < 1e-8f ? 1e-8f : s;
    float rs;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
    const uint32_t word[2] = {q4_codes(x, lo, s, rs), q4_codes(x + 4, lo, s, rs)};
    const int h = static_cast<int>(inner[k] / kPer);
    const int o = static_cast<int>(inner[k] % kPer) * 2;  // the first octet; o + 1 stands beside it
    const uint32_t off = static_cast<uint32_t>(slot[k]) & (p.block_size - 1);
    // page and row numbers are below 2^31: num_blocks * num_kv_heads * D is
    const uint32_t page = static_cast<uint32_t>(slot[k] >> bs_log2) * p.hk + h;
    const uint32_t row = (page << bs_log2) + off;
    const uint16_t s16 = __half_as_ushort(__float2half_rn(s));
    const uint16_t z16 = __half_as_ushort(__float2half_rn(lo));
    const int plane = p.block_size * G;
    const bool scale = (o & 3) == 0;
    if (!values) {
      uint8_t *dst = p.k_cache + static_cast<uint64_t>(row) * (D / 2) + q4_k_word(o, G);
      *reinterpret_cast<uint32_t *>(dst) = word[0];
      *reinterpret_cast<uint32_t *>(dst + 4 * G) = word[1];
      if (scale) {
        uint16_t *sc = p.k_scale + static_cast<uint64_t>(page) * (2 * plane) + off * G + (o >> 2);
        sc[0] = s16;
        sc[plane] = z16;
      }
    } else {
      uint8_t *dst = p.v_cache + static_cast<uint64_t>(row) * (D / 2) + q4_v_half(o, 0, G);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint16_t *>(dst + i * (2 * G)) = static_cast<uint16_t>(word[i >> 1] >> (16 * (i & 1)));
      if (scale) {
        uint16_t *sc = p.v_scale + static_cast<uint64_t>(page) * (2 * plane) + (o >> 2) * p.block_size + off;
        sc[0] = s16;
        sc[plane] = z16;
      }
    }
  }
}

cudaError_t launch_kv_store_q4(const KvStoreQ4 &p, cudaStream_t stream) {
  const uint32_t per_token = static_cast<uint32_t>(p.hk) * (p.d / 16);
  const uint32_t pieces = per_token * static_cast<uint32_t>(p.num_tokens);
  const dim3 grid((pieces + kStoreThreads * kStorePieces - 1) / (kStoreThreads * kStorePieces), 2);
  const FastDiv div(per_token);
  const int bs_log2 = p.block_size == 32 ? 5 : 4;
  switch (p.d) {
    case 64:
      return launch_kernel(kv_store_q4_kernel<64>, grid, kStoreThreads, 0, stream, p, div, pieces, bs_log2);
    case 128:
      return launch_kernel(kv_store_q4_kernel<128>, grid, kStoreThreads, 0, stream, p, div, pieces, bs_log2);
    case 256:
      return launch_kernel(kv_store_q4_kernel<256>, grid, kStoreThreads, 0, stream, p, div, pieces, bs_log2);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paq8
