// kv_store in the 4-bit format (q4.cuh).  Per (token, kv head, 32 channels) of K and V:
//   lo, hi = min, max;  s = max((hi - lo) * fp32(1 / 15), 1e-8)           (fp32)
//   code = clamp(round_half_away((x - lo) / s), 0, 15)   (the IEEE fp32 quotient)
//   scale = fp16(s), zero = fp16(lo), to nearest even.
//
// Bound by HBM: 4 D bytes read and D + D / 4 written a (token, kv head).  A thread
// takes 8 channels (one 16-byte load), four neighbouring lanes a group (two
// exchanges for its extremes).  Its codes are one word of a K row or two halves of a
// V row; a warp covers whole rows, so the pieces of a row meet in its sectors.
// Several pieces a thread keep their loads in flight together.
#include "launch.h"
#include "programmatic.cuh"
#include "q4.cuh"
#include "q4.h"
#include "q8_quant.cuh"

namespace paq8 {

constexpr int kStoreThreads = 256;
constexpr int kStorePieces = 4;  // 16-byte pieces a thread, of K and of V

// The codes of 8 values in a group with minimum lo and step s (rs = 1 / s), channel i
// at nibble i.  c = the integer next to v / s from one fused multiply-add of
// 1.5 * 2^23, exact unless v / s lies within 2^-15 of a tie, which tie_code_bits
// decides; 0 <= v <= RN(hi - lo), so 0 <= v * rs < 15.00001 and no clamp is needed.
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], float lo, float s, float rs) {
  constexpr float kShift = 12582912.0f;  // 1.5 * 2^23
  constexpr float kFar = 0.5f - 0x1p-15f;
  uint32_t tb[8];
  float v[8], d[8], nc[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __fsub_rn(x[i], lo);
    const float t = __fmaf_rn(v[i], rs, kShift);
    nc[i] = __fsub_rn(kShift, t);
    d[i] = __fmaf_rn(v[i], rs, nc[i]);
    tb[i] = __float_as_uint(t);
    near = near || fabsf(d[i]) >= kFar;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(d[i]) >= kFar)
        tb[i] = tie_code_bits(v[i], s, __fsub_rn(copysignf(0.5f, d[i]), nc[i]));
  }
  uint32_t word = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= (tb[i] & 0xfu) << (4 * i);
  return word;
}

template <int D>
__global__ void __launch_bounds__(kStoreThreads)
    kv_store_q4_kernel(const __grid_constant__ KvStoreQ4 p, const FastDiv per_token,
                       const uint32_t pieces, const int bs_log2) {
  constexpr int G = D / 32;
  constexpr int kOctets = D / 8;
  wait_for_predecessor();
  const bool values = blockIdx.y != 0;
  const uint16_t *src = values ? p.value : p.key;
  const int64_t stride = values ? p.value_stride : p.key_stride;
  const int64_t num_slots = static_cast<int64_t>(p.num_blocks) << bs_log2;
  const uint32_t first = blockIdx.x * (kStoreThreads * kStorePieces) + threadIdx.x;
  uint4 raw[kStorePieces];
  int64_t slot[kStorePieces];
  uint32_t inner[kStorePieces];  // piece within the token
#pragma unroll
  for (int k = 0; k < kStorePieces; ++k) {
    const uint32_t i = first + k * kStoreThreads;
    slot[k] = -1;
    raw[k] = make_uint4(0u, 0u, 0u, 0u);
    inner[k] = 0;
    if (i < pieces) {
      const uint32_t token = per_token.div(i);
      inner[k] = i - token * per_token.d;
      slot[k] = p.slot_mapping[token];
      raw[k] = *reinterpret_cast<const uint4 *>(src + token * stride + inner[k] * 8);
    }
  }
#pragma unroll
  for (int k = 0; k < kStorePieces; ++k) {
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
    float lo = fmin3(fmin3(x[0], x[1], x[2]), fmin3(x[3], x[4], x[5]), fminf(x[6], x[7]));
    float hi = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (slot[k] < 0) continue;  // the same for the four lanes of a group
    if (slot[k] >= num_slots) {
      if (inner[k] == 0 && !values) flag_status(p.status, PA_DEV_BAD_SLOT);
      continue;
    }
    float s = __fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f);
    s = s < 1e-8f ? 1e-8f : s;
    const uint32_t word = q4_codes(x, lo, s, __frcp_rn(s));
    const int h = static_cast<int>(inner[k] / kOctets), o = static_cast<int>(inner[k] % kOctets);
    const int off = static_cast<int>(slot[k] & (p.block_size - 1));
    const int64_t page = (slot[k] >> bs_log2) * p.hk + h;
    const int64_t row = (page << bs_log2) + off;
    const uint16_t s16 = __half_as_ushort(__float2half_rn(s));
    const uint16_t z16 = __half_as_ushort(__float2half_rn(lo));
    const int plane = p.block_size * G;
    if (!values) {
      *reinterpret_cast<uint32_t *>(p.k_cache + row * (D / 2) + q4_k_word(o, G)) = word;
      if ((o & 3) == 0) {
        uint16_t *dst = p.k_scale + page * (2 * plane) + off * G + (o >> 2);
        dst[0] = s16;
        dst[plane] = z16;
      }
    } else {
      uint8_t *dst = p.v_cache + row * (D / 2);
      *reinterpret_cast<uint16_t *>(dst + q4_v_half(o, 0, G)) = static_cast<uint16_t>(word);
      *reinterpret_cast<uint16_t *>(dst + q4_v_half(o, 1, G)) = static_cast<uint16_t>(word >> 16);
      if ((o & 3) == 0) {
        uint16_t *sc = p.v_scale + page * (2 * plane) + (o >> 2) * p.block_size + off;
        sc[0] = s16;
        sc[plane] = z16;
      }
    }
  }
}

cudaError_t launch_kv_store_q4(const KvStoreQ4 &p, cudaStream_t stream) {
  const uint32_t per_token = static_cast<uint32_t>(p.hk) * (p.d / 8);
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
