// The 4-bit cache format: codes 0 .. 15 of keys and values with one fp16 scale and
// one fp16 zero per (token, kv head, group of 32 channels), x' = code * scale + zero.
//
// A row of a page is D / 2 bytes, its codes in the order in which a lane of the
// attention's warp MMAs reads them, so that one load brings a lane its codes of all
// G = D / 32 groups:
//   K: 32-bit word t * G + gr (t = 0 .. 3) holds channels 32 gr + 8 t + i at nibble
//      i = 0 .. 7 (lane t of a score MMA's row);
//   V: 16-bit half u * G + gr (u = 0 .. 7) holds channels 32 gr + 4 u + i at nibble
//      i = 0 .. 3 (lane u of an output MMA's channel rows).
// Scales and zeros: K [2][bs][G] a page (the scales, then the zeros; a score needs
// a key's groups together), V [2][G][bs] (an output needs a group's keys together).
#pragma once

#include "common.cuh"

namespace paq8 {

// Byte of channel 8 * o (o: octet, 8 channels) in a K row: one 32-bit word.
__device__ __forceinline__ int q4_k_word(int o, int groups) { return ((o & 3) * groups + (o >> 2)) * 4; }
// Byte of channel 8 * o + 4 * half in a V row: one 16-bit half.
__device__ __forceinline__ int q4_v_half(int o, int half, int groups) {
  return ((2 * (o & 3) + half) * groups + (o >> 2)) * 2;
}

// n / d for 0 <= n < 2^31 by a multiplication (d fixed on the host): with s =
// ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1, n / d = (umulhi(m, n) + n) >> s.
struct FastDiv {
  uint32_t d, m, s;
  explicit FastDiv(uint32_t div = 1) : d(div) {
    s = 0;
    while ((uint64_t{1} << s) < d) ++s;
    m = static_cast<uint32_t>(((((uint64_t{1} << s) - d) << 32) / d) + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

}  // namespace paq8
