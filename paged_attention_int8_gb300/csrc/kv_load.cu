// kv_load: pages of a cache read back as packed bf16 rows, for each of the three
// formats.  Row j of sequence s (j below its length) is
//   q8    code * scale                    of the row's 32-channel group
//   f8v4  K: the e4m3 value;  V: code * scale + zero of the token
//   q4    code * scale + zero             of the row's 32-channel group
// in fp32 (the products are exact), rounded once more to bf16.
//
// Bound by HBM: the page bytes read and 4 D bytes written a (key, kv head).  One warp
// a (page, kv head): a page's arrays are contiguous for a head, and a lane writes
// 8 channels (16 bytes) of a row at a time.  Values that lie
// channel-major (q8, f8v4) are transposed in registers: a lane takes 8 keys of 8 channels.
// 4 bits: 199,000 keys (8 heads, D 128, 1.07 GB) 159 us, 0.96 of the copy rate; with one word
// of codes a lane and step 243.
#include "attn_common.cuh"
#include "attn_f8v4.cuh"
#include "programmatic.cuh"
#include "q4.cuh"
#include "q4.h"

namespace paq8 {

constexpr int kLoadWarps = 4;

__device__ __forceinline__ float half_at(const uint16_t *p) { return __half2float(__ushort_as_half(*p)); }
__device__ __forceinline__ float half_of(uint32_t w, int i) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> (16 * i))));
}

// N 32-bit words from memory, in loads as wide as they are aligned.
template <int N>
__device__ __forceinline__ void load_words(const void *src, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *static_cast<const uint32_t *>(src);
  } else if constexpr (N == 2) {
    const uint2 v = *static_cast<const uint2 *>(src);
    w[0] = v.x;
    w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(src) + 4 * i);
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf162(x[0], x[1]), pack_bf162(x[2], x[3]), pack_bf162(x[4], x[5]),
                    pack_bf162(x[6], x[7]));
}

__device__ __forceinline__ void store_row(uint16_t *dst, uint4 v) { *reinterpret_cast<uint4 *>(dst) = v; }

// Values of byte b of w, signed.
__device__ __forceinline__ float byte_code(uint32_t w, int b) {
  return static_cast<float>(static_cast<int8_t>((w >> (8 * b)) & 0xffu));
}

template <CacheFormat F, int D, int BS>
__global__ void __launch_bounds__(32 * kLoadWarps) kv_load_kernel(const __grid_constant__ KvLoad p) {
  constexpr int G = D / 32;
  constexpr int kOctets = D / 8;
  wait_for_predecessor();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kLoadWarps + (threadIdx.x >> 5);
  const int h = static_cast<int>(unit % p.hk);
  const int64_t item = unit / p.hk;
  if (item >= p.num_rows / BS + p.num_seqs) return;
  // row0, room and length of a sequence; whether they fit
  struct Bounds {
    int row0, room, n;
  };
  const auto bounds_of = [&](int seq) {
    const int row0 = p.cu_seqlens_k[seq], room = p.cu_seqlens_k[seq + 1] - row0;
    return Bounds{row0, room, p.load_lens ? p.load_lens[seq] : room};
  };
  const auto fit = [&](const Bounds &b) {
    return b.row0 >= 0 && b.room >= 0 && b.row0 <= p.num_rows - b.room && b.n >= 0 && b.n <= b.room;
  };
  // No item need be that of a sequence whose bounds are bad: item i looks at sequence i (there are
  // no fewer items than sequences), on its way to its own.
  Bounds other{0, 0, 0};
  if (h == 0 && item < p.num_seqs) other = bounds_of(static_cast<int>(item));
  const int seq = find_seq(p.cu_seqlens_k, p.num_seqs, BS, static_cast<int>(item), lane);
  const Bounds own = bounds_of(seq);
  if (!fit(other) && lane == 0) flag_status(p.status, PA_DEV_BAD_SEQ);
  if (!fit(own)) return;
  const int row0 = own.row0, n = own.n;
  const int page = static_cast<int>(item) - (row0 / BS + seq);
  if (page < 0 || page * BS >= n) return;
  const int block = page < p.table_columns
                        ? p.block_table[static_cast<int64_t>(seq) * p.table_stride + page]
                        : -1;
  if (block < 0 || block >= p.num_blocks) {
    if (lane == 0) flag_status(p.status, PA_DEV_BAD_BLOCK);
    return;
  }
  const int keys = min(BS, n - page * BS);
  const int64_t at = static_cast<int64_t>(block) * p.hk + h;
  const int64_t out0 = static_cast<int64_t>(row0) + page * BS;
  uint16_t *kout = p.key + out0 * p.key_stride + h * D;
  uint16_t *vout = p.value + out0 * p.value_stride + h * D;

  if constexpr (F == CacheFormat::q4) {
    // a lane takes the codes that stand together: of key row r, words 8 t .. 8 t + 7 of every
    // group; of value row r, the halves 2 t and 2 t + 1.  Four lanes write whole groups.
#pragma unroll
    for (int i0 = 0; i0 < BS * 4; i0 += 32) {
      const int r = (i0 + lane) >> 2, t = lane & 3;
      if (r >= keys) continue;
      const uint8_t *codes = static_cast<const uint8_t *>(p.array[0]) + (at * BS + r) * (D / 2) + t * (4 * G);
      const uint16_t *sc = static_cast<const uint16_t *>(p.array[1]) + at * (2 * BS * G) + r * G;
      uint32_t w[G], s[G / 2], z[G / 2];
      load_words(codes, w);
      load_words(sc, s);
      load_words(sc + BS * G, z);
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const float sf = half_of(s[gr >> 1], gr & 1), zf = half_of(z[gr >> 1], gr & 1);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(static_cast<float>((w[gr] >> (4 * i)) & 0xfu), sf, zf);
        store_row(kout + r * p.key_stride + gr * 32 + t * 8, pack_bf16x8(x));
      }
    }
#pragma unroll
    for (int i0 = 0; i0 < BS * 4; i0 += 32) {
      const int r = (i0 + lane) >> 2, t = lane & 3;
      if (r >= keys) continue;
      const uint8_t *codes = static_cast<const uint8_t *>(p.array[2]) + (at * BS + r) * (D / 2) + t * (4 * G);
      const uint16_t *sc = static_cast<const uint16_t *>(p.array[3]) + at * (2 * BS * G) + r;
      uint32_t w[G];
      load_words(codes, w);
      float sf[G], zf[G];
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        sf[gr] = half_at(sc + gr * BS);
        zf[gr] = half_at(sc + (G + gr) * BS);
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const uint32_t lo = w[gr >> 1] >> (16 * (gr & 1)), hi = w[(G + gr) >> 1] >> (16 * (gr & 1));
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = fmaf(static_cast<float>(((i < 4 ? lo : hi) >> (4 * (i & 3))) & 0xfu), sf[gr], zf[gr]);
        store_row(vout + r * p.value_stride + gr * 32 + t * 8, pack_bf16x8(x));
      }
    }
    return;
  } else {
    // ---- keys, token-major: 16 channels a lane and step
    constexpr int kRuns = D / 16;
#pragma unroll
    for (int i0 = 0; i0 < BS * kRuns; i0 += 32) {
      const int r = (i0 + lane) / kRuns, o = (i0 + lane) % kRuns;
      if (r >= keys) continue;
      uint32_t w[4];
      load_words(static_cast<const uint8_t *>(p.array[0]) + (at * BS + r) * D + o * 16, w);
      float s = 0.0f;
      if constexpr (F == CacheFormat::q8)
        s = half_at(static_cast<const uint16_t *>(p.array[1]) + (at * BS + r) * G + (o >> 1));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[8];
        if constexpr (F == CacheFormat::q8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = byte_code(w[2 * half + (i >> 2)], i & 3) * s;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = e4m3x2_to_half2(w[2 * half + (i >> 1)] >> (16 * (i & 1)));
            x[2 * i] = half_of(v, 0);
            x[2 * i + 1] = half_of(v, 1);
          }
        }
        store_row(kout + r * p.key_stride + o * 16 + half * 8, pack_bf16x8(x));
      }
    }
    // ---- values, channel-major: 8 keys of 8 channels a lane and step
#pragma unroll
    for (int i0 = 0; i0 < BS / 8 * kOctets; i0 += 32) {
      const int r = (i0 + lane) / kOctets * 8, o = (i0 + lane) % kOctets;  // keys r .. r + 7
      if (r >= keys || r >= BS) continue;
      constexpr int W = F == CacheFormat::q8 ? 2 : 1;  // words of a channel's codes
      uint32_t w[8][W], s[4], z[4];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        load_words(static_cast<const uint8_t *>(p.array[F == CacheFormat::q8 ? 2 : 1]) +
                       ((at * D + o * 8 + c) * BS + r) / (F == CacheFormat::q8 ? 1 : 2),
                   w[c]);
      if constexpr (F == CacheFormat::q8) {
        load_words(static_cast<const uint16_t *>(p.array[3]) + (at * G + (o >> 2)) * BS + r, s);
      } else {
        load_words(static_cast<const uint16_t *>(p.array[2]) + at * BS + r, s);
        load_words(static_cast<const uint16_t *>(p.array[3]) + at * BS + r, z);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sf = half_of(s[j >> 1], j & 1);
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if constexpr (F == CacheFormat::q8)
            x[c] = byte_code(w[c][j >> 2], j & 3) * sf;
          else
            x[c] = fmaf(static_cast<float>((w[c][0] >> (4 * j)) & 0xfu), sf, half_of(z[j >> 1], j & 1));
        }
        if (r + j < keys) store_row(vout + (r + j) * p.value_stride + o * 8, pack_bf16x8(x));
      }
    }
  }
}

template <CacheFormat F, int D>
static cudaError_t launch_load_d(const KvLoad &p, dim3 grid, cudaStream_t stream) {
  return p.block_size == 32
             ? launch_kernel(kv_load_kernel<F, D, 32>, grid, 32 * kLoadWarps, 0, stream, p)
             : launch_kernel(kv_load_kernel<F, D, 16>, grid, 32 * kLoadWarps, 0, stream, p);
}

template <CacheFormat F>
static cudaError_t launch_load_f(const KvLoad &p, dim3 grid, cudaStream_t stream) {
  switch (p.d) {
    case 64: return launch_load_d<F, 64>(p, grid, stream);
    case 128: return launch_load_d<F, 128>(p, grid, stream);
    case 256: return launch_load_d<F, 256>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_load(const KvLoad &p, CacheFormat format, cudaStream_t stream) {
  // pages of sequence s start at item cu[s] / bs + s: at most rows / bs + seqs items
  const int64_t units =
      (static_cast<int64_t>(p.num_rows) / p.block_size + p.num_seqs) * p.hk;
  const dim3 grid(static_cast<unsigned>((units + kLoadWarps - 1) / kLoadWarps));
  switch (format) {
    case CacheFormat::q8: return launch_load_f<CacheFormat::q8>(p, grid, stream);
    case CacheFormat::f8v4: return launch_load_f<CacheFormat::f8v4>(p, grid, stream);
    case CacheFormat::q4: return launch_load_f<CacheFormat::q4>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paq8
