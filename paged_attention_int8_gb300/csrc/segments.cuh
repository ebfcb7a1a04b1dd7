// Key segments of a query row: the fp32 triples (m, l, acc) that the blocks of an attention
// kernel leave in a workspace, and their join.
#pragma once

#include "common.cuh"

namespace paq8 {

constexpr int kMaxSegments = 64;

// Joins the n triples of a row by one warp: M = max m_k (log2 units), w_k = 2^(m_k - M),
// out = sum w_k acc_k / sum w_k l_k, the sink (log2 units, -inf: none) as one term more of
// the sum.  A triple whose m is -inf holds no acc.  A row without a term: 0 and -inf.
template <int D>
__device__ __forceinline__ void join_row(const float *acc_rows, const float2 *ml_row, int n, float sink,
                                         uint16_t *out, float *lse, int lane) {
  static_assert(kMaxSegments <= 64, "two segments a lane");
  constexpr int V = D / 32;  // channels a lane
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (lane + 32 * k < n) {
      const float2 ml = ml_row[lane + 32 * k];
      m[k] = ml.x;
      l[k] = ml.y;
    }
  // the first segments' rows come along with their weights
  constexpr int kEarly = 8;
  float2 x[kEarly][V / 2];
  const float *src = acc_rows + lane * V;
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
#pragma unroll
    for (int v = 0; v < V / 2; ++v)
      x[k][v] = k < n ? *reinterpret_cast<const float2 *>(src + k * D + 2 * v) : make_float2(0.0f, 0.0f);
  float top = fmax3(m[0], m[1], sink);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float mu = top == -INFINITY ? 0.0f : top;
  const float w[2] = {fast_exp2(m[0] - mu), fast_exp2(m[1] - mu)};
  float sum = w[0] * l[0] + w[1] * l[1];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  sum += fast_exp2(sink - mu);
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const float wk = __shfl_sync(0xffffffffu, w[0], k);
    if (wk == 0.0f) continue;
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
      acc[2 * v] = fmaf(wk, x[k][v].x, acc[2 * v]);
      acc[2 * v + 1] = fmaf(wk, x[k][v].y, acc[2 * v + 1]);
    }
  }
#pragma unroll 4
  for (int k = kEarly; k < n; ++k) {
    const float wk = __shfl_sync(0xffffffffu, k < 32 ? w[0] : w[1], k & 31);
    if (wk == 0.0f) continue;
#pragma unroll
    for (int v = 0; v < V / 2; ++v) {
      const float2 y = *reinterpret_cast<const float2 *>(src + static_cast<int64_t>(k) * D + 2 * v);
      acc[2 * v] = fmaf(wk, y.x, acc[2 * v]);
      acc[2 * v + 1] = fmaf(wk, y.y, acc[2 * v + 1]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int v = 0; v < V; v += 2)
    *reinterpret_cast<uint32_t *>(out + lane * V + v) = pack_bf162(acc[v] * inv, acc[v + 1] * inv);
  if (lane == 0 && lse) *lse = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace paq8
