// copy_blocks: whole blocks of a paged cache copied to other blocks of it,
// all arrays of the cache (codes and scales of K and V) in one launch.
//
// HBM bound: a pair reads and writes the bytes of one block.  The blocks of
// the four arrays are walked as one run of 16-byte pieces; a thread block
// takes 1024 pieces of one pair (16 KB, four loads in flight a thread before
// the first store), so that few pairs of large blocks still spread over the
// GPU and a list of unused pairs (-1) costs one read each.
#include "common.cuh"
#include "launch.h"
#include "serving.h"

namespace paq8 {

namespace {

constexpr int kThreadsCopy = 256;
constexpr int kPieces = 4;  // 16-byte pieces per thread

__global__ void __launch_bounds__(kThreadsCopy) copy_blocks_kernel(const BlockCopy p, int parts) {
  const int pair = static_cast<int>(blockIdx.x / static_cast<unsigned>(parts));
  const int part = static_cast<int>(blockIdx.x % static_cast<unsigned>(parts));
  const int2 ft = *reinterpret_cast<const int2 *>(p.pairs + 2 * static_cast<int64_t>(pair));
  if (ft.x < 0 || ft.y < 0 || ft.x == ft.y) return;
  if (ft.x >= p.num_blocks || ft.y >= p.num_blocks) {
    if (part == 0 && threadIdx.x == 0) flag_status(p.status, PA_DEV_BAD_BLOCK);
    return;
  }
  uint4 v[kPieces];
  uint4 *to[kPieces];
  const int64_t first = static_cast<int64_t>(part) * (kThreadsCopy * kPieces) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    int64_t at = (first + i * kThreadsCopy) * 16;
    to[i] = nullptr;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (at >= 0 && at < p.bytes[k]) {
        to[i] = reinterpret_cast<uint4 *>(p.base[k] + ft.y * p.bytes[k] + at);
        v[i] = *reinterpret_cast<const uint4 *>(p.base[k] + ft.x * p.bytes[k] + at);
      }
      at -= p.bytes[k];
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (to[i]) *to[i] = v[i];
}

}  // namespace

cudaError_t launch_copy_blocks(const BlockCopy &p, cudaStream_t stream) {
  const int64_t pieces = (p.bytes[0] + p.bytes[1] + p.bytes[2] + p.bytes[3]) / 16;
  const int64_t parts = (pieces + kThreadsCopy * kPieces - 1) / (kThreadsCopy * kPieces);
  const int64_t grid = parts * p.num_pairs;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  copy_blocks_kernel<<<static_cast<unsigned>(grid), kThreadsCopy, 0, stream>>>(
      p, static_cast<int>(parts));
  return cudaGetLastError();
}

}  // namespace paq8
