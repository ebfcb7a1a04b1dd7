// copy_blocks: whole blocks of a paged cache copied to other blocks of it,
// all arrays of the cache (codes and scales of K and V) in one launch.
//
// HBM bound: a pair reads and writes the bytes of one block.  The blocks of the
// four arrays are walked as one run of bytes, cut into equal parts of at most
// 13 KB.  A thread block is one warp with two parts in shared memory: bulk copies
// bring one in while the part before it goes out, five thread blocks an SM, and no
// thread holds data.  8191 blocks of 24.5 KB (fp8 / 4-bit, 8 kv heads of 128
// channels) take 65 us, 6.3 TB/s read and written (68 when the launch does not
// overlap the work before; so measured, 16-byte loads and stores of 256 threads took
// 86, and more in flight is no faster: 12 KB parts, two read ahead in a ring of four,
// four thread blocks an SM, 72; 8 KB, four ahead of six, 78).
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "programmatic.cuh"
#include "serving.h"

namespace paq8 {

namespace {

constexpr int kPartBytes = 13312;  // at most
constexpr int kRing = 2;           // parts in shared memory
constexpr int kAhead = 1;          // parts being read
constexpr int kBlocksPerSm = 5;
constexpr int kSmemCopy = kRing * kPartBytes;

// The bytes [off, off + bytes) of a block, array by array: f(array, its offset, the
// part's offset, bytes).
template <class F>
__device__ __forceinline__ void for_arrays(const BlockCopy &p, int64_t off, int64_t bytes, F &&f) {
  int64_t start = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t lo = max(off, start), hi = min(off + bytes, start + p.bytes[k]);
    if (lo < hi) f(k, lo - start, static_cast<uint32_t>(lo - off), static_cast<uint32_t>(hi - lo));
    start += p.bytes[k];
  }
}

__global__ void __launch_bounds__(32) copy_blocks_kernel(const BlockCopy p, int parts, int part_bytes) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kRing];
  __shared__ int2 what[kRing];  // destination block, part
  const int lane = threadIdx.x;
  const int64_t items = static_cast<int64_t>(p.num_pairs) * parts;
  const int64_t total = p.bytes[0] + p.bytes[1] + p.bytes[2] + p.bytes[3];
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(smem_u32(full + i), 1);
    fence_barrier_init();
  }
  __syncwarp();
  wait_for_predecessor();  // the pairs, and the blocks themselves
  bool ok = true;
  int n = 0;  // parts whose read was issued; all of this is lane 0's
  // part i has landed: write it
  auto put = [&](int i) {
    const int s = i % kRing;
    if (!mbar_wait(smem_u32(full + s), (i / kRing) & 1)) return false;
    const int2 w = what[s];
    const int64_t off = static_cast<int64_t>(w.y) * part_bytes;
    for_arrays(p, off, min(static_cast<int64_t>(part_bytes), total - off),
               [&](int k, int64_t at, uint32_t in_part, uint32_t bytes) {
                 asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                  p.base[k] + w.x * p.bytes[k] + at),
                              "r"(smem_u32(ring + s * kPartBytes) + in_part), "r"(bytes)
                              : "memory");
               });
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    return true;
  };
  for (int64_t first = blockIdx.x; first < items; first += static_cast<int64_t>(gridDim.x) * 32) {
    // the pairs of this block's next 32 items, one per lane
    const int64_t item = first + static_cast<int64_t>(gridDim.x) * lane;
    int2 ft = make_int2(-1, -1);
    int part = 0;
    if (item < items) {
      ft = *reinterpret_cast<const int2 *>(p.pairs + 2 * (item / parts));
      part = static_cast<int>(item % parts);
    }
    bool copy = ft.x >= 0 && ft.y >= 0 && ft.x != ft.y;
    if (copy && (ft.x >= p.num_blocks || ft.y >= p.num_blocks)) {
      if (part == 0) flag_status(p.status, PA_DEV_BAD_BLOCK);
      copy = false;
    }
    for (unsigned left = __ballot_sync(0xffffffffu, copy); left; left &= left - 1) {
      const int src_lane = __ffs(left) - 1;
      const int from = __shfl_sync(0xffffffffu, ft.x, src_lane);
      const int to = __shfl_sync(0xffffffffu, ft.y, src_lane);
      const int pt = __shfl_sync(0xffffffffu, part, src_lane);
      if (lane != 0 || !ok) continue;
      if (n >= kAhead && !put(n - kAhead)) {
        ok = false;
        continue;
      }
      // the slot's last part, kRing before this one, has left shared memory
      asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kRing - kAhead) : "memory");
      const int s = n % kRing;
      const int64_t off = static_cast<int64_t>(pt) * part_bytes;
      const int64_t bytes = min(static_cast<int64_t>(part_bytes), total - off);
      what[s] = make_int2(to, pt);
      mbar_arrive_expect_tx(smem_u32(full + s), static_cast<uint32_t>(bytes));
      for_arrays(p, off, bytes, [&](int k, int64_t at, uint32_t in_part, uint32_t sz) {
        bulk_load(smem_u32(ring + s * kPartBytes) + in_part, p.base[k] + from * p.bytes[k] + at, sz,
                  smem_u32(full + s));
      });
      ++n;
    }
  }
  if (lane == 0) {
    for (int i = max(0, n - kAhead); ok && i < n; ++i) ok = put(i);
    // a wait ran out: the parts being read may still land, and shared memory is theirs
    // until they do (or another wait as long runs out)
    for (int i = max(0, n - kAhead); !ok && i < n; ++i)
      mbar_wait(smem_u32(full + i % kRing), (i / kRing) & 1);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok) flag_status(p.status, PA_DEV_TIMEOUT);
  }
}

}  // namespace

cudaError_t launch_copy_blocks(const BlockCopy &p, cudaStream_t stream) {
  const int64_t total = p.bytes[0] + p.bytes[1] + p.bytes[2] + p.bytes[3];
  const int64_t parts = (total + kPartBytes - 1) / kPartBytes;
  const int64_t part_bytes = ((total + parts - 1) / parts + 15) / 16 * 16;
  const int64_t grid = std::min<int64_t>(parts * p.num_pairs, 152 * kBlocksPerSm);
  static DeviceOnce configured;
  cudaError_t e = configured.get(nullptr, [](int, int *) {
    return cudaFuncSetAttribute(copy_blocks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemCopy);
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(copy_blocks_kernel, dim3(static_cast<unsigned>(grid)), 32, kSmemCopy, stream, p,
                       static_cast<int>(parts), static_cast<int>(part_bytes));
}

}  // namespace paq8
