// What the tile kernels of a CTA pair share: the order of tiles, the row tiles of segments, and the launch.
#pragma once

#include "kernels.h"
#include "linear.cuh"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace lrm {

namespace {

constexpr int kTileRows = 256;   // rows of a pair's tile
constexpr int kBoxBytes = 2048;  // 32 rows x 64 bytes, 64-byte swizzle: 32 bf16 or 16 fp32 columns

// At most N of this thread's bulk stores have not read their shared memory yet.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Waits of whole warps that are ahead of the others: they sleep between polls.  `last`: the wait for everything this
// CTA has under way, which may take as long as the kernel does and outlives an abort; its limit counts from one.
__device__ __noinline__ bool mbar_wait_ahead(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status,
                                             bool last) {
  uint64_t t0 = globaltimer();
  for (uint32_t it = 1; it < (1u << 30); ++it) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    __nanosleep(20);
    if ((it & 63u) == 0) {
      const bool stop = __any_sync(0xffffffffu, *abort_flag != 0);
      if (stop && !last) return false;
      if (last && !stop) t0 = globaltimer();
      if (__any_sync(0xffffffffu, globaltimer() - t0 > kWaitNs)) break;
    }
  }
  *abort_flag = 1;
  set_status(status, LRM_ERR_TIMEOUT);
  return false;
}

// The i-th tile of a CTA pair: round robin, every second round backwards, so that where the tiles get
// shorter along the order (DW: longest expert first) no pair takes the longer one of every round.
__device__ __forceinline__ int nth_tile(int i, int pair, int n_pairs) {
  return i * n_pairs + (i & 1 ? n_pairs - 1 - pair : pair);
}

// The last i in [0, n) with prefix[i] <= v.
__device__ __forceinline__ int last_at_most(const int* prefix, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// Row tiles before each expert (prefix [E + 1], shared memory), formed by all THREADS threads of the CTA: each sums a
// run of experts, a scan over the threads (scan [THREADS / 32]) gives the prefix.  Returns the number of row tiles, 0
// for segments that are not valid.
template <int THREADS>
__device__ __forceinline__ int segment_tiles(const int32_t* seg, int E, int64_t R, int tile_rows, int* prefix,
                                             int* scan, int32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (E + THREADS - 1) / THREADS, e0 = threadIdx.x * per, e1 = min(E, e0 + per);
  int sum = 0, ok = 1;
  for (int e = e0; e < e1; ++e) {
    const int a = __ldg(seg + e), b = __ldg(seg + e + 1);
    ok &= a <= b ? 1 : 0;
    sum += (b - a + tile_rows - 1) / tile_rows;
  }
  if (threadIdx.x == 0) ok &= __ldg(seg) == 0 && (int64_t)__ldg(seg + E) <= R ? 1 : 0;
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  const bool valid = __syncthreads_and(ok) != 0;
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += scan[w];
  for (int e = e0; e < e1; ++e) {
    prefix[e] = run;
    run += (__ldg(seg + e + 1) - __ldg(seg + e) + tile_rows - 1) / tile_rows;
  }
  if (e0 < E && e1 == E) prefix[E] = run;
  __syncthreads();
  if (!valid && threadIdx.x == 0) set_status(status, LRM_ERR_BAD_SEGMENTS);
  return valid ? prefix[E] : 0;
}

// ---------------------------------------------------------------- host side ----------
// Most row tiles there can be.
int64_t row_tiles(const int32_t* seg, int64_t R, int E) {
  return (R + kTileRows - 1) / kTileRows + (seg != nullptr ? E : 0);
}

// `kernel` over `tiles_bound` tiles at most: persistent CTA pairs, as many as fit the GPU.
template <auto kernel, typename... Args>
lrm_status launch_pairs(size_t smem, int threads, int64_t tiles_bound, cudaStream_t s, const Args&... args) {
  if (ensure_max_smem<kernel>((int)smem) != cudaSuccess) return LRM_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // the occupancy query sees the cluster shape only
  static int resident[kDeviceSlots] = {};  // CTA pairs, per device
  const int slot = current_device_slot();
  int pairs = slot >= 0 ? resident[slot] : 0;
  if (pairs == 0) {
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs <= 0) pairs = sm_count() / 2;
    if (slot >= 0) resident[slot] = pairs;
  }
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(2 * (tiles_bound < pairs ? tiles_bound : pairs)));
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return LRM_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? LRM_OK : LRM_ERR_CUDA;
}

}  // namespace

}  // namespace lrm
