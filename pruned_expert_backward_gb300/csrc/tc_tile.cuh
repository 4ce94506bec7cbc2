// What the tile kernels of a CTA pair share: the order of tiles, the way of an epilogue's columns out of registers,
// tensor maps of outputs, and the launch.
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

// 32 columns of one row per lane go out: whole 32-row blocks through the warp's next box(es) and TMA
// (which clips columns past the tensor), others by each live lane.
template <int BOXES>
struct Out {
  uint8_t* boxes;
  uint32_t boxes_s;
  int next;
  __device__ __forceinline__ void box(const uint4 (&q)[4], const CUtensorMap* map, int lane, int n, int row, int e) {
    if (lane == 0) bulk_wait_read<BOXES - 1>();  // the store that used this box has read it
    __syncwarp();
    uint8_t* line = boxes + next * kBoxBytes + lane * 64;
    const int swz = (lane >> 1) & 3;  // 64-byte swizzle: piece j of row r sits at j ^ ((r >> 1) & 3)
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(line + ((j ^ swz) << 4)) = q[j];
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_3d(map, boxes_s + next * kBoxBytes, n, row, e);
    next = next + 1 == BOXES ? 0 : next + 1;
  }
  template <typename T>
  __device__ __forceinline__ void put(const float (&v)[32], const CUtensorMap* map, int lane, int n, int cols, int row,
                                      int e, bool whole, bool live, T* row_ptr) {
    constexpr int VN = VecTraits<T>::N;
    constexpr int PC = 4 * VN;  // columns of a box
#pragma unroll
    for (int h = 0; h < 32 / PC; ++h) {
      uint4 q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) f[i] = v[h * PC + j * VN + i];
        q[j] = pack(f);
      }
      const int c0 = n + h * PC;
      if (whole) {
        if (c0 < cols) box(q, map, lane, c0, row, e);  // warp-uniform
      } else if (live) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + j * VN < cols) st16(row_ptr + c0 + j * VN, q[j]);
      }
    }
  }
};

// v += 32 values of a row of T at column n (columns past `cols` are left alone).
template <typename T>
__device__ __forceinline__ void add_row(float (&v)[32], const T* row, int n, int cols) {
  constexpr int VN = VecTraits<T>::N;
#pragma unroll
  for (int j = 0; j < 32 / VN; ++j)
    if (n + j * VN < cols) {
      float f[VN];
      unpack(*reinterpret_cast<const uint4*>(row + n + j * VN), f);
#pragma unroll
      for (int i = 0; i < VN; ++i) v[j * VN + i] += f[i];
    }
}

template <typename T>
__device__ __forceinline__ void add_vectors(float (&v)[32], const uint4* r) {
  constexpr int VN = VecTraits<T>::N;
#pragma unroll
  for (int j = 0; j < 32 / VN; ++j) {
    float f[VN];
    unpack(r[j], f);
#pragma unroll
    for (int i = 0; i < VN; ++i) v[j * VN + i] += f[i];
  }
}

template <int ACT>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act_value<ACT>(v[i]);
}

// ---------------------------------------------------------------- host side ----------
// [d2][d1][d0] of 2- or 4-byte elements, d0 contiguous (a multiple of 16 bytes), with a {b0, b1, 1} box.
bool make_map(CUtensorMap* m, const void* base, bool f32, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1,
              uint64_t stride2, uint32_t b0, uint32_t b1, bool operand) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {b0, b1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     operand ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     operand ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An output [groups][rows][cols] in 32-row boxes of 64 bytes; halves: [rows][2][cols] seen as two groups.
bool output_map(CUtensorMap* m, const void* base, bool f32, uint64_t cols, uint64_t rows, uint64_t groups,
                bool halves = false) {
  const uint64_t b = f32 ? 4 : 2, line = cols * b * (halves ? 2 : 1);
  return make_map(m, base, f32, cols, rows, groups, line, halves ? cols * b : rows * line, f32 ? 16 : 32, 32, false);
}

// Most row tiles there can be, and about how many (every segment ends in half a tile).
int64_t row_tiles(const int32_t* seg, int64_t R, int E) {
  return (R + kTileRows - 1) / kTileRows + (seg != nullptr ? E : 0);
}
int64_t likely_row_tiles(const int32_t* seg, int64_t R, int E) {
  return (R + kTileRows - 1) / kTileRows + (seg != nullptr ? (R < E ? R : E) / 2 : 0);
}

// Tile width by the waves of tiles over the CTA pairs: a K slice of a 256-column tile takes 0.26 us (its
// products), one of a 128- or 64-column tile 0.155 us (the operands' way in).  On a tie the narrower: more
// SMs then share the reading of the weights.
template <typename F>
lrm_status with_width(int64_t tiles_m, int N, int least, F&& f) {
  const int64_t pairs = sm_count() / 2;
  auto cost = [&](int bn, int slice) { return (tiles_m * ((N + bn - 1) / bn) + pairs - 1) / pairs * slice; };
  const int64_t c256 = cost(256, 5), c128 = cost(128, 3), c64 = least > 64 ? INT64_MAX : cost(64, 3);
  if (c64 <= c128 && c64 <= c256) return f(IntTag<64>{});
  return c128 <= c256 ? f(IntTag<128>{}) : f(IntTag<256>{});
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
