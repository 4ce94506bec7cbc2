// lrm_fp8_quantize and lrm_fp8_quantize_weight: values in e4m3 with an fp32 scale for each block of 128.
//
//   top = max(largest magnitude of the block, 2^-100),  scale = top / 448,  q = e4m3(x * (448 / top))
//
// with divisions rounded to nearest, so that a block's largest value is +-448 and an infinity or a NaN makes its
// whole block NaN.  (2^-100 keeps 448 / top finite; all-zero blocks need no branch.)
//
// Rows: 16 lanes take a block of 128 columns of one row, 8 values each, and write its 128 bytes to every row of the
// sorted batch that the token has: a token's row is read and rounded once, whatever k is.  Bound by memory (mostly the
// k writes): 8192 tokens of 2048 bf16 to 65536 rows 28 us, 0.90 of the copy rate.
// Weights: a CTA takes a block of 128 x 128, 16 lanes a row, 8 rows in flight each; the maximum goes through
// shared memory while the block stays in registers.  Bound by reading W: 128 x 1536 x 2048 bf16 186 us, 0.96 of the
// copy rate with three CTAs a multiprocessor (two 222 us, five, which spill, 231 us).
#include "fp8.cuh"
#include "kernels.h"

namespace lrm {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // blocks of columns a CTA has under way at a time

// 8 consecutive values; `now` keeps the loads of a batch in front of their first use.
struct Eight {
  uint4 lo, hi;
};
template <typename T>
__device__ __forceinline__ Eight load8(const T* p) {
  Eight v;
  v.lo = ld_stream16_now(p);
  v.hi = VecTraits<T>::N == 4 ? ld_stream16_now(p + 4) : make_uint4(0, 0, 0, 0);
  return v;
}
__device__ __forceinline__ Eight none8() { return Eight{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
template <typename T>
__device__ __forceinline__ void values8(const Eight& v, float (&f)[8]) {
  if constexpr (VecTraits<T>::N == 8) {
    unpack(v.lo, f);
  } else {
    float a[4], b[4];
    unpack(v.lo, a);
    unpack(v.hi, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
}
__device__ __forceinline__ uint32_t top8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  return m;
}
__device__ __forceinline__ float block_top(uint32_t bits) {
  return __uint_as_float(max(bits, __float_as_uint(kQLeast)));
}
__device__ __forceinline__ uint2 to_e4m3(const float (&f)[8], float inv) {
  return make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// Unit u = t * nb + b is block b of row t, one to a group of 16 lanes.  With row_of_pair, row t goes to the rows of its
// k pairs.  (Two units a group: 64 tokens to 512 rows of 2048 2.8 us, 2.1 us so; long batches alike.)
template <typename T, bool SORTED>
__global__ void __launch_bounds__(kThreads)
    quantize_rows_kernel(const T* __restrict__ x, const int32_t* __restrict__ row_of_pair, int64_t units, int k, int K,
                         int nb, int64_t cap, uint8_t* __restrict__ q, float* __restrict__ scale,
                         int32_t* __restrict__ status) {
  chain_wait();
  const int lane = threadIdx.x & 15;
  const int64_t u = (int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4), t = u / nb;
  const int b = (int)(u - t * nb), c = b * kQBlock + lane * 8;
  const bool here = u < units;  // the same in all 16 lanes
  const Eight v = here && c < K ? load8(x + t * K + c) : none8();
  const int32_t row = SORTED && here && lane < k ? __ldg(row_of_pair + t * k + lane) : -1;
  float f[8];
  values8<T>(v, f);
  uint32_t m = top8(f);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float top = block_top(m);
  const float s = __fdiv_rn(top, kQTop);
  const uint2 out = to_e4m3(f, __fdiv_rn(kQTop, top));
  if (SORTED) {
    const int64_t mine = checked_row(row, cap, b == 0 ? status : nullptr);
    if (mine >= 0) scale[mine * nb + b] = s;
    for (int j = 0; j < k; ++j) {
      const int64_t r = __shfl_sync(0xffffffffu, mine, j, 16);
      if (r >= 0 && c < K) *reinterpret_cast<uint2*>(q + r * K + c) = out;
    }
  } else if (here) {
    if (lane == 0) scale[t * nb + b] = s;
    if (c < K) *reinterpret_cast<uint2*>(q + t * K + c) = out;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, VecTraits<T>::N == 8 ? 3 : 2)
    quantize_weight_kernel(const T* __restrict__ w, int N, int K, int nb, int kb, uint8_t* __restrict__ q,
                           float* __restrict__ scale) {
  constexpr int U = kQBlock / kGroups;  // rows of a group of 16 lanes
  __shared__ uint32_t s_top[kThreads / 32];
  chain_wait();
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int bk = blockIdx.x % kb, gn = blockIdx.x / kb;
  const int g = gn / nb, n0 = (gn - g * nb) * kQBlock, c = bk * kQBlock + lane * 8;
  const int64_t base = ((int64_t)g * N + n0) * K + c;
  Eight v[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int r = group + i * kGroups;
    v[i] = n0 + r < N && c < K ? load8(w + base + (int64_t)r * K) : none8();
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float f[8];
    values8<T>(v[i], f);
    m = max(m, top8(f));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max(m, s_top[i]);
  const float top = block_top(m), inv = __fdiv_rn(kQTop, top);
  if (threadIdx.x == 0) scale[(int64_t)gn * kb + bk] = __fdiv_rn(top, kQTop);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int r = group + i * kGroups;
    if (n0 + r < N && c < K) {
      float f[8];
      values8<T>(v[i], f);
      *reinterpret_cast<uint2*>(q + base + (int64_t)r * K) = to_e4m3(f, inv);
    }
  }
}

}  // namespace

void launch_fp8_quantize(const void* x, const int32_t* row_of_pair, int64_t T, int32_t k, int32_t K, lrm_dtype dt,
                         int64_t cap, void* q, float* scale, int32_t* status, cudaStream_t s) {
  const int nb = (K + kQBlock - 1) / kQBlock;
  const int64_t units = T * nb, blocks = (units + kGroups - 1) / kGroups;
  auto go = [&](auto kernel, auto* at) {
    launch_chained(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, at, row_of_pair, units, (int)k, (int)K, nb,
                   cap, static_cast<uint8_t*>(q), scale, status);
  };
  auto typed = [&](auto* at) {
    using T_ = std::remove_cv_t<std::remove_pointer_t<decltype(at)>>;
    row_of_pair != nullptr ? go(quantize_rows_kernel<T_, true>, at) : go(quantize_rows_kernel<T_, false>, at);
  };
  dt == LRM_BF16 ? typed(static_cast<const __nv_bfloat16*>(x)) : typed(static_cast<const float*>(x));
}

void launch_fp8_quantize_weight(const void* w, int32_t G, int32_t N, int32_t K, lrm_dtype dt, void* q, float* scale,
                                cudaStream_t s) {
  const int nb = (N + kQBlock - 1) / kQBlock, kb = (K + kQBlock - 1) / kQBlock;
  const dim3 grid((unsigned)((int64_t)G * nb * kb));
  if (dt == LRM_BF16)
    launch_chained(quantize_weight_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s,
                   static_cast<const __nv_bfloat16*>(w), (int)N, (int)K, nb, kb, static_cast<uint8_t*>(q), scale);
  else
    launch_chained(quantize_weight_kernel<float>, grid, dim3(kThreads), 0, s, static_cast<const float*>(w), (int)N,
                   (int)K, nb, kb, static_cast<uint8_t*>(q), scale);
}

}  // namespace lrm
