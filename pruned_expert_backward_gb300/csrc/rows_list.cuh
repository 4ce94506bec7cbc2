// The experts of a sorted batch that have rows, for the one-pass kernels of few rows.
#pragma once

#include "linear.cuh"

namespace lrm {

namespace {

constexpr int kWarps = 8;  // of a CTA of such a kernel

// The experts that have rows, listed in shared memory by the whole block;
// returns their number, 0 when the segments are not valid.
struct Rows {
  int e, begin, end;
};
__device__ __forceinline__ int list_experts(const int32_t* seg, int E, int64_t R, Rows* list, int32_t* status) {
  __shared__ int s_count[kWarps];
  __shared__ int s_total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (E + 32 * kWarps - 1) / (32 * kWarps), e0 = threadIdx.x * per, e1 = min(E, e0 + per);
  int ok = 1, count = 0;
  for (int e = e0; e < e1; ++e) {
    const int a = seg[e], b = seg[e + 1];
    ok &= a <= b ? 1 : 0;
    count += a < b ? 1 : 0;
  }
  if (threadIdx.x == 0) ok &= seg[0] == 0 && (int64_t)seg[E] <= R ? 1 : 0;
  int incl = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_count[warp] = incl;
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) set_status(status, LRM_ERR_BAD_SEGMENTS);
    return 0;
  }
  int at = incl - count;
  for (int w = 0; w < warp; ++w) at += s_count[w];
  for (int e = e0; e < e1 && count > 0; ++e) {
    const int a = seg[e], b = seg[e + 1];
    if (a < b) list[at++] = Rows{e, a, b};
  }
  if (threadIdx.x == blockDim.x - 1) s_total = at;
  __syncthreads();
  return s_total;
}

}  // namespace

}  // namespace lrm
