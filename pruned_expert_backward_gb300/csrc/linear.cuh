// Activations of lrm_linear and their derivatives, and the rows of an expert.
#pragma once

#include "common.cuh"

namespace lrm {

// sigmoid(z) and the normal distribution's Phi(z), phi(z) in fp32.  The fast exponential and quotient
// err by a few units of 2^-23 (2 + 1.2 |z| of them for exp(z), where the result is near 0 or z); the
// exact ones took the gradient kernel from the memory's rate to a third of it.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float norm_cdf(float z) { return 0.5f * (1.f + erff(z * 0.70710678118654752f)); }
__device__ __forceinline__ float norm_pdf(float z) { return 0.39894228040143268f * __expf(-0.5f * z * z); }

// act(z) of the one-input activations (SwiGLU takes two: SiLU(gate) * up).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == LRM_ACT_RELU) return fmaxf(z, 0.f);
  if (ACT == LRM_ACT_GELU) return z * norm_cdf(z);
  if (ACT == LRM_ACT_SILU || ACT == LRM_ACT_SWIGLU) return z * sigmoid_f(z);
  return z;
}
// act'(z); ReLU's derivative at 0 is 0.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == LRM_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (ACT == LRM_ACT_GELU) return fmaf(z, norm_pdf(z), norm_cdf(z));
  if (ACT == LRM_ACT_SILU || ACT == LRM_ACT_SWIGLU) {
    const float s = sigmoid_f(z);
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

// Calls f with the activation as a compile-time constant (IntTag<ACT>).
template <int V>
struct IntTag {
  static constexpr int value = V;
};
template <typename F>
inline void with_act(lrm_act act, F&& f) {
  switch (act) {
    case LRM_ACT_RELU: f(IntTag<LRM_ACT_RELU>{}); break;
    case LRM_ACT_GELU: f(IntTag<LRM_ACT_GELU>{}); break;
    case LRM_ACT_SILU: f(IntTag<LRM_ACT_SILU>{}); break;
    case LRM_ACT_SWIGLU: f(IntTag<LRM_ACT_SWIGLU>{}); break;
    default: f(IntTag<LRM_ACT_NONE>{}); break;
  }
}

// seg is NULL for one dense problem of R rows, else [E + 1] and a segmentation of [0, seg[E]] within
// [0, R].  Block-wide vote; a broken one is recorded and the block computes nothing.
__device__ __forceinline__ bool rows_valid(const int32_t* seg, int E, int64_t R, int32_t* status) {
  if (seg == nullptr) return true;
  int ok = 1;
  for (int e = threadIdx.x; e < E; e += blockDim.x) ok &= seg[e] <= seg[e + 1] ? 1 : 0;
  if (threadIdx.x == 0) ok &= (seg[0] == 0 && (int64_t)seg[E] <= R) ? 1 : 0;
  const bool valid = __syncthreads_and(ok) != 0;
  if (!valid && threadIdx.x == 0) set_status(status, LRM_ERR_BAD_SEGMENTS);
  return valid;
}
__device__ __forceinline__ int seg_at(const int32_t* seg, int e, int64_t R) {
  return seg == nullptr ? (e == 0 ? 0 : (int)R) : seg[e];
}

}  // namespace lrm
