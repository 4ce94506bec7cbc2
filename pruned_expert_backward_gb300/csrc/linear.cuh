// Activations of lrm_linear and their derivatives, and the rows of an expert.
#pragma once

#include "common.cuh"

namespace lrm {

// sigmoid(z) in fp32.  The fast exponential and quotient err by a few units of 2^-23 (2 + 1.2 |z| of them
// for exp(z), where the result is near 0 or z); with the exact ones the gradient kernel took 195 us
// instead of 138 us on 65536 x 768.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// The normal distribution's Phi(z), and exp(-z^2 / 2) on the way.  With x = |z| / sqrt 2 the tail is
// erfc(x) / 2, and erfc(x) = t P(t) exp(-x^2) for t = 1 / (1 + 0.45 x): P is a polynomial fitted here to
// exp(x^2) erfc(x) / t for the least relative error over x in [0, 9.5] (5e-7 in fp32 arithmetic, so small
// values of Phi keep their relative accuracy).  No branch, one exponential, one quotient.
__device__ __forceinline__ float norm_cdf(float z, float* exp_out) {
  const float t = __fdividef(1.f, fmaf(0.45f * 0.70710678118654752f, fabsf(z), 1.f));
  float p = 0.06631968915462494f;
  p = fmaf(p, t, -0.23788957297801971f);
  p = fmaf(p, t, 0.20455458760261536f);
  p = fmaf(p, t, 0.044410206377506256f);
  p = fmaf(p, t, 0.18637916445732117f);
  p = fmaf(p, t, 0.22879089415073395f);
  p = fmaf(p, t, 0.2535184919834137f);
  p = fmaf(p, t, 0.25391680002212524f);
  const float e = __expf(-0.5f * z * z), tail = 0.5f * t * p * e;
  *exp_out = e;
  return z < 0.f ? tail : 1.f - tail;
}

// act(z) of the one-input activations (SwiGLU takes two: SiLU(gate) * up).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == LRM_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays
  if (ACT == LRM_ACT_GELU) {
    float e;
    return z * norm_cdf(z, &e);
  }
  if (ACT == LRM_ACT_SILU || ACT == LRM_ACT_SWIGLU) return z * sigmoid_f(z);
  return z;
}
// act'(z); ReLU's derivative at 0 is 0.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == LRM_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (ACT == LRM_ACT_GELU) {
    float e;
    const float phi = norm_cdf(z, &e);
    return fmaf(0.39894228040143268f * z, e, phi);  // Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi)
  }
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
