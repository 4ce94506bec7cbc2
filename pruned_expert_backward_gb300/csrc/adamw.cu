// lrm_adamw and lrm_grad_norm: one optimiser step over many tensors at once.
//
//   g = gradient * min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by memory: every tensor is read once and written once.  The tensors' addresses travel in the kernel's
// parameters (no table on the device), a CTA takes chunks of 8192 elements in turn, a warp 256 of them at a time: lane
// l has elements 4 l .. 4 l + 3 and 128 more on, so that loads of every type are whole sectors in a row.
// GB300, 100M bf16 weights with fp32 gradients: 32-bit states 392 us (0.95 of the copy rate), 8-bit ones 251 us (0.74:
// neither the 474 instructions a block of 256, issued in 61 % of the cycles, nor DRAM, at 59 % of its peak, is full: the
// latency of a block's loads shows); 429M of them in 8 bits with the norm 1219 us.
//
// States in 8 bits: m and sqrt(v) in e4m3, the largest magnitude of each 256 elements of a tensor held as 448 with an
// fp32 scale, one block to a warp.  They are rounded up or down at random, with the odds that keep the mean: to nearest
// they would stand still (b2 = 0.999 moves sqrt(v) by 0.05 % a step at most where it shrinks, half a step of e4m3 is 3
// to 6 %), and a block that once had a large gradient would keep its neighbours' sqrt(v) in proportion.  The random
// bits are a hash of seed, step, tensor and element, so a step can be repeated.  The update itself uses the new m and v
// before they are rounded.  A sqrt(v) that is not 0 is never held as 0: m / eps would follow when the gradient stops.
#include "fp8.cuh"
#include "kernels.h"
#include "tc_host.h"

namespace lrm {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 256;                 // elements of a warp at a time, and of a state's scale
constexpr int kChunk = 8192;                // elements of a CTA's task
constexpr int kTable = 384;                 // tensors of a launch (32 KB of parameters, the most there can be)
constexpr int kAdamCtas = 4, kNormCtas = 8;  // of a multiprocessor
// Blocks of smaller states, all zeros among them, are scaled as if this were their largest.  448 over it has to be an
// fp32 value: over 2^-120 it is infinite, and 0 times that a NaN.
constexpr float kStateLeast = 0x1p-119f;

struct Table {
  lrm_adamw_tensor t[kTable];
  uint32_t first[kTable + 1];  // chunks before each tensor
  int count;
};

// The tensor of a chunk: the last i with first[i] <= c (tensors without elements have no chunk).
__device__ __forceinline__ int tensor_of(const Table& a, uint32_t c) {
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

// Four consecutive values; past the end (only in a tensor's last block) zeros.
template <bool TAIL>
__device__ __forceinline__ void load4(const float* p, int64_t i, int64_t n, float (&f)[4]) {
  if (!TAIL || i + 4 <= n) {
    float4 v;
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p + i));
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = i + j < n ? p[i + j] : 0.f;
  }
}
template <bool TAIL>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, int64_t i, int64_t n, float (&f)[4]) {
  if (!TAIL || i + 4 <= n) {
    uint32_t a, b;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "l"(p + i));
    f[0] = __uint_as_float(a << 16);
    f[1] = __uint_as_float(a & 0xffff0000u);
    f[2] = __uint_as_float(b << 16);
    f[3] = __uint_as_float(b & 0xffff0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = i + j < n ? __bfloat162float(p[i + j]) : 0.f;
  }
}
template <bool TAIL>
__device__ __forceinline__ uint32_t load4(const uint8_t* p, int64_t i, int64_t n) {
  uint32_t v = 0;
  if (!TAIL || i + 4 <= n) {
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p + i));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v |= i + j < n ? (uint32_t)p[i + j] << (8 * j) : 0u;
  }
  return v;
}
template <bool TAIL>
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, const float (&f)[4]) {
  if (!TAIL || i + 4 <= n) {
    *reinterpret_cast<float4*>(p + i) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = f[j];
  }
}
template <bool TAIL>
__device__ __forceinline__ void store4(__nv_bfloat16* p, int64_t i, int64_t n, const float (&f)[4]) {
  if (!TAIL || i + 4 <= n) {
    uint2 v;
    *reinterpret_cast<__nv_bfloat162*>(&v.x) = __floats2bfloat162_rn(f[0], f[1]);
    *reinterpret_cast<__nv_bfloat162*>(&v.y) = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(p + i) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = __float2bfloat16_rn(f[j]);
  }
}
template <bool TAIL>
__device__ __forceinline__ void store4(uint8_t* p, int64_t i, int64_t n, uint32_t v) {
  if (!TAIL || i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p + i) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(v >> (8 * j));
  }
}

// The larger magnitude, NaN above all.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// A unit in the last place off; roots of fp32 values and what is added to them stay clear of what it flushes.
__device__ __forceinline__ float recip(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The root, a unit in the last place off (32-bit states keep none).
__device__ __forceinline__ float sqrt_f(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The finaliser of MurmurHash3 (A. Appleby).  The multipliers of what goes into it, 0x9E3779B1 and 0xC2B2AE3D, are two
// of the 32-bit primes of xxHash (Y. Collet); 0x9E3779B9 is 2^32 over the golden ratio.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
  h = (h ^ (h >> 13)) * 0xC2B2AE35u;
  return h ^ (h >> 16);
}

// The finaliser's halves without its last exclusive or in full: m takes the low 16 bits, sqrt(v) the high ones.
__device__ __forceinline__ uint2 mix_halves(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
  h = (h ^ (h >> 13)) * 0xC2B2AE35u;
  const uint32_t high = h >> 16;
  return make_uint2((h ^ high) & 0xffffu, high);
}

// Random rounding of y (448 and a little in magnitude at most, of either sign) to an e4m3 value: 16 random bits are
// added below the 4-bit significand, what stays below it is cut.  Values below the normal ones have the smallest normal
// one's spacing: they are rounded with that one added.
__device__ __forceinline__ float raised(float y, uint32_t rnd16) {
  return __uint_as_float((__float_as_uint(y) + (rnd16 << 4)) & 0xfff00000u);
}

// The 8-bit states of a lane's two runs: y is m and sqrt(v) over their scales.
template <bool TAIL, bool SMALL>
__device__ __forceinline__ void store_states(const lrm_adamw_tensor& t, const int64_t (&i)[2], int64_t n,
                                             const float2 (&y)[2][4], uint32_t key) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float qm[4], qv[4];
    const uint32_t base = (uint32_t)i[s] * 0x9E3779B1u + (uint32_t)((uint64_t)i[s] >> 32) * 0xC2B2AE3Du + key;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint2 rnd = mix_halves(base + (uint32_t)j * 0x9E3779B1u);
      if (SMALL) {
        float2 z = make_float2(fabsf(y[s][j].x), y[s][j].y);
        const float2 shift = make_float2(z.x < 0x1p-6f ? 0x1p-6f : 0.f, z.y < 0x1p-6f ? 0x1p-6f : 0.f);
        z = __fadd2_rn(z, shift);
        z = make_float2(raised(z.x, rnd.x), raised(z.y, rnd.y));
        z = __fadd2_rn(z, make_float2(-shift.x, -shift.y));
        if (y[s][j].y > 0.f) z.y = fmaxf(z.y, 0x1p-9f);
        qm[j] = copysignf(z.x, y[s][j].x);
        qv[j] = z.y;
      } else {
        qm[j] = raised(y[s][j].x, rnd.x);
        qv[j] = raised(y[s][j].y, rnd.y);
      }
    }
    store4<TAIL>(static_cast<uint8_t*>(t.m), i[s], n, e4m3x4(qm[0], qm[1], qm[2], qm[3]));
    store4<TAIL>(static_cast<uint8_t*>(t.v), i[s], n, e4m3x4(qv[0], qv[1], qv[2], qv[3]));
  }
}

struct Hyper {
  float lr, b1, b2, one_b1, one_b2, eps, one;
  float c1, c2;  // 1 - b^t, where the step is the host's
  double log_b1, log_b2;
  float max_norm;
  uint32_t seed, step;
  const float *lr_dev, *norm;
  const int32_t* step_dev;
};

// One block of 256 elements from i0 of a tensor.
template <typename W, typename G, bool BITS8, bool COPY, bool TAIL>
__device__ __forceinline__ void update_block(const lrm_adamw_tensor& t, int64_t i0, int lane, const Hyper& h,
                                             float factor, float decay, float rate, float inv_c2, uint32_t key) {
  const int64_t n = t.n, i[2] = {i0 + 4 * lane, i0 + 128 + 4 * lane};
  float g[2][4], w[2][4], m[2][4], v[2][4];
  uint32_t mq[2], vq[2];
  float ms = 0.f, vs = 0.f;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    load4<TAIL>(static_cast<const G*>(t.g), i[s], n, g[s]);
    load4<TAIL>(static_cast<const W*>(t.w), i[s], n, w[s]);
    if (BITS8) {
      mq[s] = load4<TAIL>(static_cast<const uint8_t*>(t.m), i[s], n);
      vq[s] = load4<TAIL>(static_cast<const uint8_t*>(t.v), i[s], n);
    } else {
      load4<TAIL>(static_cast<const float*>(t.m), i[s], n, m[s]);
      load4<TAIL>(static_cast<const float*>(t.v), i[s], n, v[s]);
    }
  }
  if (BITS8) {
    ms = t.m_scale[i0 / kBlock];
    vs = t.v_scale[i0 / kBlock];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      from_e4m3x4(mq[s], m[s]);
      from_e4m3x4(vq[s], v[s]);
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const float2 mm = __fmul2_rn(make_float2(m[s][j], m[s][j + 1]), make_float2(ms, ms));
        const float2 rr = __fmul2_rn(make_float2(v[s][j], v[s][j + 1]), make_float2(vs, vs));
        const float2 vv = __fmul2_rn(rr, rr);
        m[s][j] = mm.x;
        m[s][j + 1] = mm.y;
        v[s][j] = vv.x;
        v[s][j + 1] = vv.y;
      }
    }
  }
  float top_m = 0.f, top_v = 0.f;
  const float2 f2 = make_float2(factor, factor), b1 = make_float2(h.b1, h.b1), b2 = make_float2(h.b2, h.b2),
               c1 = make_float2(h.one_b1, h.one_b1), c2 = make_float2(h.one_b2, h.one_b2),
               one = make_float2(h.one, h.one);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 4; j += 2) {  // two at a time: half the instructions
      // Each step is rounded by itself, so that a host program's fp32 repeats the 8-bit states to the bit.  (The sum is
      // x * 1 + y with a 1 that the compiler does not know: it would make a product and a plain sum one multiply-add.)
      const float2 gf = __fmul2_rn(make_float2(g[s][j], g[s][j + 1]), f2);
      float2 mm = make_float2(m[s][j], m[s][j + 1]), vv = make_float2(v[s][j], v[s][j + 1]);
      mm = __ffma2_rn(__fmul2_rn(mm, b1), one, __fmul2_rn(gf, c1));
      vv = __ffma2_rn(__fmul2_rn(vv, b2), one, __fmul2_rn(__fmul2_rn(gf, gf), c2));
      m[s][j] = mm.x;
      m[s][j + 1] = mm.y;
      v[s][j] = vv.x;
      v[s][j + 1] = vv.y;
      if (BITS8) {
        top_m = max_abs(max_abs(top_m, mm.x), mm.y);
        top_v = max_abs(max_abs(top_v, vv.x), vv.y);
      }
    }
  float tm = 0.f, tv = 0.f, rv = 0.f;  // of the block: largest m, v and sqrt(v)
  if (BITS8) {  // (as bits a NaN is above every value)
    tm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_m)));
    tv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_v)));
    rv = __fsqrt_rn(tv);
  }
  float r[2][4];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[s][j] = BITS8 ? __fsqrt_rn(v[s][j]) : sqrt_f(v[s][j]);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float2 den = __ffma2_rn(make_float2(r[s][j], r[s][j + 1]), make_float2(inv_c2, inv_c2),
                                    make_float2(h.eps, h.eps));
      const float2 up = __fmul2_rn(make_float2(m[s][j], m[s][j + 1]), make_float2(recip(den.x), recip(den.y)));
      const float2 ww = __ffma2_rn(up, make_float2(-rate, -rate),
                                   __fmul2_rn(make_float2(w[s][j], w[s][j + 1]), make_float2(decay, decay)));
      w[s][j] = ww.x;
      w[s][j + 1] = ww.y;
    }
    store4<TAIL>(static_cast<W*>(t.w), i[s], n, w[s]);
    if (COPY) store4<TAIL>(static_cast<__nv_bfloat16*>(t.copy), i[s], n, w[s]);
    if (!BITS8) {
      store4<TAIL>(static_cast<float*>(t.m), i[s], n, m[s]);
      store4<TAIL>(static_cast<float*>(t.v), i[s], n, v[s]);
    }
  }
  if (BITS8) {
    if (tm < kStateLeast) tm = kStateLeast;  // (a NaN stays)
    if (rv < kStateLeast) rv = kStateLeast;
    if (lane == 0) {
      t.m_scale[i0 / kBlock] = tm * (1.f / kQTop);
      t.v_scale[i0 / kBlock] = rv * (1.f / kQTop);
    }
    const float im = kQTop * __frcp_rn(tm), iv = kQTop * __frcp_rn(rv);
    float2 y[2][4];  // m and sqrt(v) side by side
    float least = kQTop;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[s][j] = __fmul2_rn(make_float2(m[s][j], r[s][j]), make_float2(im, iv));
        least = fminf(fminf(fabsf(y[s][j].x), y[s][j].y), least);
      }
    // most blocks have no value below e4m3's normal ones
    if (__all_sync(0xffffffffu, least >= 0x1p-6f))
      store_states<TAIL, false>(t, i, n, y, key);
    else
      store_states<TAIL, true>(t, i, n, y, key);
  }
}

// Asks L2 for the lines of a block with 8-bit states, a line to a lane.
template <typename W, typename G>
__device__ __forceinline__ void ahead(const lrm_adamw_tensor& t, int64_t i, int lane) {
  constexpr int kG = kBlock * sizeof(G) / 128, kW = kBlock * sizeof(W) / 128, kS = kBlock / 128;
  const char* p = nullptr;
  if (lane < kG)
    p = static_cast<const char*>(t.g) + i * (int64_t)sizeof(G) + lane * 128;
  else if (lane < kG + kW)
    p = static_cast<const char*>(t.w) + i * (int64_t)sizeof(W) + (lane - kG) * 128;
  else if (lane < kG + kW + kS)
    p = static_cast<const char*>(t.m) + i + (lane - kG - kW) * 128;
  else if (lane < kG + kW + 2 * kS)
    p = static_cast<const char*>(t.v) + i + (lane - kG - kW - kS) * 128;
  if (p != nullptr) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

template <typename W, typename G, bool BITS8, bool COPY>
__global__ void __launch_bounds__(kThreads, kAdamCtas) adamw_kernel(const __grid_constant__ Table a, const Hyper h) {
  chain_wait();
  __shared__ float s_lr, s_c1, s_c2, s_factor;
  __shared__ uint32_t s_step;
  if (threadIdx.x == 0) {
    s_lr = h.lr_dev != nullptr ? *h.lr_dev : h.lr;
    s_step = h.step_dev != nullptr ? (uint32_t)max(*h.step_dev, 1) : h.step;
    s_c1 = h.c1;
    s_c2 = h.c2;
    if (h.step_dev != nullptr) {
      const double t = (double)s_step;
      s_c1 = (float)-expm1(t * h.log_b1);
      s_c2 = (float)-expm1(t * h.log_b2);
    }
    float f = 1.f;
    if (h.norm != nullptr) {
      const float norm = *h.norm;
      f = isfinite(norm) ? fminf(1.f, h.max_norm * __frcp_rn(norm + 1e-6f)) : -1.f;
    }
    s_factor = f;
  }
  __syncthreads();
  const float factor = s_factor;
  if (factor < 0.f) return;  // a norm that is not finite: nothing is touched (recorded by lrm_grad_norm)
  const float inv_c2 = __frsqrt_rn(s_c2), lr_c1 = __fdiv_rn(s_lr, s_c1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t chunks = a.first[a.count];
  int ti = -1;
  uint32_t t_first = 0, t_end = 0, key = 0;
  float decay = 0.f, rate = 0.f;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    if (c >= t_end) {  // (always at first)
      ti = tensor_of(a, c);
      t_first = a.first[ti];
      t_end = a.first[ti + 1];
      decay = 1.f - s_lr * a.t[ti].lr_scale * a.t[ti].weight_decay;
      rate = lr_c1 * a.t[ti].lr_scale;
      key = mix32(mix32(h.seed + 0x9E3779B9u * (uint32_t)(a.t[ti].id + 1)) ^ s_step);
    }
    const lrm_adamw_tensor& t = a.t[ti];
    const int64_t begin = (int64_t)(c - t_first) * kChunk, end = min(t.n, begin + kChunk);
    constexpr int64_t kNext = (kThreads / 32) * kBlock;
    for (int64_t i = begin + warp * kBlock; i < end; i += kNext) {
      // 8-bit states: the warp's next block of the chunk is fetched under this one's arithmetic (100M fp32 weights 265
      // us, 301 without; bf16 ones 251 and 270; across chunks, or a fifth CTA instead, less; 32-bit states gain nothing)
      if (BITS8 && i + kNext + kBlock <= end) ahead<W, G>(t, i + kNext, lane);
      if (i + kBlock <= t.n)
        update_block<W, G, BITS8, COPY, false>(t, i, lane, h, factor, decay, rate, inv_c2, key);
      else
        update_block<W, G, BITS8, COPY, true>(t, i, lane, h, factor, decay, rate, inv_c2, key);
    }
  }
}

// Sums of squares: each CTA's of its chunks, in fp64 beyond 32 values, to part[blockIdx].
template <typename G>
__global__ void __launch_bounds__(kThreads)
    norm_parts_kernel(const __grid_constant__ Table a, double* __restrict__ part) {
  chain_wait();
  __shared__ double s_sum[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t chunks = a.first[a.count];
  double sum = 0.;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const lrm_adamw_tensor& t = a.t[tensor_of(a, c)];
    const int64_t begin = (int64_t)(c - a.first[&t - a.t]) * kChunk;
    float s = 0.f;
    if (begin + kChunk <= t.n) {
      float f[kChunk / kThreads / 4][4];
#pragma unroll
      for (int k = 0; k < kChunk / kThreads / 4; ++k)
        load4<false>(static_cast<const G*>(t.g), begin + (k * kThreads + threadIdx.x) * 4, t.n, f[k]);
#pragma unroll
      for (int k = 0; k < kChunk / kThreads / 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(f[k][j], f[k][j], s);
    } else {
      for (int64_t i = begin + threadIdx.x * 4; i < t.n; i += kThreads * 4) {
        float f[4];
        load4<true>(static_cast<const G*>(t.g), i, t.n, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fmaf(f[j], f[j], s);
      }
    }
    sum += (double)s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += s_sum[w];
    part[blockIdx.x] = sum;
  }
}

__global__ void __launch_bounds__(1024) norm_kernel(const double* __restrict__ part, int n, float* __restrict__ norm,
                                                    int32_t* __restrict__ status) {
  chain_wait();
  __shared__ double s_sum[32];
  double sum = 0.;
  for (int i = threadIdx.x; i < n; i += blockDim.x) sum += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) sum += s_sum[w];
    const float r = (float)sqrt(sum);
    *norm = r;
    if (!isfinite(r)) set_status(status, LRM_ERR_NONFINITE);
  }
}

// Calls f with tables of at most kTable of the tensors that have elements, and their chunks.
template <typename F>
void for_tables(const lrm_adamw_tensor* tensors, int32_t count, F&& f) {
  Table a;
  a.count = 0;
  a.first[0] = 0;
  auto flush = [&] {
    if (a.count > 0) f(a, a.first[a.count]);
    a.count = 0;
  };
  for (int32_t i = 0; i < count; ++i) {
    if (tensors[i].n == 0) continue;
    const int64_t chunks = (tensors[i].n + kChunk - 1) / kChunk;
    if (a.count == kTable || (a.count > 0 && a.first[a.count] + chunks > INT32_MAX)) flush();
    a.t[a.count] = tensors[i];
    a.first[a.count + 1] = a.first[a.count] + (uint32_t)chunks;
    ++a.count;
  }
  flush();
}

unsigned ctas(uint32_t chunks, int per_sm) {
  const uint32_t room = (uint32_t)(per_sm * sm_count());
  return chunks < room ? chunks : room;
}

}  // namespace

// Partial sums that lrm_grad_norm may write: full launches' worth for each table.
size_t grad_norm_parts(const lrm_adamw_tensor* tensors, int32_t count) {
  size_t n = 0;
  for_tables(tensors, count, [&](const Table&, uint32_t chunks) { n += chunks < 2048 ? chunks : 2048; });
  return n > 0 ? n : 1;
}

void launch_grad_norm(const lrm_adamw_tensor* tensors, int32_t count, lrm_dtype g_dt, float* norm, double* part,
                      int32_t* status, cudaStream_t s) {
  int n = 0;
  for_tables(tensors, count, [&](const Table& a, uint32_t chunks) {
    unsigned grid = ctas(chunks, kNormCtas);
    if (grid > 2048) grid = 2048;
    launch_chained(g_dt == LRM_BF16 ? norm_parts_kernel<__nv_bfloat16> : norm_parts_kernel<float>, dim3(grid),
                   dim3(kThreads), 0, s, a, part + n);
    n += (int)grid;
  });
  launch_chained(norm_kernel, dim3(1), dim3(1024), 0, s, (const double*)part, n, norm, status);
}

void launch_adamw(const lrm_adamw_tensor* tensors, int32_t count, lrm_dtype w_dt, lrm_dtype g_dt, int32_t state_bits,
                  bool copy, const lrm_adamw_hyper& p, cudaStream_t s) {
  Hyper h{};
  h.lr = (float)p.lr;
  h.b1 = (float)p.beta1;
  h.b2 = (float)p.beta2;
  h.one_b1 = (float)(1. - p.beta1);
  h.one_b2 = (float)(1. - p.beta2);
  h.eps = (float)p.eps;
  h.one = 1.f;
  h.log_b1 = log(p.beta1);
  h.log_b2 = log(p.beta2);
  h.c1 = (float)-expm1((double)p.step * h.log_b1);
  h.c2 = (float)-expm1((double)p.step * h.log_b2);
  h.max_norm = (float)p.max_norm;
  h.seed = p.seed;
  h.step = (uint32_t)p.step;
  h.lr_dev = p.lr_dev;
  h.step_dev = p.step_dev;
  h.norm = p.grad_norm;
  for_tables(tensors, count, [&](const Table& a, uint32_t chunks) {
    const dim3 grid(ctas(chunks, kAdamCtas));
    auto go = [&](auto kernel) { launch_chained(kernel, grid, dim3(kThreads), 0, s, a, h); };
    auto typed = [&](auto* w, auto* g) {
      using W = std::remove_pointer_t<decltype(w)>;
      using G = std::remove_pointer_t<decltype(g)>;
      if constexpr (sizeof(W) == 4) {
        if (copy) return state_bits == 8 ? go(adamw_kernel<W, G, true, true>) : go(adamw_kernel<W, G, false, true>);
      }
      state_bits == 8 ? go(adamw_kernel<W, G, true, false>) : go(adamw_kernel<W, G, false, false>);
    };
    float* f = nullptr;
    __nv_bfloat16* b = nullptr;
    if (w_dt == LRM_BF16)
      g_dt == LRM_BF16 ? typed(b, b) : typed(b, f);
    else
      g_dt == LRM_BF16 ? typed(f, b) : typed(f, f);
  });
}

}  // namespace lrm
