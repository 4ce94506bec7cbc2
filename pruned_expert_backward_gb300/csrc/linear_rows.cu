// lrm_linear for few rows (tokens being generated): bound by reading W once.
//
// A CTA takes 16 rows of W (16 output columns; SwiGLU: 8 gate rows and their 8 up rows) over the whole
// K; its 8 warps split K in steps of 32 and their sums meet in shared memory in a fixed order.  Lane
// (g, t) of a warp loads 16 bytes of W rows g and g + 8 and of x row g at the same K offset 8 t, so that
// no operand is staged or shuffled: within a 32-deep step the products run over K in the order the
// lanes hold it, which both operands share.
//   bf16: mma.sync m16n8k16, W as the 16 x 16 operand and 8 rows of x as the 16 x 8 one.  The tensor
//         core idles: at 8 rows a step moves 1 KB of W for 16 KFLOP.  (tcgen05 tiles of 256 rows of x
//         leave the same bytes to few CTAs with less in flight.)
//   fp32: fused multiply-adds, 8 rows of x at a time.
// Each lane has 16 loads of 16 bytes in flight (with half of them, and the compiler free to sink them to
// their use, 4 rows x (1408+1408) x 4096 took 12.9 us, not 6.7).  x is read by every CTA through L2, R / 16
// of W's bytes, which bounds the rows this form is used for.
// With segments a CTA first lists the experts that have rows (at most R), then takes their column blocks in
// turn, two CTAs per SM: one CTA for every block of every expert spent 29 us on a token's 8 rows over 8 of 128
// experts of (768+768) x 2048, mostly starting CTAs with nothing to do, where this takes 13 us (50 MB of weights: 7.4
// us at the copy rate).
// GB300, bf16 8 rows: 4096 x 4096 8.4 us, (768+768) x 2048 3.8 us; fp32 8 rows x 4096 x 4096 23 us, 24 rows 57 us.
#include "kernels.h"
#include "linear.cuh"
#include "tc_host.h"

namespace lrm {

namespace {

constexpr int kWarps = 8;
constexpr int kStep = 32;  // K of a warp's step

__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sums of 16 W rows with 8 * NT rows of x over this warp's share of K, as sum[W row][x row] in `out`.
template <int NT>
__device__ __forceinline__ void warp_products(const __nv_bfloat16* w0, const __nv_bfloat16* w1,
                                              const __nv_bfloat16* x, int rows, int K, int warp, int lane,
                                              float (*out)[8 * NT + 1]) {
  constexpr int U = NT == 1 ? 8 : 4;  // steps whose loads are in flight
  const int g = lane >> 2, t = lane & 3;
  float c[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) c[i][q] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * kStep + t * 8; k0 - t * 8 < K; k0 += U * kWarps * kStep) {
    uint4 a[U], b[U], v[NT][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kWarps * kStep;
      a[u] = k < K ? ld_stream16_now(w0 + k) : zero;
      b[u] = k < K ? ld_stream16_now(w1 + k) : zero;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * kWarps * kStep;
        v[i][u] = k < K && i * 8 + g < rows ? ldg16_now(x + (int64_t)(i * 8 + g) * K + k) : zero;
      }
    // This round's products apart: the tensor core truncates as it adds, the sum of the rounds is to nearest (65536
    // products of one sign were 2.9e-5 off in one accumulator, and take as long; 4096 x 4096 with 16 rows 9.0 us, 8.6
    // us in one).
    float s[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[i][q] = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        mma_16x8(s[i], a[u].x, b[u].x, a[u].y, b[u].y, v[i][u].x, v[i][u].y);
        mma_16x8(s[i], a[u].z, b[u].z, a[u].w, b[u].w, v[i][u].z, v[i][u].w);
      }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) c[i][q] += s[i][q];
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    out[g][i * 8 + 2 * t] = c[i][0];
    out[g][i * 8 + 2 * t + 1] = c[i][1];
    out[g + 8][i * 8 + 2 * t] = c[i][2];
    out[g + 8][i * 8 + 2 * t + 1] = c[i][3];
  }
}

template <int NT>
__device__ __forceinline__ void warp_products(const float* w0, const float* w1, const float* x, int rows, int K,
                                              int warp, int lane, float (*out)[8 * NT + 1]) {
  static_assert(NT == 1, "fp32 takes 8 rows at a time");
  constexpr int U = 2, XR = 4;  // steps of W, and rows of x, whose loads are in flight
  const int g = lane >> 2, t = lane & 3;
  float c[2][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) c[0][r] = c[1][r] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * kStep + t * 8; k0 - t * 8 < K; k0 += U * kWarps * kStep) {
    uint4 a[U][2], b[U][2];  // 8 values of each row
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kWarps * kStep;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[u][h] = k < K ? ld_stream16_now(w0 + k + 4 * h) : zero;
        b[u][h] = k < K ? ld_stream16_now(w1 + k + 4 * h) : zero;
      }
    }
#pragma unroll
    for (int r0 = 0; r0 < 8; r0 += XR) {
      if (r0 >= rows) break;
      uint4 v[XR][U][2];
#pragma unroll
      for (int r = 0; r < XR; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + u * kWarps * kStep;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[r][u][h] = k < K && r0 + r < rows ? ldg16_now(x + (int64_t)(r0 + r) * K + k + 4 * h) : zero;
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float fa[4], fb[4];
          unpack(a[u][h], fa);
          unpack(b[u][h], fb);
#pragma unroll
          for (int r = 0; r < XR; ++r) {
            float f[4];
            unpack(v[r][u][h], f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              c[0][r0 + r] = fmaf(fa[q], f[q], c[0][r0 + r]);
              c[1][r0 + r] = fmaf(fb[q], f[q], c[1][r0 + r]);
            }
          }
        }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      c[h][r] += __shfl_xor_sync(0xffffffffu, c[h][r], 1);
      c[h][r] += __shfl_xor_sync(0xffffffffu, c[h][r], 2);
      if (t == 0) out[g + 8 * h][r] = c[h][r];
    }
}

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

template <typename TI, typename TO, bool GLU, int NT>
__global__ void __launch_bounds__(32 * kWarps, 2) rows_kernel(const int32_t* __restrict__ seg, int E, int64_t R,
                                                           const TI* __restrict__ x, const TI* __restrict__ w,
                                                           const TI* __restrict__ bias, const TO* __restrict__ residual,
                                                           int N, int K, int act, TO* __restrict__ y,
                                                           TI* __restrict__ z, int32_t* __restrict__ status) {
  constexpr int CN = GLU ? 8 : 16;  // output columns
  constexpr int RT = 8 * NT;        // rows of x at a time
  __shared__ float s_sum[kWarps][16][RT + 1];
  __shared__ Rows s_list[LRM_MAX_EXPERTS];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
  const int blocks = (N + CN - 1) / CN, NP = GLU ? 2 * N : N;
  const int experts = seg != nullptr ? list_experts(seg, E, R, s_list, status) : 1;
  // a task is one block of output columns of one expert
  for (int task = blockIdx.x; task < experts * blocks; task += gridDim.x) {
    const int i_e = task / blocks, n0 = (task - i_e * blocks) * CN;
    const Rows seg_e = seg != nullptr ? s_list[i_e] : Rows{0, 0, (int)R};
    const int e = seg_e.e, r_begin = seg_e.begin, r_end = seg_e.end;
    const TI* we = w + (int64_t)e * NP * K;
    // rows g and g + 8 of this CTA's 16 (N is a multiple of 8: the second half may not exist; it repeats the first)
    const int second = GLU ? N + n0 : (n0 + 8 < N ? n0 + 8 : n0);
    const TI* w0 = we + (int64_t)(n0 + g) * K;
    const TI* w1 = we + (int64_t)(second + g) * K;
    for (int r0 = r_begin; r0 < r_end; r0 += RT) {
      const int rows = min(RT, r_end - r0);
      warp_products<NT>(w0, w1, x + (int64_t)r0 * K, rows, K, warp, lane, s_sum[warp]);
      __syncthreads();
      for (int i = threadIdx.x; i < CN * RT; i += blockDim.x) {
        const int c = i % CN, r = i / CN, n = n0 + c;
        if (r >= rows || n >= N || !LRM_DCHECK(r0 >= 0 && r0 + r < R, status, LRM_ERR_BAD_INDEX)) continue;
        float v = 0.f, u = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
          v += s_sum[q][c][r];
          if (GLU) u += s_sum[q][c + 8][r];
        }
        const int64_t row = r0 + r, at = row * N + n;
        if (bias != nullptr) {
          v += to_f(bias[(int64_t)e * NP + n]);
          if (GLU) u += to_f(bias[(int64_t)e * NP + N + n]);
        }
        if (z != nullptr) {
          z[row * NP + n] = from_f<TI>(v);
          if (GLU) z[row * NP + N + n] = from_f<TI>(u);
        }
        if (GLU) {
          v = act_value<LRM_ACT_SWIGLU>(v) * u;
        } else {
          switch (act) {
            case LRM_ACT_RELU: v = act_value<LRM_ACT_RELU>(v); break;
            case LRM_ACT_GELU: v = act_value<LRM_ACT_GELU>(v); break;
            case LRM_ACT_SILU: v = act_value<LRM_ACT_SILU>(v); break;
            default: break;
          }
        }
        if (residual != nullptr) v += to_f(residual[at]);
        y[at] = from_f<TO>(v);
      }
      __syncthreads();
    }
  }
}

template <typename TI, typename TO, bool GLU, int NT>
void launch(const LinearArgs& a, cudaStream_t s) {
  constexpr int CN = GLU ? 8 : 16;
  const int64_t tasks = (a.R < a.E ? a.R : a.E) * ((a.N + CN - 1) / CN), room = 2 * (int64_t)sm_count();
  launch_chained(rows_kernel<TI, TO, GLU, NT>, dim3((unsigned)(tasks < room ? tasks : room)), dim3(32 * kWarps), 0, s,
                 a.seg_offsets, a.E, a.R, (const TI*)a.x, (const TI*)a.w, (const TI*)a.bias, (const TO*)a.residual, a.N,
                 a.K, (int)a.act, (TO*)a.y, (TI*)a.z, a.status);
}

template <typename TO, bool GLU>
void launch_bf16(const LinearArgs& a, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (a.seg_offsets != nullptr || a.R <= 8)
    launch<B, TO, GLU, 1>(a, s);
  else if (a.R <= 16)
    launch<B, TO, GLU, 2>(a, s);
  else
    launch<B, TO, GLU, 4>(a, s);
}

}  // namespace

void launch_linear_rows(const LinearArgs& a, lrm_dtype dt, lrm_dtype out_dt, cudaStream_t s) {
  const bool glu = a.act == LRM_ACT_SWIGLU;
  if (dt == LRM_F32)
    glu ? launch<float, float, true, 1>(a, s) : launch<float, float, false, 1>(a, s);
  else if (out_dt == LRM_F32)
    glu ? launch_bf16<float, true>(a, s) : launch_bf16<float, false>(a, s);
  else
    glu ? launch_bf16<__nv_bfloat16, true>(a, s) : launch_bf16<__nv_bfloat16, false>(a, s);
}

}  // namespace lrm
