// lrm_fp8_linear for few rows (tokens being generated): bound by reading W, once for each 8 rows of an expert (dense:
// 16).
//
// The form of linear_rows.cu in 8 bits: a CTA takes 16 rows of W (SwiGLU: 8 gate rows and their 8 up rows) over the
// whole K, its 8 warps the blocks of 128 columns in turn, and their sums meet in shared memory in a fixed order.
// Lane (g, t) loads 16 bytes of W rows g and g + 8 and of x row g at the same K offset 16 t, which is two steps of
// mma.sync m16n8k32 with K in the order the lanes hold it.  A block's products are summed on their own, then scaled
// by the row's and the weight's scale and added up in fp32.
//
// Little is in flight a warp (one block), but where tasks fill the GPU three CTAs share a multiprocessor and hide one
// another's latencies: with four blocks and two CTAs a token's 8 rows over 8 of 128 experts of (768+768) x 2048 (768
// tasks, 1.7 waves) took 12.2 us, not 7.9 (25 MB of weights: 3.7 us at the copy rate), and 2048 x 768 13.9 us, not 6.3.
// A dense token has fewer tasks ((1408+1408) x 4096: 176, one CTA on most multiprocessors) and is bound by its warps'
// trips to memory one after the other.  GB300, dense, 1 to 8 rows: (1408+1408) x 4096 6.0 to 6.3 us, 4096 x 4096 6.6 to
// 6.8 us, (768+768) x 2048 2.7 us.
#include "fp8.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "rows_list.cuh"
#include "tc_host.h"

namespace lrm {

namespace {

using B16 = __nv_bfloat16;

__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sums of 16 W rows with 8 * NT rows of x over this warp's share of K, as sum[W row][x row] in `out`.  sw0, sw1: the
// scales of the first and the second 8 rows of W; sx: those of x, kb a row.
template <int NT>
__device__ __forceinline__ void warp_products(const uint8_t* w0, const uint8_t* w1, const uint8_t* x, const float* sw0,
                                              const float* sw1, const float* sx, int rows, int K, int kb, int warp,
                                              int lane, float (*out)[8 * NT + 1]) {
  constexpr int U = NT == 1 ? 1 : 2;  // blocks whose loads are in flight
  const int g = lane >> 2, t = lane & 3;
  float c[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) c[i][q] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int b0 = warp; b0 < kb; b0 += U * kWarps) {
    uint4 a[U][2], b[U][2], v[NT][U][2];
    float s0[U], s1[U], r[NT][U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (b0 + u * kWarps) * kQBlock + h * 64 + t * 16;
        a[u][h] = k < K ? ld_stream16_now(w0 + k) : zero;
        b[u][h] = k < K ? ld_stream16_now(w1 + k) : zero;
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = b0 + u * kWarps;
      s0[u] = at < kb ? __ldg(sw0 + at) : 0.f;
      s1[u] = at < kb ? __ldg(sw1 + at) : 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = at * kQBlock + h * 64 + t * 16;
          v[i][u][h] = k < K && i * 8 + g < rows ? ldg16_now(x + (int64_t)(i * 8 + g) * K + k) : zero;
          const int row = i * 8 + 2 * t + h;
          r[i][u][h] = at < kb && row < rows ? __ldg(sx + (int64_t)row * kb + at) : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_16x8(s, a[u][h].x, b[u][h].x, a[u][h].y, b[u][h].y, v[i][u][h].x, v[i][u][h].y);
          mma_16x8(s, a[u][h].z, b[u][h].z, a[u][h].w, b[u][h].w, v[i][u][h].z, v[i][u][h].w);
        }
        c[i][0] = fmaf(s0[u] * r[i][u][0], s[0], c[i][0]);
        c[i][1] = fmaf(s0[u] * r[i][u][1], s[1], c[i][1]);
        c[i][2] = fmaf(s1[u] * r[i][u][0], s[2], c[i][2]);
        c[i][3] = fmaf(s1[u] * r[i][u][1], s[3], c[i][3]);
      }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    out[g][i * 8 + 2 * t] = c[i][0];
    out[g][i * 8 + 2 * t + 1] = c[i][1];
    out[g + 8][i * 8 + 2 * t] = c[i][2];
    out[g + 8][i * 8 + 2 * t + 1] = c[i][3];
  }
}

// CTAs of a multiprocessor.
constexpr int ctas(int nt) { return nt == 1 ? 3 : 2; }

template <bool GLU, int NT>
__global__ void __launch_bounds__(32 * kWarps, ctas(NT)) fp8_rows_kernel(const __grid_constant__ Fp8Args p) {
  constexpr int CN = GLU ? 8 : 16;  // output columns
  constexpr int RT = 8 * NT;        // rows of x at a time
  __shared__ float s_sum[kWarps][16][RT + 1];
  __shared__ Rows s_list[LRM_MAX_EXPERTS];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
  const int N = p.N, K = p.K, NP = GLU ? 2 * N : N;
  const int blocks = (N + CN - 1) / CN, nb = (N + kQBlock - 1) / kQBlock, kb = (K + kQBlock - 1) / kQBlock;
  const uint8_t* w = static_cast<const uint8_t*>(p.w);
  const uint8_t* x = static_cast<const uint8_t*>(p.x);
  const B16 *bias = static_cast<const B16*>(p.bias), *residual = static_cast<const B16*>(p.residual);
  B16 *y = static_cast<B16*>(p.y), *z = static_cast<B16*>(p.z);
  const int experts = p.seg_offsets != nullptr ? list_experts(p.seg_offsets, p.E, p.R, s_list, p.status) : 1;
  // a task is one block of output columns of one expert
  for (int task = blockIdx.x; task < experts * blocks; task += gridDim.x) {
    const int i_e = task / blocks, n0 = (task - i_e * blocks) * CN;
    const Rows seg_e = p.seg_offsets != nullptr ? s_list[i_e] : Rows{0, 0, (int)p.R};
    const int e = seg_e.e, r_begin = seg_e.begin, r_end = seg_e.end;
    const uint8_t* we = w + (int64_t)e * NP * K;
    // rows g and g + 8 of this CTA's 16 (N is a multiple of 8: the second half may not exist; it repeats the first)
    const int second = GLU ? N + n0 : (n0 + 8 < N ? n0 + 8 : n0);
    const uint8_t* w0 = we + (int64_t)(n0 + g) * K;
    const uint8_t* w1 = we + (int64_t)(second + g) * K;
    const float* sw0 = p.w_scale + ((int64_t)e * (GLU ? 2 * nb : nb) + n0 / kQBlock) * kb;
    const float* sw1 = GLU ? sw0 + (int64_t)nb * kb : sw0;
    for (int r0 = r_begin; r0 < r_end; r0 += RT) {
      const int rows = min(RT, r_end - r0);
      warp_products<NT>(w0, w1, x + (int64_t)r0 * K, sw0, sw1, p.x_scale + (int64_t)r0 * kb, rows, K, kb, warp, lane,
                        s_sum[warp]);
      __syncthreads();
      for (int i = threadIdx.x; i < CN * RT; i += blockDim.x) {
        const int c = i % CN, r = i / CN, n = n0 + c;
        if (r >= rows || n >= N || !LRM_DCHECK(r0 >= 0 && r0 + r < p.R, p.status, LRM_ERR_BAD_INDEX)) continue;
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
          z[row * NP + n] = from_f<B16>(v);
          if (GLU) z[row * NP + N + n] = from_f<B16>(u);
        }
        if (GLU) {
          v = act_value<LRM_ACT_SWIGLU>(v) * u;
        } else {
          switch (p.act) {
            case LRM_ACT_RELU: v = act_value<LRM_ACT_RELU>(v); break;
            case LRM_ACT_GELU: v = act_value<LRM_ACT_GELU>(v); break;
            case LRM_ACT_SILU: v = act_value<LRM_ACT_SILU>(v); break;
            default: break;
          }
        }
        if (residual != nullptr) v += to_f(residual[at]);
        y[at] = from_f<B16>(v);
      }
      __syncthreads();
    }
  }
}

template <bool GLU, int NT>
void launch(const Fp8Args& a, cudaStream_t s) {
  constexpr int CN = GLU ? 8 : 16;
  const int64_t tasks = (a.R < a.E ? a.R : a.E) * ((a.N + CN - 1) / CN), room = ctas(NT) * (int64_t)sm_count();
  launch_chained(fp8_rows_kernel<GLU, NT>, dim3((unsigned)(tasks < room ? tasks : room)), dim3(32 * kWarps), 0, s, a);
}

}  // namespace

void launch_fp8_rows(const Fp8Args& a, cudaStream_t s) {
  const bool glu = a.act == LRM_ACT_SWIGLU;
  if (a.seg_offsets != nullptr || a.R <= 8)
    glu ? launch<true, 1>(a, s) : launch<false, 1>(a, s);
  else
    glu ? launch<true, 2>(a, s) : launch<false, 2>(a, s);
}

}  // namespace lrm
