// lrm_act_backward: dz = dy * act'(z) and the bias gradient db[e] = sum over the segment's rows of dz.
//
// One pass over dy and z (HBM bound: dy and z read, dz written once).  A CTA covers kRowBlock rows and
// 32 lanes of 16-byte columns; its 8 warps take the rows in turn and keep the column sums of the values
// before rounding in registers.
// The sums leave as partials part[b + e][column] of (row block b, expert e): along the rows either b or
// e grows at every step, so b + e names each meeting of a block and a segment once, and no prefix of
// block counts is needed.  A second launch adds an expert's partials in block order.  No atomics: db
// does not depend on scheduling.
#include "kernels.h"
#include "linear.cuh"

namespace lrm {

namespace {

constexpr int kRowBlock = 128;
constexpr int kWarps = 8;
// CTAs an SM holds: many warps with one row's loads each hide the memory better than few with several
// (65536 x 768 SwiGLU without sums, bf16: 84 us with 4 CTAs and 1 row, 97 us with 3 and 2, 101 us with 2 and
// 4; GELU of 65536 x 1536: 117 us with 5 CTAs, 123 us with 4, 124 us with 6).
template <typename T, int ACT>
constexpr int kCtas = sizeof(T) == 4 ? 6 : (ACT == LRM_ACT_SWIGLU ? 4 : 5);

template <typename T, int ACT>
__global__ void __launch_bounds__(32 * kWarps, (kCtas<T, ACT>)) act_backward_kernel(
    const int32_t* __restrict__ seg, int E, int64_t R, int N, const T* __restrict__ dy, const T* __restrict__ z,
    T* __restrict__ dz, float* __restrict__ part, int32_t* __restrict__ status) {
  chain_wait();
  constexpr int VN = VecTraits<T>::N;
  constexpr bool GLU = ACT == LRM_ACT_SWIGLU;
  constexpr int G = GLU ? 2 : 1;
  const int NP = G * N;
  __shared__ float s_sum[kWarps][32 * VN * G];
  __shared__ int s_seg[LRM_MAX_EXPERTS + 1];
  if (seg != nullptr) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) s_seg[e] = seg[e];
    __syncthreads();
    if (!rows_valid(s_seg, E, R, status)) return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x, b0 = b * kRowBlock;
  const int64_t end = seg == nullptr ? R : s_seg[E];
  const int64_t b1 = b0 + kRowBlock < end ? b0 + kRowBlock : end;
  const int slab = wide_y(), col = (slab * 32 + lane) * VN;
  const bool live = col < N;
  int e = 0;
  if (seg != nullptr && part != nullptr) {  // the expert of row b0: the last e with seg[e] <= b0
    int lo = 0, hi = E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_seg[mid] <= b0) lo = mid; else hi = mid;
    }
    e = lo;
  }
  // the rows of one expert in the block at a time (all of the block's when no sum is wanted)
  for (int64_t ra = b0; ra < b1; ++e) {
    const int64_t seg_end = seg != nullptr && part != nullptr ? s_seg[e + 1] : b1;
    const int64_t rb = seg_end < b1 ? seg_end : b1;
    if (rb <= ra) continue;  // an expert without rows
    float sum[G][VN];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int q = 0; q < VN; ++q) sum[g][q] = 0.f;
    for (int64_t r = ra + warp; r < rb && live; r += kWarps) {
      const uint4 d4 = ld_stream16_now(dy + r * N + col);
      uint4 z4[G];
      if (ACT != LRM_ACT_NONE)
#pragma unroll
        for (int g = 0; g < G; ++g) z4[g] = ld_stream16_now(z + r * NP + g * N + col);
      float d[VN], zf[G][VN], o[G][VN];
      unpack(d4, d);
      if (ACT != LRM_ACT_NONE)
#pragma unroll
        for (int g = 0; g < G; ++g) unpack(z4[g], zf[g]);
#pragma unroll
      for (int q = 0; q < VN; ++q) {
        if (GLU) {
          const float gate = zf[0][q], up = zf[G - 1][q], sg = sigmoid_f(gate);
          o[0][q] = d[q] * up * sg * (1.f + gate * (1.f - sg));
          o[G - 1][q] = d[q] * gate * sg;
        } else {
          o[0][q] = ACT == LRM_ACT_NONE ? d[q] : d[q] * act_slope<ACT>(zf[0][q]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) sum[g][q] += o[g][q];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) st16(dz + r * NP + g * N + col, pack(o[g]));
    }
    if (part != nullptr) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int q = 0; q < VN; ++q) s_sum[warp][(g * 32 + lane) * VN + q] = sum[g][q];
      __syncthreads();
      for (int i = threadIdx.x; i < 32 * VN * G; i += blockDim.x) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += s_sum[w][i];
        const int g = i / (32 * VN), c = slab * 32 * VN + i % (32 * VN);
        if (c < N && LRM_DCHECK(b + e < (int64_t)gridDim.x + E, status, LRM_ERR_BAD_INDEX))
          part[(b + e) * NP + g * N + c] = s;
      }
      __syncthreads();
    }
    ra = rb;
  }
}

// db[e][column] from the partials of the expert's row blocks: 128 columns per CTA (a lane has four), its
// warps taking the blocks in turn, added in a fixed order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) bias_sum_kernel(const int32_t* __restrict__ seg, int E, int64_t R,
                                                                  int NP, const float* __restrict__ part,
                                                                  float* __restrict__ db,
                                                                  int32_t* __restrict__ status) {
  chain_wait();
  extern __shared__ float s_part[];  // [warps][128]
  if (!rows_valid(seg, E, R, status)) return;
  const int e = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int col = blockIdx.x * 128 + lane * 4;  // NP is a multiple of 8
  const int64_t r0 = seg_at(seg, e, R), r1 = seg_at(seg, e + 1, R);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < NP && r1 > r0) {
    const int64_t last = (r1 - 1) / kRowBlock;
#pragma unroll 8
    for (int64_t b = r0 / kRowBlock + warp; b <= last; b += nw) {
      if (!LRM_DCHECK(b + e < (R + kRowBlock - 1) / kRowBlock + E, status, LRM_ERR_BAD_INDEX)) break;
      float f[4];
      unpack(ldg16(part + (b + e) * NP + col), f);
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += f[q];
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) s_part[warp * 128 + lane * 4 + q] = s[q];
  __syncthreads();
  if (warp == 0 && col < NP) {
    for (int w = 1; w < nw; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += s_part[w * 128 + lane * 4 + q];
    st16(db + (int64_t)e * NP + col, pack(s));
  }
}

template <typename T>
void act_backward_all(const ActGradArgs& a, cudaStream_t s) {
  constexpr int VN = VecTraits<T>::N;
  const int slabs = (a.N + 32 * VN - 1) / (32 * VN);
  if (a.R > 0)
    with_act(a.act, [&](auto tag) {
      launch_chained(act_backward_kernel<T, decltype(tag)::value>,
                     grid_wide((a.R + kRowBlock - 1) / kRowBlock, slabs), dim3(32 * kWarps), 0, s,
                     a.seg_offsets, a.E, a.R, a.N, (const T*)a.dy, (const T*)a.z, (T*)a.dz,
                     a.db != nullptr ? a.part : (float*)nullptr, a.status);
    });
  if (a.db != nullptr) {
    const int NP = a.act == LRM_ACT_SWIGLU ? 2 * a.N : a.N;
    // A warp for every four blocks of a mean segment, and where there are rows enough (16 blocks a warp) no fewer
    // than eight: a popular expert's blocks are many times the mean's, and its CTAs end last (65536 x 768 SwiGLU
    // over 128 experts, both launches: zipf 1 95.5 us, 103.7 us by the mean alone, 97.5 us with four warps, 96.1
    // us with 16; zipf 2 109, 139, 119, 104 us; even segments 92.0, 92.5, 91.9, 94.2 us).
    const int64_t blocks = (a.R + kRowBlock - 1) / kRowBlock, mean = (a.R / kRowBlock / a.E + 3) / 4 + 1;
    const int64_t least = (blocks + 15) / 16 < 8 ? (blocks + 15) / 16 : 8, want = mean > least ? mean : least;
    const unsigned warps = (unsigned)(want < kSumWarps ? want : kSumWarps);
    launch_chained(bias_sum_kernel, dim3((unsigned)((NP + 127) / 128), (unsigned)a.E), dim3(32 * warps),
                   warps * 128 * sizeof(float), s, a.seg_offsets, a.E, a.R, NP, (const float*)a.part, a.db, a.status);
  }
}

}  // namespace

size_t act_backward_part_rows(int64_t R, int32_t E) { return (size_t)((R + kRowBlock - 1) / kRowBlock + E); }

void launch_act_backward(const ActGradArgs& a, lrm_dtype dt, cudaStream_t s) {
  if (dt == LRM_BF16)
    act_backward_all<__nv_bfloat16>(a, s);
  else
    act_backward_all<float>(a, s);
}

}  // namespace lrm
