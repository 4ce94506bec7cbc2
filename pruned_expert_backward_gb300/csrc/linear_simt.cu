// lrm_linear and lrm_linear_backward on the CUDA cores (fp32 products and sums), on request
// (LRM_GEMM_FORCE_SIMT): the plain form the tensor-core kernels are checked beside.
//
//   forward   z = x W[e]^T + b[e], y = act(z) + residual
//   gradient  dx = dz W[e];  dW[e] = dz^T x over the segment's rows
// 64 x 64 output tiles, 16-deep K slices in shared memory, 256 threads with 4 x 4 outputs each.
// A SwiGLU tile holds 32 gate columns and their 32 up columns; a thread owns two of each.
#include "kernels.h"
#include "linear.cuh"

namespace lrm {

namespace {

constexpr int BM = 64, BN = 64, BK = 16, NT = 256;

// Virtual row tile vt -> (expert, first row, end row); prefix is built by the whole block.
__device__ bool find_rows(const int32_t* seg, int E, int64_t R, int64_t vt, int* s_prefix, int* e_out, int* r0_out,
                          int* r1_out) {
  if (seg == nullptr) {
    *e_out = 0;
    *r0_out = (int)(vt * BM);
    *r1_out = (int)min(R, (vt + 1) * BM);
    return vt * BM < R;
  }
  if (threadIdx.x == 0) {
    int acc = 0;
    for (int e = 0; e < E; ++e) {
      s_prefix[e] = acc;
      acc += (seg[e + 1] - seg[e] + BM - 1) / BM;
    }
    s_prefix[E] = acc;
  }
  __syncthreads();
  if (vt >= s_prefix[E]) return false;
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_prefix[mid] <= vt) lo = mid; else hi = mid;
  }
  *e_out = lo;
  *r0_out = seg[lo] + (int)(vt - s_prefix[lo]) * BM;
  *r1_out = min(seg[lo + 1], *r0_out + BM);
  return true;
}

enum { FWD = 0, DX = 1 };

// FWD: C[r, n] = sum_k A[r, k] B_e[n, k] (B_e [NP, K]) with the epilogue; DX: C[r, n] = sum_k A[r, k] B_e[k, n].
// N: output columns (FWD: of y, B_e then has 2N rows for SwiGLU); K: the reduction.
template <typename T, typename TO, int MODE, int ACT>
__global__ void __launch_bounds__(NT) rows_kernel(const int32_t* __restrict__ seg, int E, int64_t R,
                                                  const T* __restrict__ A, const T* __restrict__ B, int N, int K,
                                                  const T* __restrict__ bias, const TO* __restrict__ residual,
                                                  TO* __restrict__ out, T* __restrict__ z,
                                                  int32_t* __restrict__ status) {
  constexpr bool GLU = MODE == FWD && ACT == LRM_ACT_SWIGLU;
  constexpr int CN = GLU ? BN / 2 : BN;  // output columns of a tile
  __shared__ int s_prefix[LRM_MAX_EXPERTS + 1];
  __shared__ float As[BK][BM + 4];
  __shared__ float Bs[BK][BN + 4];
  chain_wait();
  if (!rows_valid(seg, E, R, status)) return;
  int e, r0, r1;
  if (!find_rows(seg, E, R, blockIdx.x, s_prefix, &e, &r0, &r1)) return;
  const int NP = GLU ? 2 * N : N;
  const int n0 = wide_y() * CN;
  const T* Be = B + (int64_t)e * NP * K;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  // product column held at tile column c, and whether its output column exists
  auto col_of = [&](int c) { return GLU ? ((c & 2) ? N : 0) + n0 + (c >> 2) * 2 + (c & 1) : n0 + c; };
  auto col_in = [&](int c) { return GLU ? n0 + (c >> 2) * 2 + (c & 1) < N : n0 + c < N; };
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += BK) {
    {
      const int m = threadIdx.x / 4, kq = (threadIdx.x % 4) * 4, r = r0 + m;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        As[kq + q][m] = (r < r1 && k0 + kq + q < K) ? to_f(A[(int64_t)r * K + k0 + kq + q]) : 0.f;
    }
    if (MODE == FWD) {  // a thread takes 4 consecutive k of one row of B_e
      const int c = threadIdx.x / 4, kq = (threadIdx.x % 4) * 4;
      const bool in = col_in(c);
      const int64_t row = (int64_t)col_of(c) * K;
#pragma unroll
      for (int q = 0; q < 4; ++q) Bs[kq + q][c] = (in && k0 + kq + q < K) ? to_f(Be[row + k0 + kq + q]) : 0.f;
    } else {
      const int kk = threadIdx.x / 16, nq = (threadIdx.x % 16) * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        Bs[kk][nq + q] = (k0 + kk < K && n0 + nq + q < N) ? to_f(Be[(int64_t)(k0 + kk) * N + n0 + nq + q]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = As[kk][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = Bs[kk][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + ty * 4 + i;
    if (r >= r1 || !LRM_DCHECK(r >= 0 && r < R, status, LRM_ERR_BAD_INDEX)) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = tx * 4 + j;
      if (!col_in(c)) continue;
      const int col = col_of(c);
      if (MODE == DX) {
        out[r * N + col] = from_f<TO>(acc[i][j]);
        continue;
      }
      const float b = bias != nullptr ? to_f(bias[(int64_t)e * NP + col]) : 0.f;
      acc[i][j] += b;
      if (z != nullptr) z[r * NP + col] = from_f<T>(acc[i][j]);
    }
    if (MODE == DX) continue;
#pragma unroll
    for (int j = 0; j < (GLU ? 2 : 4); ++j) {
      const int c = tx * 4 + j;
      if (!col_in(c)) continue;
      const int64_t at = r * N + col_of(c);
      float v = act_value<ACT>(acc[i][j]);
      if (GLU) v *= acc[i][j + 2];
      if (residual != nullptr) v += to_f(residual[at]);
      out[at] = from_f<TO>(v);
    }
  }
}

// dW[e][m, n] = sum over the segment's rows of A[r, m] B[r, n].
template <typename T>
__global__ void __launch_bounds__(NT) weights_kernel(const int32_t* __restrict__ seg, int E, int64_t R,
                                                     const T* __restrict__ A, const T* __restrict__ B, int M, int N,
                                                     float* __restrict__ C, int32_t* __restrict__ status) {
  __shared__ float As[BK][BM + 4];
  __shared__ float Bs[BK][BN + 4];
  chain_wait();
  if (!rows_valid(seg, E, R, status)) return;
  const int blocks_n = (N + BN - 1) / BN;  // (blocks of rows and columns in one grid dimension: both may be many)
  const int e = blockIdx.y, m0 = blockIdx.x / blocks_n * BM, n0 = blockIdx.x % blocks_n * BN;
  const int r0 = seg_at(seg, e, R), r1 = seg_at(seg, e + 1, R);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int k0 = r0; k0 < r1; k0 += BK) {
    const int kk = threadIdx.x / 16, q4 = (threadIdx.x % 16) * 4;
    const int64_t r = k0 + kk;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int m = m0 + q4 + q, n = n0 + q4 + q;
      As[kk][q4 + q] = (r < r1 && m < M) ? to_f(A[r * M + m]) : 0.f;
      Bs[kk][q4 + q] = (r < r1 && n < N) ? to_f(B[r * N + n]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk2 = 0; kk2 < BK; ++kk2) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = As[kk2][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = Bs[kk2][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  float* Ce = C + (int64_t)e * M * N;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) Ce[(int64_t)m * N + n] = acc[i][j];
    }
}

int64_t row_tiles(const int32_t* seg, int64_t R, int E) { return (R + BM - 1) / BM + (seg != nullptr ? E : 0); }

template <typename T, typename TO>
void forward_all(const LinearArgs& a, cudaStream_t s) {
  with_act(a.act, [&](auto tag) {
    constexpr int ACT = decltype(tag)::value;
    constexpr int CN = ACT == LRM_ACT_SWIGLU ? BN / 2 : BN;
    launch_chained(rows_kernel<T, TO, FWD, ACT>,
                   grid_wide(row_tiles(a.seg_offsets, a.R, a.E), (a.N + CN - 1) / CN), dim3(NT), 0, s,
                   a.seg_offsets, a.E, a.R, (const T*)a.x, (const T*)a.w, a.N, a.K, (const T*)a.bias,
                   (const TO*)a.residual, (TO*)a.y, (T*)a.z, a.status);
  });
}

template <typename T>
void backward_all(const LinearGradArgs& a, cudaStream_t s) {
  if (a.dx != nullptr && a.R > 0)
    launch_chained(rows_kernel<T, T, DX, LRM_ACT_NONE>,
                   grid_wide(row_tiles(a.seg_offsets, a.R, a.E), (a.K + BN - 1) / BN), dim3(NT), 0, s,
                   a.seg_offsets, a.E, a.R, (const T*)a.dz, (const T*)a.w, a.K, a.N, (const T*)nullptr,
                   (const T*)nullptr, (T*)a.dx, (T*)nullptr, a.status);
  if (a.dw != nullptr)
    launch_chained(weights_kernel<T>,
                   dim3((unsigned)((int64_t)((a.K + BN - 1) / BN) * ((a.N + BM - 1) / BM)), (unsigned)a.E), dim3(NT), 0,
                   s, a.seg_offsets, a.E, a.R, (const T*)a.dz, (const T*)a.x, a.N, a.K, a.dw, a.status);
}

}  // namespace

void launch_linear_simt(const LinearArgs& a, lrm_dtype dt, lrm_dtype out_dt, cudaStream_t s) {
  if (dt == LRM_F32)
    forward_all<float, float>(a, s);
  else if (out_dt == LRM_F32)
    forward_all<__nv_bfloat16, float>(a, s);
  else
    forward_all<__nv_bfloat16, __nv_bfloat16>(a, s);
}

void launch_linear_backward_simt(const LinearGradArgs& a, lrm_dtype dt, cudaStream_t s) {
  if (dt == LRM_F32)
    backward_all<float>(a, s);
  else
    backward_all<__nv_bfloat16>(a, s);
}

}  // namespace lrm
