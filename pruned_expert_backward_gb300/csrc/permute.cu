// Tokens sorted by expert (lrm_sort_tokens) and the weighted way back (lrm_combine) with its
// gradient (lrm_combine_backward).
//
// Pair u = (t, j) of expert e = topk_idx[u] goes to row
//     row(u) = #{v : expert(v) < e} + #{v < u : expert(v) = e},
// a stable counting sort; unrouted pairs (expert -1) form one more bucket behind the last expert's
// whose rows are zeroed.  The way back is y_t = residual_t + sum_j alpha_tj y_s[row(tj)].
// All three move each byte once and are bound by HBM at training size and by launch latency for a
// few tokens.  GB300, bf16, k = 8, 128 experts, of the measured HBM copy rate: sort 0.95 and combine 1.00 at
// T = 32768, H = 4096 (370 and 398 us), combine's gradient 0.99 at H = 2048 (339 us); at T = 64, H = 2048
// they take 4.2, 3.3 and 3.8 us.
//
// sort: up to kSmallPairs pairs one launch does everything: every CTA ranks all pairs for itself
// (a few hundred nanoseconds in shared memory) and copies the rows of its own tokens.  Beyond that
// several launches: counts of each chunk of pairs, the scan of every expert's counts down the chunks
// (neither up to kSelfPairs pairs), and the ranking of each chunk's pairs.  A token's row is read once and
// written k times, by a launch of its own with a CTA per token, or beside the ranking where rows are narrow.
// No atomics on anything that decides an order: all results are deterministic.
#include "common.cuh"
#include "kernels.h"

namespace lrm {

namespace {

// One launch up to this many pairs and experts (each warp keeps a count per bucket in shared memory):
// k = 8, 128 experts, H = 2048: 64 tokens 4.2 us against 4.9 in two launches, 128 tokens 4.6 : 4.9, 192 9.0 : 6.0.
constexpr int kSmallPairs = 1024;
constexpr int kSmallExperts = 256;
// Up to this many pairs every chunk's ranking counts all pairs itself, which saves two launches and the
// scratch (128 experts, H = 512: 4096 pairs 6.3 us on the device against 7.3, 8192 pairs 8.3 and 8.3, 16384
// pairs 12.8 and 10.0; a call through the binding 21 against 26 us).
constexpr int kSelfPairs = 8192;
constexpr int kChunkThreads = 256;  // multi-launch form: pairs of a chunk (whole tokens), at most one per thread

// Bucket of a pair: its expert, or E when it is not routed (-1) or its id is out of range (recorded).
__device__ __forceinline__ int bucket_of(int32_t id, int E, int32_t* status) {
  if (id >= 0 && id < E) return id;
  if (id != -1) set_status(status, LRM_ERR_BAD_INDEX);
  return E;
}

// Exclusive block-wide prefix sum of one int per thread (blockDim.x a multiple of 32); sm: 33 ints.
__device__ __forceinline__ int block_prefix(int v, int* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = lane < nw ? sm[lane] : 0;
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < nw) sm[lane] = w - own;
    if (lane == 31) sm[32] = w;
  }
  __syncthreads();
  const int res = sm[warp] + incl - v;
  __syncthreads();
  return res;
}

// Copies x rows of `ntok` tokens from t0 into their pairs' rows: s_dst[i * k + j] >= 0 is the row of
// pair (t0 + i, j); a negative entry -1 - r zeroes row r (an unrouted pair's place).  (token, 16-byte
// column) items are dealt to the threads, four tokens' loads in flight.  x_s has n_rows rows.
template <typename T>
__device__ __forceinline__ void copy_rows(const T* __restrict__ x, T* __restrict__ x_s, const int* s_dst, int64_t t0,
                                          int ntok, int k, int H, [[maybe_unused]] int64_t n_rows,
                                          [[maybe_unused]] int32_t* status) {
  constexpr int VN = VecTraits<T>::N;
  const int nv = H / VN;
  const int n = ntok * nv, step = blockDim.x;
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * step) {
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q * step;
      if (i < n) v[q] = ld_stream16_now(x + t0 * H + (int64_t)i * VN);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = i0 + q * step;
      if (i >= n) break;
      const int tok = i / nv, col = (i - tok * nv) * VN;
      for (int j = 0; j < k; ++j) {
        const int r = s_dst[tok * k + j];
        if (!LRM_DCHECK(r < n_rows && -1 - r < n_rows, status, LRM_ERR_BAD_INDEX)) continue;
        st16(x_s + (int64_t)(r >= 0 ? r : -1 - r) * H + col, r >= 0 ? v[q] : make_uint4(0, 0, 0, 0));
      }
    }
  }
}

// ---------------------------------------------------------------- one launch ---------
// Warp w ranks pairs [w * ppw, (w + 1) * ppw), 32 at a time in order, with __match_any_sync; counts
// are [warp][bucket] in shared memory, scanned down the warps and then across the buckets.
template <typename T>
__global__ void __launch_bounds__(1024) sort_small_kernel(const int32_t* __restrict__ idx, const T* __restrict__ x,
                                                          int n_tok, int k, int E, int H, int32_t* __restrict__ seg,
                                                          int32_t* __restrict__ pair_of_row,
                                                          int32_t* __restrict__ row_of_pair, T* __restrict__ x_s,
                                                          int32_t* __restrict__ status) {
  chain_wait();
  extern __shared__ int sh[];
  const int B = E + 1, nw = blockDim.x >> 5, P = n_tok * k;
  int* s_cnt = sh;             // [nw][B] counts, then the warps' exclusive offsets
  int* s_start = s_cnt + nw * B;  // [B] bucket starts
  int* s_row = s_start + B;    // [P] rows (-1 - r where the pair is not routed)
  int* s_scan = s_row + P;     // [33]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < nw * B; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  const int ppw = ((P + nw - 1) / nw + 31) / 32 * 32;
  int* cnt = s_cnt + warp * B;
  for (int u0 = warp * ppw; u0 < min(P, (warp + 1) * ppw); u0 += 32) {
    const int u = u0 + lane;
    const bool in = u < P;
    const int e = in ? bucket_of(idx[u], E, blockIdx.x == 0 ? status : nullptr) : B;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int before = in ? cnt[e] : 0;
    if (in) s_row[u] = before + __popc(same & ((1u << lane) - 1u)) + (e << 16);  // rank < 2^16, bucket
    __syncwarp();
    if (in && (same >> lane) == 1u) cnt[e] = before + __popc(same);  // the last lane of a group
    __syncwarp();
  }
  __syncthreads();
  for (int b0 = 0, run = 0; b0 < B; b0 += blockDim.x) {
    const int e = b0 + threadIdx.x;
    int tot = 0;
    if (e < B)
      for (int w = 0; w < nw; ++w) {
        const int c = s_cnt[w * B + e];
        s_cnt[w * B + e] = tot;
        tot += c;
      }
    const int ex = block_prefix(tot, s_scan);
    if (e < B) s_start[e] = run + ex;
    run += s_scan[32];
    __syncthreads();
  }
  for (int u = threadIdx.x; u < P; u += blockDim.x) {
    const int e = s_row[u] >> 16, r = s_start[e] + s_cnt[(u / ppw) * B + e] + (s_row[u] & 0xffff);
    s_row[u] = e < E ? r : -1 - r;
    if (blockIdx.x == 0 && LRM_DCHECK(r >= 0 && r < P, status, LRM_ERR_BAD_INDEX)) {
      row_of_pair[u] = e < E ? r : -1;
      pair_of_row[r] = e < E ? u : -1;
    }
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < B; e += blockDim.x) seg[e] = s_start[e];
  __syncthreads();
  if (x_s != nullptr)
    for (int t = blockIdx.x; t < n_tok; t += gridDim.x) copy_rows(x, x_s, s_row + t * k, t, 1, k, H, P, status);
}

// ---------------------------------------------------------------- several launches ---
__global__ void __launch_bounds__(kChunkThreads) sort_count_kernel(const int32_t* __restrict__ idx, int64_t P, int E,
                                                                   int chunk, int32_t* __restrict__ counts,
                                                                   int32_t* __restrict__ status) {
  chain_wait();
  extern __shared__ int hist[];  // [E + 1]
  const int B = E + 1;
  for (int e = threadIdx.x; e < B; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t c = blockIdx.x, u = c * chunk + threadIdx.x;
  if (threadIdx.x < chunk && u < P) atomicAdd(&hist[bucket_of(idx[u], E, status)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < B; e += blockDim.x) counts[c * B + e] = hist[e];
}

// One CTA per bucket: exclusive scan down its column of chunk counts; loads[e] = the bucket's size.
__global__ void __launch_bounds__(1024) sort_colscan_kernel(int32_t* __restrict__ counts, int64_t n_chunks, int B,
                                                            int32_t* __restrict__ loads) {
  chain_wait();
  __shared__ int sm[33];
  const int e = blockIdx.x;
  int run = 0;
  for (int64_t c0 = 0; c0 < n_chunks; c0 += blockDim.x) {
    const int64_t c = c0 + threadIdx.x;
    const int v = c < n_chunks ? counts[c * B + e] : 0;
    const int ex = block_prefix(v, sm);
    if (c < n_chunks) counts[c * B + e] = run + ex;
    run += sm[32];
    __syncthreads();
  }
  if (threadIdx.x == 0) loads[e] = run;
}

// SELF: every CTA counts all pairs itself, those before its chunk and the others, instead of reading the
// scanned counts of two launches before it.
template <typename T, bool SELF>
__global__ void __launch_bounds__(kChunkThreads) sort_rows_kernel(
    const int32_t* __restrict__ idx, const T* __restrict__ x, int64_t n_tok, int k, int E, int H, int chunk_tok,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ loads, int32_t* __restrict__ seg,
    int32_t* __restrict__ pair_of_row, int32_t* __restrict__ row_of_pair, T* __restrict__ x_s,
    int32_t* __restrict__ status) {
  chain_wait();
  constexpr int kWarps = kChunkThreads / 32;
  extern __shared__ int sh[];
  const int B = E + 1;
  int* s_start = sh;                // [B] this chunk's first row of each bucket
  int* s_cnt = s_start + B;         // [kWarps][B]
  int* s_row = s_cnt + kWarps * B;  // [kChunkThreads]
  __shared__ int s_scan[33];
  const int64_t c = blockIdx.x, t0 = c * chunk_tok;
  const int ntok = (int)min((int64_t)chunk_tok, n_tok - t0), np = ntok * k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kWarps * B; i += blockDim.x) s_cnt[i] = 0;
  int* s_before = s_cnt;  // SELF: pairs of each bucket before the chunk, and the others
  int* s_after = s_cnt + B;
  if (SELF) {
    __syncthreads();
    const int P = (int)(n_tok * k), first = (int)(t0 * k);
    for (int u0 = threadIdx.x; u0 < P; u0 += 4 * kChunkThreads) {
      int id[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) id[q] = u0 + q * kChunkThreads < P ? idx[u0 + q * kChunkThreads] : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = u0 + q * kChunkThreads;
        if (u < P) atomicAdd((u < first ? s_before : s_after) + bucket_of(id[q], E, c == 0 ? status : nullptr), 1);
      }
    }
    __syncthreads();
  }
  for (int b0 = 0, run = 0; b0 < B; b0 += blockDim.x) {
    const int e = b0 + threadIdx.x;
    const int load = e >= B ? 0 : (SELF ? s_before[e] + s_after[e] : loads[e]);
    const int ex = block_prefix(load, s_scan);
    if (e < B) {
      s_start[e] = run + ex + (SELF ? s_before[e] : counts[c * B + e]);
      if (c == 0) seg[e] = run + ex;
    }
    run += s_scan[32];
    __syncthreads();
  }
  if (SELF) {  // their place becomes the warps' counts
    for (int i = threadIdx.x; i < 2 * B; i += blockDim.x) s_cnt[i] = 0;
    __syncthreads();
  }
  const bool in = threadIdx.x < np;
  const int64_t u = t0 * k + threadIdx.x;
  const int e = in ? bucket_of(idx[u], E, nullptr) : B;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  if (in && (same >> lane) == 1u) s_cnt[warp * B + e] = __popc(same);
  __syncthreads();
  if (in) {
    int r = s_start[e] + __popc(same & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) r += s_cnt[w * B + e];
    s_row[threadIdx.x] = e < E ? r : -1 - r;
    if (LRM_DCHECK(r >= 0 && r < n_tok * k, status, LRM_ERR_BAD_INDEX)) {
      row_of_pair[u] = e < E ? r : -1;
      pair_of_row[r] = e < E ? (int32_t)u : -1;
    }
  }
  __syncthreads();
  if (x_s != nullptr) copy_rows(x, x_s, s_row, t0, ntok, k, H, n_tok * k, status);
}

// One CTA per token copies its row into its pairs' rows; CTA t also zeroes every n_tok-th row behind the
// last segment, from seg[E] + t on.
template <typename T>
__global__ void __launch_bounds__(256) sort_copy_kernel(const int32_t* __restrict__ row_of_pair,
                                                        const int32_t* __restrict__ seg, const T* __restrict__ x,
                                                        int64_t n_tok, int k, int E, int H, T* __restrict__ x_s,
                                                        [[maybe_unused]] int32_t* status) {
  chain_wait();
  constexpr int VN = VecTraits<T>::N;
  __shared__ int s_row[LRM_MAX_TOPK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < k) {
    const int r = row_of_pair[t * k + threadIdx.x];
    s_row[threadIdx.x] = LRM_DCHECK(r >= -1 && r < n_tok * k, status, LRM_ERR_BAD_INDEX) ? r : -1;
  }
  __syncthreads();
  const int nv = H / VN;
  for (int v0 = threadIdx.x; v0 < nv; v0 += 2 * blockDim.x) {
    const int v1 = v0 + blockDim.x;
    const uint4 a = ld_stream16_now(x + t * H + (int64_t)v0 * VN);
    uint4 b = a;
    if (v1 < nv) b = ld_stream16_now(x + t * H + (int64_t)v1 * VN);
    for (int j = 0; j < k; ++j) {
      if (s_row[j] < 0) continue;
      T* row = x_s + (int64_t)s_row[j] * H;
      st16(row + (int64_t)v0 * VN, a);
      if (v1 < nv) st16(row + (int64_t)v1 * VN, b);
    }
  }
  for (int64_t r = seg[E] + t; r < n_tok * k; r += n_tok)
    for (int v = threadIdx.x; v < nv; v += blockDim.x) st16(x_s + r * H + (int64_t)v * VN, make_uint4(0, 0, 0, 0));
}

// ---------------------------------------------------------------- the way back -------
// A CTA covers TOK tokens and blockDim.x 16-byte columns (times a loop); each thread walks the CTA's
// routed pairs with 8 row loads in flight and adds each token's in j order in fp32.
constexpr int kCombineLoads = 8;

template <typename T, int TOK>
__global__ void __launch_bounds__(256) combine_kernel(const int32_t* __restrict__ row_of_pair,
                                                      const float* __restrict__ alpha, const T* __restrict__ y_s,
                                                      const T* residual, int64_t n_tok, int k, int H, int64_t cap,
                                                      T* y, int32_t* __restrict__ status) {
  // y may be the residual's buffer: each 16 bytes are read and then written by one thread
  chain_wait();
  constexpr int VN = VecTraits<T>::N;
  constexpr int L = kCombineLoads;
  __shared__ int2 s_item[TOK * LRM_MAX_TOPK];  // (token within the CTA, row), routed pairs in order
  __shared__ float s_w[TOK * LRM_MAX_TOPK];
  __shared__ int s_n;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  const int ntok = (int)min((int64_t)TOK, n_tok - t0);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int base = 0;
    for (int q0 = 0; q0 < ntok * k; q0 += 32) {
      const int q = q0 + lane;
      const int r = q < ntok * k ? (int)checked_row(row_of_pair[t0 * k + q], cap, status) : -1;
      const unsigned m = __ballot_sync(0xffffffffu, r >= 0);
      if (r >= 0) {
        const int at = base + __popc(m & ((1u << lane) - 1u));
        s_item[at] = make_int2(q / k, r);
        s_w[at] = alpha[t0 * k + q];
      }
      base += __popc(m);
    }
    if (lane == 0) s_n = base;
  }
  __syncthreads();
  const int n = s_n, nv = H / VN;
  for (int v = blockIdx.y * blockDim.x + threadIdx.x; v < nv; v += gridDim.y * blockDim.x) {
    float acc[VN];
#pragma unroll
    for (int q = 0; q < VN; ++q) acc[q] = 0.f;
    int cur = 0;  // the token acc belongs to; tokens before it are written
    auto flush = [&]() {
      const int64_t at = (t0 + cur) * H + (int64_t)v * VN;
      if (residual != nullptr) {
        float f[VN];
        unpack(*reinterpret_cast<const uint4*>(residual + at), f);
#pragma unroll
        for (int q = 0; q < VN; ++q) acc[q] += f[q];
      }
      st16(y + at, pack(acc));
#pragma unroll
      for (int q = 0; q < VN; ++q) acc[q] = 0.f;
      ++cur;
    };
    for (int b0 = 0; b0 < n; b0 += L) {
      uint4 vals[L];
#pragma unroll
      for (int m = 0; m < L; ++m)
        if (b0 + m < n) vals[m] = ld_stream16_now(y_s + (int64_t)s_item[b0 + m].y * H + (int64_t)v * VN);
#pragma unroll
      for (int m = 0; m < L; ++m) {
        if (b0 + m >= n) break;
        const int tok = s_item[b0 + m].x;
        const float w = s_w[b0 + m];
        while (cur < tok) flush();
        float f[VN];
        unpack(vals[m], f);
#pragma unroll
        for (int q = 0; q < VN; ++q) acc[q] = fmaf(w, f[q], acc[q]);
      }
    }
    while (cur < ntok) flush();
  }
}

// Narrow rows (at most 32 columns of 16 bytes): a warp per token, a lane per column, 8 row loads in flight.
template <typename T>
__global__ void __launch_bounds__(256) combine_narrow_kernel(const int32_t* __restrict__ row_of_pair,
                                                             const float* __restrict__ alpha,
                                                             const T* __restrict__ y_s, const T* residual,
                                                             int64_t n_tok, int k, int H, int64_t cap, T* y,
                                                             int32_t* __restrict__ status) {
  chain_wait();
  constexpr int VN = VecTraits<T>::N;
  constexpr int L = kCombineLoads;
  const int lane = threadIdx.x & 31, nv = H / VN;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= n_tok) return;
  const bool in = lane < nv;
  int r = -1;  // lane j holds pair j's row and weight
  float w = 0.f;
  if (lane < k) {
    r = (int)checked_row(row_of_pair[t * k + lane], cap, status);
    w = alpha[t * k + lane];
  }
  float acc[VN];
#pragma unroll
  for (int q = 0; q < VN; ++q) acc[q] = 0.f;
  for (int j0 = 0; j0 < k; j0 += L) {
    uint4 vals[L];
#pragma unroll
    for (int m = 0; m < L; ++m) {
      const int row = __shfl_sync(0xffffffffu, r, (j0 + m) & 31);
      if (in && j0 + m < k && row >= 0) vals[m] = ld_stream16_now(y_s + (int64_t)row * H + lane * VN);
    }
#pragma unroll
    for (int m = 0; m < L; ++m) {
      const int row = __shfl_sync(0xffffffffu, r, (j0 + m) & 31);
      const float wj = __shfl_sync(0xffffffffu, w, (j0 + m) & 31);
      if (!in || j0 + m >= k || row < 0) continue;
      float f[VN];
      unpack(vals[m], f);
#pragma unroll
      for (int q = 0; q < VN; ++q) acc[q] = fmaf(wj, f[q], acc[q]);
    }
  }
  if (!in) return;
  if (residual != nullptr) {
    float f[VN];
    unpack(*reinterpret_cast<const uint4*>(residual + t * H + lane * VN), f);
#pragma unroll
    for (int q = 0; q < VN; ++q) acc[q] += f[q];
  }
  st16(y + t * H + lane * VN, pack(acc));
}

// The gradient for narrow rows: a warp per token.
template <typename T>
__global__ void __launch_bounds__(256) combine_backward_narrow_kernel(
    const int32_t* __restrict__ row_of_pair, const float* __restrict__ alpha, const T* __restrict__ dy,
    const T* __restrict__ y_s, int64_t n_tok, int k, int H, int64_t cap, T* __restrict__ dy_s,
    float* __restrict__ dalpha, int32_t* __restrict__ status) {
  chain_wait();
  constexpr int VN = VecTraits<T>::N;
  constexpr int L = kCombineLoads;
  const int lane = threadIdx.x & 31, nv = H / VN;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= n_tok) return;
  const bool in = lane < nv;
  int r = -1;
  float w = 0.f, mine = 0.f;  // lane j ends with pair j's dot product
  if (lane < k) {
    r = (int)checked_row(row_of_pair[t * k + lane], cap, status);
    w = alpha[t * k + lane];
  }
  float d[VN];
  unpack(in ? ldg16(dy + t * H + lane * VN) : make_uint4(0, 0, 0, 0), d);
  for (int j0 = 0; j0 < k; j0 += L) {
    uint4 vals[L];
#pragma unroll
    for (int m = 0; m < L; ++m) {
      const int row = __shfl_sync(0xffffffffu, r, (j0 + m) & 31);
      if (y_s != nullptr && in && j0 + m < k && row >= 0)
        vals[m] = ld_stream16_now(y_s + (int64_t)row * H + lane * VN);
    }
#pragma unroll
    for (int m = 0; m < L; ++m) {
      const int row = __shfl_sync(0xffffffffu, r, (j0 + m) & 31);
      const float wj = __shfl_sync(0xffffffffu, w, (j0 + m) & 31);
      if (j0 + m >= k || row < 0) continue;  // warp-uniform
      float dot = 0.f, f[VN];
      if (in) {
        if (y_s != nullptr) {
          unpack(vals[m], f);
#pragma unroll
          for (int q = 0; q < VN; ++q) dot = fmaf(d[q], f[q], dot);
        }
#pragma unroll
        for (int q = 0; q < VN; ++q) f[q] = wj * d[q];
        st16(dy_s + (int64_t)row * H + lane * VN, pack(f));
      }
      dot = warp_sum(dot);
      if (lane == j0 + m) mine = dot;
    }
  }
  if (dalpha != nullptr && lane < k) dalpha[t * k + lane] = mine;
}

// One CTA per token: dy_t is read once; every routed pair's y_s row is read for its dot product with
// dy_t and its dy_s row written, KB pairs at a time (their loads in flight together).
template <typename T, int KB>
__global__ void __launch_bounds__(256) combine_backward_kernel(const int32_t* __restrict__ row_of_pair,
                                                               const float* __restrict__ alpha,
                                                               const T* __restrict__ dy, const T* __restrict__ y_s,
                                                               int k, int H, int64_t cap, T* __restrict__ dy_s,
                                                               float* __restrict__ dalpha,
                                                               int32_t* __restrict__ status) {
  chain_wait();
  constexpr int VN = VecTraits<T>::N;
  __shared__ int64_t s_row[LRM_MAX_TOPK];
  __shared__ float s_w[LRM_MAX_TOPK];
  __shared__ float s_dot[8][LRM_MAX_TOPK];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (threadIdx.x < k) {
    s_row[threadIdx.x] = checked_row(row_of_pair[t * k + threadIdx.x], cap, status);
    s_w[threadIdx.x] = alpha[t * k + threadIdx.x];
  }
  __syncthreads();
  const int nv = H / VN;
  for (int j0 = 0; j0 < k; j0 += KB) {
    float dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) dot[j] = 0.f;
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
      const uint4 d4 = ldg16(dy + t * H + (int64_t)v * VN);
      uint4 rows[KB];
      if (y_s != nullptr)
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (j0 + j < k && s_row[j0 + j] >= 0) rows[j] = ld_stream16_now(y_s + s_row[j0 + j] * H + (int64_t)v * VN);
      float d[VN];
      unpack(d4, d);
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (j0 + j >= k || s_row[j0 + j] < 0) continue;
        float f[VN];
        if (y_s != nullptr) {
          unpack(rows[j], f);
#pragma unroll
          for (int q = 0; q < VN; ++q) dot[j] = fmaf(d[q], f[q], dot[j]);
        }
#pragma unroll
        for (int q = 0; q < VN; ++q) f[q] = s_w[j0 + j] * d[q];
        st16(dy_s + s_row[j0 + j] * H + (int64_t)v * VN, pack(f));
      }
    }
    if (dalpha != nullptr)
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        dot[j] = warp_sum(dot[j]);
        if (lane == 0 && j0 + j < k) s_dot[warp][j0 + j] = dot[j];
      }
  }
  if (dalpha == nullptr) return;
  __syncthreads();
  if (threadIdx.x < k) {
    float s = 0.f;
    for (int w = 0; w < nw; ++w) s += s_dot[w][threadIdx.x];
    dalpha[t * k + threadIdx.x] = s_row[threadIdx.x] >= 0 ? s : 0.f;
  }
}

// Threads of a row of `nv` 16-byte columns: up to 256, and as few as the same number of passes needs.
int row_threads(int nv) {
  const int passes = (nv + 255) / 256;
  return ((nv + passes - 1) / passes + 31) / 32 * 32;
}

template <typename T>
lrm_status sort_all(const SortArgs& a, cudaStream_t s) {
  const int64_t P = a.T * a.k;
  const int B = a.E + 1;
  if (sort_in_one_launch(a.T, a.k, a.E)) {
    // a warp for every 64 pairs, at least as many threads as a row has 16-byte columns (up to 256)
    int threads = (int)((P + 63) / 64) * 32;
    const int cols = (a.H / VecTraits<T>::N + 31) / 32 * 32;
    threads = threads < cols ? (cols < 256 ? cols : 256) : threads;
    threads = threads < 32 ? 32 : threads;
    const int nw = threads / 32;
    const size_t smem = sizeof(int) * ((size_t)(nw + 1) * B + (size_t)P + 33);
    const int64_t blocks = a.x_s != nullptr && a.T > 0 ? a.T : 1;
    launch_chained(sort_small_kernel<T>, dim3((unsigned)(blocks < 608 ? blocks : 608)), dim3(threads), smem, s,
                   a.topk_idx, (const T*)a.x, (int)a.T, a.k, a.E, a.H, a.seg_offsets, a.pair_of_row, a.row_of_pair,
                   (T*)a.x_s, a.status);
  } else {
    const int chunk_tok = sort_chunk_tokens(a.k);
    const int64_t nc = a.T > 0 ? (a.T + chunk_tok - 1) / chunk_tok : 1;
    // Rows of 1 KB and more are copied by a launch of their own, a CTA per token (T = 32768, k = 8, H = 4096:
    // 370 against 394 us; T = 2048, H = 2048: 16 against 56 us), narrower ones beside the ranking (T = 30000,
    // H = 72: 16 against 41 us).
    const bool apart = a.x_s != nullptr && a.T > 0 && a.H >= 64 * VecTraits<T>::N;
    T* beside = apart ? nullptr : (T*)a.x_s;
    const size_t smem = sizeof(int) * ((size_t)B * (1 + kChunkThreads / 32) + kChunkThreads);
    if (sort_self_counted(a.T, a.k)) {
      launch_chained(sort_rows_kernel<T, true>, dim3((unsigned)nc), dim3(kChunkThreads), smem, s, a.topk_idx,
                     (const T*)a.x, a.T, a.k, a.E, a.H, chunk_tok, (const int32_t*)nullptr, (const int32_t*)nullptr,
                     a.seg_offsets, a.pair_of_row, a.row_of_pair, beside, a.status);
    } else {
      launch_chained(sort_count_kernel, dim3((unsigned)nc), dim3(kChunkThreads), sizeof(int) * B, s, a.topk_idx, P,
                     a.E, chunk_tok * a.k, a.counts, a.status);
      launch_chained(sort_colscan_kernel, dim3(B), dim3(nc > 256 ? 1024 : 256), 0, s, a.counts, nc, B, a.loads);
      launch_chained(sort_rows_kernel<T, false>, dim3((unsigned)nc), dim3(kChunkThreads), smem, s, a.topk_idx,
                     (const T*)a.x, a.T, a.k, a.E, a.H, chunk_tok, (const int32_t*)a.counts, (const int32_t*)a.loads,
                     a.seg_offsets, a.pair_of_row, a.row_of_pair, beside, a.status);
    }
    if (apart) {
      const int cols = row_threads((a.H / VecTraits<T>::N + 1) / 2);
      launch_chained(sort_copy_kernel<T>, dim3((unsigned)a.T), dim3(cols < 64 ? 64 : cols), 0, s,
                     (const int32_t*)a.row_of_pair, (const int32_t*)a.seg_offsets, (const T*)a.x, a.T, a.k, a.E, a.H,
                     (T*)a.x_s, a.status);
    }
  }
  return cudaGetLastError() == cudaSuccess ? LRM_OK : LRM_ERR_CUDA;
}

template <typename T>
void combine_all(const int32_t* row_of_pair, const float* alpha, const void* y_s, const void* residual, int64_t n_tok,
                 int32_t k, int32_t H, int64_t cap, void* y, int32_t* status, cudaStream_t s) {
  const int nv = H / VecTraits<T>::N;
  if (nv <= 32) {
    launch_chained(combine_narrow_kernel<T>, dim3((unsigned)((n_tok + 7) / 8)), dim3(256), 0, s, row_of_pair, alpha,
                   (const T*)y_s, (const T*)residual, n_tok, k, H, cap, (T*)y, status);
    return;
  }
  // few tokens: one token and 64 columns per CTA, so that the rows spread over the GPU
  if (n_tok < 2048) {
    const int blocks = (nv + 63) / 64;
    const dim3 grid((unsigned)n_tok, (unsigned)(blocks < 65535 ? blocks : 65535));
    launch_chained(combine_kernel<T, 1>, grid, dim3(64), 0, s, row_of_pair, alpha, (const T*)y_s,
                   (const T*)residual, n_tok, k, H, cap, (T*)y, status);
    return;
  }
  // tokens of a CTA: about 32 rows to walk (T = 8192, H = 2048, bf16: k = 8 50 us with 4 tokens, 55 us with 8;
  // k = 1 19 and 18 us)
  if (k >= 6)
    launch_chained(combine_kernel<T, 4>, dim3((unsigned)((n_tok + 3) / 4)), dim3(row_threads(nv)), 0, s, row_of_pair,
                   alpha, (const T*)y_s, (const T*)residual, n_tok, k, H, cap, (T*)y, status);
  else
    launch_chained(combine_kernel<T, 8>, dim3((unsigned)((n_tok + 7) / 8)), dim3(row_threads(nv)), 0, s, row_of_pair,
                   alpha, (const T*)y_s, (const T*)residual, n_tok, k, H, cap, (T*)y, status);
}

template <typename T>
void combine_backward_all(const int32_t* row_of_pair, const float* alpha, const void* dy, const void* y_s,
                          int64_t n_tok, int32_t k, int32_t H, int64_t cap, void* dy_s, float* dalpha, int32_t* status,
                          cudaStream_t s) {
  if (H / VecTraits<T>::N <= 32) {
    launch_chained(combine_backward_narrow_kernel<T>, dim3((unsigned)((n_tok + 7) / 8)), dim3(256), 0, s, row_of_pair,
                   alpha, (const T*)dy, (const T*)y_s, n_tok, k, H, cap, (T*)dy_s, dalpha, status);
    return;
  }
  // few experts a token: fewer rows' registers, so more tokens in flight (T = 8192, H = 2048, k = 1: 21 against
  // 33 us)
  auto kernel = k <= 2   ? combine_backward_kernel<T, 2>
                : k <= 4 ? combine_backward_kernel<T, 4>
                         : combine_backward_kernel<T, 8>;
  launch_chained(kernel, dim3((unsigned)n_tok), dim3(row_threads(H / VecTraits<T>::N)), 0, s, row_of_pair, alpha,
                 (const T*)dy, (const T*)y_s, k, H, cap, (T*)dy_s, dalpha, status);
}

}  // namespace

bool sort_in_one_launch(int64_t T, int32_t k, int32_t E) { return T * k <= kSmallPairs && E <= kSmallExperts; }
bool sort_self_counted(int64_t T, int32_t k) { return T * k <= kSelfPairs; }
bool sort_needs_scratch(int64_t T, int32_t k, int32_t E) {
  return !sort_in_one_launch(T, k, E) && !sort_self_counted(T, k);
}
int sort_chunk_tokens(int32_t k) { return kChunkThreads / k; }

lrm_status launch_sort_tokens(const SortArgs& a, lrm_dtype dt, cudaStream_t s) {
  return dt == LRM_BF16 ? sort_all<__nv_bfloat16>(a, s) : sort_all<float>(a, s);
}

void launch_combine(const int32_t* row_of_pair, const float* alpha, const void* y_s, const void* residual, int64_t T,
                    int32_t k, int32_t H, lrm_dtype dt, int64_t cap, void* y, int32_t* status, cudaStream_t s) {
  if (dt == LRM_BF16)
    combine_all<__nv_bfloat16>(row_of_pair, alpha, y_s, residual, T, k, H, cap, y, status, s);
  else
    combine_all<float>(row_of_pair, alpha, y_s, residual, T, k, H, cap, y, status, s);
}

void launch_combine_backward(const int32_t* row_of_pair, const float* alpha, const void* dy, const void* y_s, int64_t T,
                             int32_t k, int32_t H, lrm_dtype dt, int64_t cap, void* dy_s, float* dalpha,
                             int32_t* status, cudaStream_t s) {
  if (dt == LRM_BF16)
    combine_backward_all<__nv_bfloat16>(row_of_pair, alpha, dy, y_s, T, k, H, cap, dy_s, dalpha, status, s);
  else
    combine_backward_all<float>(row_of_pair, alpha, dy, y_s, T, k, H, cap, dy_s, dalpha, status, s);
}

}  // namespace lrm
