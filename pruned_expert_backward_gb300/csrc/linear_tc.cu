// lrm_linear and lrm_linear_backward on the tensor cores of sm_103a (tcgen05, TMEM, TMA).
//
//   FWD  y  = act(x W[e]^T + b[e]) + residual   (M = the segment's rows, N columns, K = hidden)
//   DX   dx = dz W[e]                           (M = the segment's rows, N = hidden, K = columns of dz)
//   DW   dW[e] = dz^T x                         (M = columns of dz, N = hidden, K = the segment's rows)
//
// CTAs run in pairs (a cluster of two) over a persistent grid; a pair computes a 256 x BN tile with
// tcgen05.mma.cta_group::2: each CTA stages its own 128 rows of A and half of the BN columns of B per
// 64-deep K slice and holds 128 rows of the fp32 accumulator in TMEM, twice, so that one tile's
// epilogue runs under the next tile's products.  Warp 0 issues the TMA loads, warp 1 of the leader the
// MMAs, warps 2-9 are the epilogue: two per 32-row TMEM quarter, each taking half of the columns.  Warps
// 0 and 1 run their loops whole and one elected lane issues: under a lane test instead, an MMA took 62-75
// cycles to issue, not 26, and a narrow tile 0.21 us a K slice, not 0.155.
//
// GB300, bf16.  32768 x 4096 x 4096 with bias, GELU and residual: 577 us, the tensor pipe 89 % active; back
// to back for seconds the power limit makes it 700 us.  65536 rows over 128 experts, zipf 1, to 2 x 768 with
// SwiGLU, K = 2048: 313 us, 330 us with z, the pipe 85 % active (1.37 times the rows' products: every
// segment ends in a partial 256-row tile); its dx 317 us (87 %), its dW 420 us (1.6 GB of fp32 stores and
// 3.4 GB of operands through L2: 248 us and 291 us apart).
// A SwiGLU tile's columns are BN / 2 gate columns (the leader's half of B) and the BN / 2 up columns
// that go with them (the other CTA's).
//
// Rows of a segment's last tile that belong to the next expert are computed and not stored: full
// 32-row blocks leave by TMA from a ring of swizzled 2 KB boxes, partial ones by per-lane stores.  The
// row-tile prefix of the segments is formed by every CTA for itself in shared memory (E <= 1024 sums,
// below a microsecond), so FWD and DX are one launch without scratch.  DW reduces over rows, which
// must not run into the next segment: its operands come through per-expert tensor maps whose row
// extent ends at the segment's end (a small launch before it writes them), so TMA fills with zeros.
//
// fp32 accumulation.  The tensor core adds into its fp32 accumulator by truncation: against 64 bits a
// sum of 2048 products is 2e-6 off (5.6e-6 when all have one sign), one of 32768 3.8e-5 (1.8e-4).
// That is far below one bf16 rounding, so bf16 results of up to 65536 products are taken as they are.  For fp32
// results and longer sums (PROMOTE) the accumulator is moved out of TMEM every `pk` K slices and added up in
// registers, rounding to nearest.
//
// fp32 inputs are split into three bf16 planes, x = x0 + x1 + x2 (24 bits), and the six products of
// weight 2^-16 and more are summed, the smallest first: x2 w0, x0 w2, x1 w1, x1 w0, x0 w1, x0 w0.  Only
// the producer knows: it walks the K range once per term with the planes as the outer coordinate of
// the operand maps.  What is left out is below 2^-24 of |x||w|.
#include "kernels.h"
#include "linear.cuh"
#include "tc_host.h"
#include "tc_ptx.cuh"

#include <type_traits>

namespace lrm {

namespace {

constexpr int kBM = 128;  // rows per CTA; a pair tile has 256
constexpr int kBK = 64;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kABytes = kBM * kBK * 2;
constexpr int kPairs = 76;  // CTA pairs of the GPU, for the choices that fix the scratch
constexpr int kBoxBytes = 2048;  // 32 rows x 64 bytes, 64-byte swizzle: 32 bf16 or 16 fp32 columns

enum Kind { FWD = 0, DX = 1, DW = 2 };

template <int KIND, int BN>
struct Cfg {
  static constexpr int kBBytes = BN / 2 * kBK * 2;  // this CTA's half of the columns
  static constexpr int kSlice = kABytes + kBBytes;
  static constexpr int kSub = BN == 256 ? 1 : 2;  // K slices of a stage
  static constexpr int kStage = kSub * kSlice;
  static constexpr int kStages = BN == 256 ? 6 : (BN == 128 ? 3 : 4);
  // Store boxes that an epilogue warp uses in turn.  In the 256-column tile operand stages are worth more:
  // with 5 stages and 3 boxes 65536 rows over 128 experts took 339 us (SwiGLU, K = 2048) and 334 us (DX)
  // against 331 and 319 us; 16 epilogue warps and 5 stages 358 and 336 us.
  static constexpr int kBoxes = BN == 256 ? (KIND == DW ? 2 : 1) : 3;
  static constexpr uint32_t kEpi = kStages * kStage;
  static constexpr uint32_t kBars = kEpi + kEpiWarps * kBoxes * kBoxBytes;
  static constexpr int kNBars = 2 * kStages + 5;  // full, empty, accumulator full[2] and empty[2], drain
  static constexpr int kTmem = BN == 64 ? 128 : 2 * BN;
  static constexpr int kPrefix = KIND == DW ? 0 : LRM_MAX_EXPERTS + 2;
  static constexpr size_t smem() { return 1024 + kBars + kNBars * 8 + 16 + 4 * (kPrefix + kThreads / 32); }
  static_assert(1024 + kBars + kNBars * 8 + 16 + 4 * (kPrefix + kThreads / 32) <= 232448, "shared memory");
};

struct Params {
  int E;
  int64_t R;
  int N;          // columns of the output (FWD: of y)
  int M;          // DW: rows of dW[e]
  int red;        // FWD, DX: length of the reduction
  int tiles_n;
  int tiles_m;    // DW: pair tiles along M
  int part_rows;  // DW without segments: rows of each part of the reduction (E parts, each with its own output)
  int terms;      // 1, or 6 for fp32 inputs in three planes
  int pk;         // K slices per accumulator (PROMOTE)
  int parts;      // FWD, DX: parts of the reduction, each a tile of its own with its own output [R][N]
  int part_len;   // K slices of a part (of all terms together)
  // operands that are contiguous along M or N (DX: B, DW: both): both 64-column blocks of a CTA's 128 columns
  // come in one box, where the columns are a multiple of 64 (else a box would wrap into the next row)
  bool one_box_a, one_box_b;
  const int32_t* seg;       // NULL: one dense problem
  const int32_t* plan;      // DW with segments: [0] 1 if they are valid, [1 ..] experts, longest first
  const CUtensorMap* maps;  // DW with segments: [2][E] operand maps cut at the segment's end
  int act;
  const void *bias, *residual;
  void *y, *z;
  int32_t* status;
};

// Term i of the split product: which plane of A and of B (the smallest products first).
__device__ __forceinline__ int plane_a(int term) { return (0x001102 >> (4 * term)) & 15; }
__device__ __forceinline__ int plane_b(int term) { return (0x010120 >> (4 * term)) & 15; }

template <int BN>
__host__ __device__ constexpr uint32_t instr_desc(uint32_t a_mn, uint32_t b_mn) {  // D fp32, A and B bf16, M = 256
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) | ((uint32_t)(BN >> 3) << 17) |
         ((uint32_t)((2 * kBM) >> 4) << 24);
}

// At most N of this thread's bulk stores have not read their shared memory yet.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// The i-th tile of a CTA pair: round robin, every second round backwards, so that where the tiles get
// shorter along the order (DW: longest expert first) no pair takes the longer one of every round.
__device__ __forceinline__ int nth_tile(int i, int pair, int n_pairs) {
  return i * n_pairs + (i & 1 ? n_pairs - 1 - pair : pair);
}

struct Tile {
  int e;
  int row0, row_end;  // FWD, DX: this CTA's output rows; DW: the rows summed over
  int m0, n0;         // DW: this CTA's first output row; n0: first output column
  int slices;         // K slices of one term
  int part, lo, hi;   // part of the reduction, and its K slices, counted over all terms
  bool has_rows;
};

template <int KIND, int BN, bool GLU>
__device__ __forceinline__ Tile decode(const Params& p, const int* prefix, int t, int rank) {
  Tile d;
  d.part = 0;
  if (KIND != DW && p.parts > 1) {
    d.part = t % p.parts;
    t /= p.parts;
  }
  const int mg = t / p.tiles_n, nt = t - mg * p.tiles_n;
  d.n0 = nt * (GLU ? BN / 2 : BN);
  if (KIND == DW) {
    const int ei = mg / p.tiles_m;
    d.e = p.seg != nullptr ? __ldg(p.plan + 1 + ei) : ei;
    d.m0 = (2 * (mg - ei * p.tiles_m) + rank) * kBM;
    d.row0 = p.seg != nullptr ? __ldg(p.seg + d.e) : d.e * p.part_rows;
    d.row_end = p.seg != nullptr ? __ldg(p.seg + d.e + 1) : (int)min(p.R, (int64_t)d.row0 + p.part_rows);
    d.slices = (d.row_end - d.row0 + kBK - 1) / kBK;
    d.lo = 0;
    d.hi = d.slices * p.terms;
    d.has_rows = d.m0 < p.M;
    return d;
  }
  d.m0 = 0;
  d.e = 0;
  int end = (int)p.R;
  if (p.seg != nullptr) {
    int lo = 0, hi = p.E;  // the last e with prefix[e] <= mg
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= mg) lo = mid; else hi = mid;
    }
    d.e = lo;
    end = __ldg(p.seg + lo + 1);
    d.row0 = __ldg(p.seg + lo) + (mg - prefix[lo]) * (2 * kBM) + rank * kBM;
  } else {
    d.row0 = mg * (2 * kBM) + rank * kBM;
  }
  d.row_end = min(end, d.row0 + kBM);
  d.slices = (p.red + kBK - 1) / kBK;
  d.lo = d.part * p.part_len;
  d.hi = min(d.slices * p.terms, d.lo + p.part_len);
  d.has_rows = d.row0 < end;
  return d;
}

// BLOCKS blocks of 64 columns from column c0 and 64 rows from r of matrix g.
template <int BLOCKS>
__device__ __forceinline__ void load_columns(uint32_t dst, const CUtensorMap* map, int c0, int r, int g, bool one_box,
                                             uint32_t bar) {
  if (one_box) {
    tma_load_4d_pair(dst, map, 0, r, c0 / 64, g, bar);
  } else {
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c) tma_load_3d_pair(dst + c * 8192, map, c0 + c * 64, r, g, bar);
  }
}

// 32 columns of one row per lane go out: whole 32-row blocks through the warp's next box(es) and TMA
// (which clips columns past the tensor), others by each live lane.
template <int BOXES>
struct Out {
  uint8_t* boxes;
  uint32_t boxes_s;
  int next;
  __device__ __forceinline__ void box(const uint4 (&q)[4], const CUtensorMap* map, int lane, int n, int row, int e) {
    if (lane == 0) bulk_wait_read<BOXES - 1>();  // the store that used this box has read it
    __syncwarp();
    uint8_t* line = boxes + next * kBoxBytes + lane * 64;
    const int swz = (lane >> 1) & 3;  // 64-byte swizzle: piece j of row r sits at j ^ ((r >> 1) & 3)
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(line + ((j ^ swz) << 4)) = q[j];
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_3d(map, boxes_s + next * kBoxBytes, n, row, e);
    next = next + 1 == BOXES ? 0 : next + 1;
  }
  template <typename T>
  __device__ __forceinline__ void put(const float (&v)[32], const CUtensorMap* map, int lane, int n, int cols, int row,
                                      int e, bool whole, bool live, T* row_ptr) {
    constexpr int VN = VecTraits<T>::N;
    constexpr int PC = 4 * VN;  // columns of a box
#pragma unroll
    for (int h = 0; h < 32 / PC; ++h) {
      uint4 q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) f[i] = v[h * PC + j * VN + i];
        q[j] = pack(f);
      }
      const int c0 = n + h * PC;
      if (whole) {
        if (c0 < cols) box(q, map, lane, c0, row, e);  // warp-uniform
      } else if (live) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + j * VN < cols) st16(row_ptr + c0 + j * VN, q[j]);
      }
    }
  }
};

// v += 32 values of a row of T at column n (columns past `cols` are left alone).
template <typename T>
__device__ __forceinline__ void add_row(float (&v)[32], const T* row, int n, int cols) {
  constexpr int VN = VecTraits<T>::N;
#pragma unroll
  for (int j = 0; j < 32 / VN; ++j)
    if (n + j * VN < cols) {
      float f[VN];
      unpack(*reinterpret_cast<const uint4*>(row + n + j * VN), f);
#pragma unroll
      for (int i = 0; i < VN; ++i) v[j * VN + i] += f[i];
    }
}

template <typename T>
__device__ __forceinline__ void add_vectors(float (&v)[32], const uint4* r) {
  constexpr int VN = VecTraits<T>::N;
#pragma unroll
  for (int j = 0; j < 32 / VN; ++j) {
    float f[VN];
    unpack(r[j], f);
#pragma unroll
    for (int i = 0; i < VN; ++i) v[j * VN + i] += f[i];
  }
}

template <int ACT>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = act_value<ACT>(v[i]);
}

template <int KIND, int BN, bool GLU, bool PROMOTE, typename TI, typename TO>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ, const Params p) {
  using C = Cfg<KIND, BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kNBars);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
  int* prefix = abort_flag + 3;                   // [E + 1] row tiles before each expert
  int* scan = prefix + C::kPrefix;       // [kThreads / 32]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
  const uint32_t accf0 = smem_u32(bars + 2 * S), acce0 = smem_u32(bars + 2 * S + 2);
  const uint32_t drain = smem_u32(bars + 2 * S + 4);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 2);   // leader's: both producers arrive with their byte counts
      mbar_init(empty0 + 8 * s, 1);  // the leader's commit, multicast to the pair
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(accf0 + 8 * i, 1);
      mbar_init(acce0 + 8 * i, 2 * kEpiWarps);  // leader's: the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_holder), C::kTmem);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any remote operation targets them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  chain_wait();  // the set-up above touches no global memory

  int n_tiles;
  if (KIND == DW) {
    n_tiles = p.seg == nullptr || __ldg(p.plan) == 1 ? p.E * p.tiles_m * p.tiles_n : 0;
  } else if (p.seg == nullptr) {
    n_tiles = (int)((p.R + 2 * kBM - 1) / (2 * kBM)) * p.tiles_n * p.parts;
  } else {
    // each thread sums a run of experts; a scan over the threads gives the prefix
    const int per = (p.E + kThreads - 1) / kThreads, e0 = threadIdx.x * per, e1 = min(p.E, e0 + per);
    int sum = 0, ok = 1;
    for (int e = e0; e < e1; ++e) {
      const int a = __ldg(p.seg + e), b = __ldg(p.seg + e + 1);
      ok &= a <= b ? 1 : 0;
      sum += (b - a + 2 * kBM - 1) / (2 * kBM);
    }
    if (threadIdx.x == 0) ok &= __ldg(p.seg) == 0 && (int64_t)__ldg(p.seg + p.E) <= p.R ? 1 : 0;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    const bool valid = __syncthreads_and(ok) != 0;
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += scan[w];
    for (int e = e0; e < e1; ++e) {
      prefix[e] = run;
      run += (__ldg(p.seg + e + 1) - __ldg(p.seg + e) + 2 * kBM - 1) / (2 * kBM);
    }
    if (e0 < p.E && e1 == p.E) prefix[p.E] = run;
    __syncthreads();
    n_tiles = valid ? prefix[p.E] * p.tiles_n * p.parts : 0;
    if (!valid && threadIdx.x == 0) set_status(p.status, LRM_ERR_BAD_SEGMENTS);
  }

  const int rounds = (n_tiles + n_pairs - 1) / n_pairs;
  volatile int* abortv = abort_flag;
  const uint32_t full_lead = cluster_addr(full0, 0), acce_lead = cluster_addr(acce0, 0);

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer ----
    uint32_t it = 0, st = 0, sph = 0;
    bool ok = true;
    int last_e = -1;
    for (int i = 0, t; i < rounds && ok; ++i) {
      t = nth_tile(i, pair, n_pairs);
      if (t >= n_tiles) continue;  // (a last round may leave some pairs without one)
      const Tile d = decode<KIND, BN, GLU>(p, prefix, t, rank);
      const CUtensorMap *ma = &tmA, *mb = &tmB;
      if (KIND == DW && p.seg != nullptr) {
        ma = p.maps + d.e;
        mb = p.maps + p.E + d.e;
        if (d.e != last_e && d.slices > 0) {
          tensormap_acquire(ma);
          tensormap_acquire(mb);
          last_e = d.e;
        }
      }
      // first B row (FWD: rows of w, a SwiGLU pair stages gate rows and up rows) or column of this CTA
      const int nb = GLU ? d.n0 + rank * p.N : d.n0 + rank * (BN / 2);
      const uint32_t bytes = C::kBBytes + (d.has_rows ? kABytes : 0);
      const int planes = p.terms > 1 ? 3 : 1;
      int term = 6 - p.terms, kb = d.lo;
      if (d.lo > 0) {
        term += d.lo / d.slices;
        kb = d.lo % d.slices;
      }
      for (int k0 = d.lo; k0 < d.hi; k0 += C::kSub, ++it) {
        const uint32_t s = st, ph = sph;
        if (++st == (uint32_t)S) { st = 0; sph ^= 1u; }
        if (!mbar_wait_warp(empty0 + 8 * s, ph ^ 1u, abortv, p.status)) { ok = false; break; }
        const int n_sub = min(C::kSub, d.hi - k0);
        const uint32_t fb = full_lead + 8 * s;
        if (elect_one()) mbar_expect_tx_cluster(fb, n_sub * bytes);
        for (int j = 0; j < n_sub; ++j) {
          const int pa = plane_a(term), pb = plane_b(term), k = kb * kBK;
          const uint32_t a_dst = smem_u32(smem + s * C::kStage + j * C::kSlice), b_dst = a_dst + kABytes;
          if (elect_one()) {
            if (KIND == DW) {
              const int r = d.row0 + k;
              if (d.has_rows) load_columns<2>(a_dst, ma, d.m0, r, pa, p.one_box_a, fb);
              load_columns<BN / 128>(b_dst, mb, nb, r, pb, p.one_box_b, fb);
            } else {
              if (d.has_rows) tma_load_3d_pair(a_dst, ma, k, d.row0, pa, fb);
              const int eb = d.e * planes + pb;
              if (KIND == FWD) {
                tma_load_3d_pair(b_dst, mb, k, nb, eb, fb);
              } else {
                load_columns<BN / 128>(b_dst, mb, nb, k, eb, p.one_box_b, fb);
              }
            }
          }
          __syncwarp();
          if (++kb == d.slices) { kb = 0; ++term; }
        }
      }
    }
    // drain: every stage this warp filled has been consumed (so its data landed)
    const uint32_t first = it > (uint32_t)S ? it - S : 0u;
    for (uint32_t i = first; i < it; ++i) mbar_wait(empty0 + 8 * (i % S), (i / S) & 1u, abortv, p.status, false);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer ------
    if (leader) {
      constexpr uint32_t idesc = instr_desc<BN>(KIND == DW ? 1u : 0u, KIND == FWD ? 0u : 1u);
      const uint32_t a0 = smem_u32(smem), b0 = a0 + kABytes;
      const uint64_t adesc0 = KIND == DW ? smem_desc(a0, 8192, 1024) : smem_desc(a0, 16, 1024);
      const uint64_t bdesc0 = KIND == FWD ? smem_desc(b0, 16, 1024) : smem_desc(b0, 8192, 1024);
      constexpr uint64_t a_step = KIND == DW ? (2048 >> 4) : (32 >> 4);
      constexpr uint64_t b_step = KIND == FWD ? (32 >> 4) : (2048 >> 4);
      uint32_t st = 0, sph = 0, use = 0;  // operand stage and phase; accumulators used so far
      bool ok = true;
      for (int i = 0, t; i < rounds && ok; ++i) {
        t = nth_tile(i, pair, n_pairs);
        if (t >= n_tiles) continue;
        const Tile d = decode<KIND, BN, GLU>(p, prefix, t, 0);
        for (int k0 = d.lo; k0 < d.hi && ok; k0 += PROMOTE ? p.pk : d.hi, ++use) {
          const int k1 = PROMOTE ? min(d.hi, k0 + p.pk) : d.hi;
          const uint32_t acc = use & 1u;
          if (!mbar_wait_warp(acce0 + 8 * acc, ((use >> 1) & 1u) ^ 1u, abortv, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t tmem_d = tmem_base + acc * BN;
          for (int kb = k0; kb < k1; kb += C::kSub) {
            const uint32_t s = st, ph = sph;
            if (++st == (uint32_t)S) { st = 0; sph ^= 1u; }
            if (!mbar_wait_warp(full0 + 8 * s, ph, abortv, p.status)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < C::kSub; ++j) {
                if (j > 0 && kb + j >= k1) break;
                const uint64_t soff = (uint64_t)((s * C::kStage + j * C::kSlice) >> 4);
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                  mma_bf16(tmem_d, adesc0 + soff + kk * a_step, bdesc0 + soff + kk * b_step, idesc,
                           kb != k0 || j != 0 || kk != 0 ? 1u : 0u);
              }
              mma_commit_pair(empty0 + 8 * s);
            }
            __syncwarp();
          }
          if (ok && elect_one()) mma_commit_pair(accf0 + 8 * acc);
          __syncwarp();
        }
      }
      if (elect_one()) mma_commit_pair(drain);
    }
    __syncwarp();
    mbar_wait(drain, 0, abortv, p.status, false);  // all MMAs into this CTA's TMEM are done before it is freed
  } else {
    // ---------------------------------------------------------------- epilogue --------
    // a warp reads one 32-row quarter of TMEM and its group's half of the columns
    constexpr int GROUPS = kEpiWarps / 4;
    constexpr int NC = BN / GROUPS / 32;  // 32-column chunks of a warp (SwiGLU: the second half are up columns)
    constexpr int NO = GLU ? NC / 2 : NC;
    static_assert(NO > 0, "a warp needs a chunk of output columns");
    const int ew = warp - 2, q = warp & 3, group = ew >> 2;
    uint8_t* boxes = smem + C::kEpi + ew * C::kBoxes * kBoxBytes;
    Out<C::kBoxes> out{boxes, smem_u32(boxes), 0};
    constexpr int NR = 32 / VecTraits<TO>::N;  // 16-byte pieces of a chunk's row
    const int NP = GLU ? 2 * p.N : p.N;
    // TMEM column of chunk c
    auto tcol = [&](int c) {
      return GLU ? (c < NO ? (group * NO + c) * 32 : BN / 2 + (group * NO + c - NO) * 32) : (group * NC + c) * 32;
    };
    uint32_t use = 0;
    bool ok = true;
    for (int i = 0, t; i < rounds && ok; ++i) {
      t = nth_tile(i, pair, n_pairs);
      if (t >= n_tiles) continue;  // (a last round may leave some pairs without one)
      const Tile d = decode<KIND, BN, GLU>(p, prefix, t, rank);
      const int row_base = (KIND == DW ? d.m0 : d.row0) + q * 32;
      const int row_lim = KIND == DW ? p.M : d.row_end;
      // (the check, where it is on, covers what this warp's stores address: the expert, and its first and last row)
      const int nrows =
          d.has_rows && LRM_DCHECK(d.e >= 0 && d.e < p.E && row_base >= 0 && row_lim <= (KIND == DW ? p.M : p.R),
                                   p.status, LRM_ERR_BAD_INDEX)
              ? min(32, row_lim - row_base)
              : 0;
      // without segments the output map ends where the rows end, so TMA clips a partial block
      const bool whole = nrows == 32 || (nrows > 0 && (KIND == DW || p.seg == nullptr));
      const bool live = lane < nrows;
      const int64_t row = row_base + lane;
      const int n_first = d.n0 + group * NO * 32;
      const TO* res =
          KIND == FWD && p.residual != nullptr && live ? static_cast<const TO*>(p.residual) + row * p.N : nullptr;
      const int out_group = KIND == DW ? d.e : d.part;
      TO* y_row = static_cast<TO*>(p.y) + (out_group * (KIND == DW ? (int64_t)p.M : p.R) + row) * p.N;

      // the residual of chunk c (zeros past the last column)
      auto load_residual = [&](int c, uint4* r) {
        const int n = n_first + c * 32;
#pragma unroll
        for (int j = 0; j < NR; ++j)
          r[j] = res != nullptr && n + j * VecTraits<TO>::N < p.N
                     ? *reinterpret_cast<const uint4*>(res + n + j * VecTraits<TO>::N)
                     : make_uint4(0, 0, 0, 0);
      };
      // one chunk of 32 output columns: v holds the products (and u, for SwiGLU, the up columns')
      auto finish = [&](int c, float (&v)[32], float (&u)[32], const uint4* r) {
        const int n = n_first + c * 32;
        if (nrows <= 0 || n >= p.N) return;  // warp-uniform
        if (KIND == FWD) {
          if (p.bias != nullptr) {
            const TI* b = static_cast<const TI*>(p.bias) + (int64_t)d.e * NP;
            add_row(v, b, n, p.N);
            if (GLU) add_row(u, b + p.N, n, p.N);
          }
          if (p.z != nullptr) {
            TI* z_row = static_cast<TI*>(p.z) + row * NP;
            // (a bf16 z beside an fp32 y has no map of its own)
            const bool z_whole = whole && sizeof(TI) == sizeof(TO);
            const bool z_live = live || (whole && row < d.row_end);
            out.put(v, &tmZ, lane, n, p.N, row_base, 0, z_whole, z_live, z_row);
            if (GLU) out.put(u, &tmZ, lane, n, p.N, row_base, 1, z_whole, z_live, z_row + p.N);
          }
          if (GLU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = act_value<LRM_ACT_SWIGLU>(v[i]) * u[i];
          } else {
            switch (p.act) {
              case LRM_ACT_RELU: act32<LRM_ACT_RELU>(v); break;
              case LRM_ACT_GELU: act32<LRM_ACT_GELU>(v); break;
              case LRM_ACT_SILU: act32<LRM_ACT_SILU>(v); break;
              default: break;
            }
          }
          if (res != nullptr) add_vectors<TO>(v, r);
        }
        out.put(v, &tmY, lane, n, p.N, row_base, out_group, whole, live, y_row);
      };

      if (PROMOTE) {
        float acc[NC][32];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
        for (int k0 = d.lo; k0 < d.hi; k0 += p.pk, ++use) {
          const uint32_t a = use & 1u;
          if (!mbar_wait(accf0 + 8 * a, (use >> 1) & 1u, abortv, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t tbase = tmem_base + a * BN + ((uint32_t)(q * 32) << 16);
#pragma unroll
          for (int c = 0; c < 2 * NC; ++c) {
            uint32_t r[16];
            tmem_ld16(tbase + tcol(c / 2) + (c & 1) * 16, r);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c / 2][(c & 1) * 16 + i] += __uint_as_float(r[i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(acce_lead + 8 * a);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < NO; ++c) {
          uint4 r[NR];
          load_residual(c, r);
          finish(c, acc[c], acc[GLU ? NO + c : c], r);
        }
      } else {
        uint4 res_next[NR];  // loaded a chunk ahead, the first before the products are done
        load_residual(0, res_next);
        const uint32_t a = use & 1u;
        if (!mbar_wait(accf0 + 8 * a, (use >> 1) & 1u, abortv, p.status)) { ok = false; break; }
        ++use;
        tc_fence_after();
        const uint32_t tbase = tmem_base + a * BN + ((uint32_t)(q * 32) << 16);
        for (int c = 0; c < NO; ++c) {
          uint32_t r[32], w[32];
          uint4 res_now[NR];
#pragma unroll
          for (int j = 0; j < NR; ++j) res_now[j] = res_next[j];
          if (c + 1 < NO) load_residual(c + 1, res_next);
          tmem_ld32(tbase + tcol(c), r);
          if (GLU) tmem_ld32(tbase + tcol(NO + c), w);
          float v[32], u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            v[i] = __uint_as_float(r[i]);
            u[i] = GLU ? __uint_as_float(w[i]) : 0.f;
          }
          finish(c, v, u, res_now);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acce_lead + 8 * a);
      }
    }
    if (lane == 0) bulk_wait_all();  // stores complete before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no remote arrive may target a CTA that has exited
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmem);
  }
}

// DW with segments: plan[0] = 1 if they are valid, plan[1 ..] the experts by row count, longest first
// (ties by id), and the operand maps of every expert, the templates with their row extent (dimension
// 1) cut at the segment's end.
struct MapPair {
  CUtensorMap t[2];
};
__global__ void __launch_bounds__(1024) linear_plan_kernel(const int32_t* __restrict__ seg, int E, int64_t R,
                                                           int32_t* __restrict__ plan, CUtensorMap* __restrict__ maps,
                                                           const __grid_constant__ MapPair tpl,
                                                           int32_t* __restrict__ status) {
  chain_wait();
  __shared__ int s_rows[LRM_MAX_EXPERTS];
  const bool valid = rows_valid(seg, E, R, status);
  if (threadIdx.x == 0) plan[0] = valid ? 1 : 0;
  const int e = threadIdx.x;
  const int rows = e < E && valid ? seg[e + 1] - seg[e] : 0;
  if (e < E) s_rows[e] = rows;
  __syncthreads();
  if (e < E) {
    int before = 0;
    for (int j = 0; j < E; ++j) before += s_rows[j] > rows || (s_rows[j] == rows && j < e);
    if (LRM_DCHECK(before < E, status, LRM_ERR_BAD_INDEX)) plan[1 + before] = e;
  }
  for (int i = threadIdx.x; i < 2 * E; i += blockDim.x) {
    const int j = i / E, ee = i - j * E;
    const uint32_t end = valid ? (uint32_t)max(1, seg[ee + 1]) : 1u;
    uint4* dst = reinterpret_cast<uint4*>(maps + i);
    const uint4* src = reinterpret_cast<const uint4*>(&tpl.t[j]);
#pragma unroll
    for (int w = 0; w < 8; ++w) dst[w] = src[w];
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(
                     reinterpret_cast<uint64_t>(maps + i)),
                 "r"(end)
                 : "memory");
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
  }
}

// The segments cut into runs of at most `chunk` rows: vseg [EV + 1], a segmentation of the same rows whose first
// runs are those of expert 0 and so on (first_run [E + 1]); runs that are not needed are empty, at the end.  Segments
// that are not valid give none that is (vseg[0] = 1), so that the product computes nothing.
__global__ void __launch_bounds__(1024) cut_segments_kernel(const int32_t* __restrict__ seg, int E, int64_t R,
                                                            int chunk, int EV, int32_t* __restrict__ vseg,
                                                            int32_t* __restrict__ first_run,
                                                            int32_t* __restrict__ status) {
  chain_wait();
  __shared__ int s_seg[LRM_MAX_EXPERTS + 1];
  __shared__ int s_first[LRM_MAX_EXPERTS + 1];
  const bool valid = rows_valid(seg, E, R, status);
  for (int e = threadIdx.x; e <= E; e += blockDim.x) s_seg[e] = seg[e];
  __syncthreads();
  if (threadIdx.x == 0) {  // (this form is for products of few tiles, so of few experts)
    int run = 0;
    for (int e = 0; e < E; ++e) {
      s_first[e] = run;
      if (valid) run += (int)(((int64_t)s_seg[e + 1] - s_seg[e] + chunk - 1) / chunk);
    }
    s_first[E] = run;
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) first_run[e] = s_first[e];
  const int runs = s_first[E], end = s_seg[E];
  for (int v = threadIdx.x; v <= EV; v += blockDim.x) {
    int at = end;
    if (v < runs) {
      int lo = 0, hi = E;  // the expert of run v: the last e with first[e] <= v
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= v) lo = mid; else hi = mid;
      }
      at = s_seg[lo] + (v - s_first[lo]) * chunk;
    }
    if (!LRM_DCHECK(runs <= EV && at >= 0 && at <= end, status, LRM_ERR_BAD_INDEX)) at = end;
    vseg[v] = valid ? at : 1;
  }
}

// dw[e] = the sum of the expert's runs' weight gradients, in order (0 without a run).
__global__ void __launch_bounds__(256) sum_runs_kernel(const int32_t* __restrict__ vseg,
                                                       const int32_t* __restrict__ first_run,
                                                       const float* __restrict__ part, int64_t n,
                                                       float* __restrict__ out) {
  chain_wait();
  if (vseg[0] != 0) return;  // (recorded by cut_segments_kernel)
  const int e = blockIdx.y, r0 = first_run[e], r1 = first_run[e + 1];
  const int64_t step = (int64_t)gridDim.x * blockDim.x * 4;
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4; i < n; i += step) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      float f[4];
      unpack(ld_stream16(part + r * n + i), f);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] += f[q];
    }
    st16(out + e * n + i, pack(acc));
  }
}

// fp32 tensors [groups][rows][cols] as three bf16 planes [groups][3][rows][pitch] whose sum is the tensor to
// 24 bits.  A value that is not finite stays in the first plane alone, so that no infinity is subtracted
// from itself; one that bf16 would round to infinity is cut instead.  The pitch is a multiple of 64: rows
// that do not start on a 128-byte line cost TMA two lines for one.
struct Split {
  const float* x;
  int64_t groups, rows, cols, pitch;
  __nv_bfloat16* out;
};
struct Splits {
  Split t[3];
  int count;
};
__global__ void __launch_bounds__(256) split_planes_kernel(const __grid_constant__ Splits a) {
  chain_wait();
  for (int k = 0; k < a.count; ++k) {
    const Split& s = a.t[k];
    const int64_t nv = s.cols / 8, total = s.groups * s.rows * nv;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
      const int64_t row = i / nv, g = row / s.rows;
      const uint4 lo = ld_stream16_now(s.x + i * 8), hi = ld_stream16_now(s.x + i * 8 + 4);
      float a4[4], b4[4], p[3][8];
      unpack(lo, a4);
      unpack(hi, b4);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float v = q < 4 ? a4[q & 3] : b4[q & 3];
        p[0][q] = __bfloat162float(__float2bfloat16_rn(v));
        if (isinf(p[0][q])) p[0][q] = __bfloat162float(__float2bfloat16_rz(v));
        const float r1 = isfinite(v) ? v - p[0][q] : 0.f;  // exact
        p[1][q] = __bfloat162float(__float2bfloat16_rn(r1));
        p[2][q] = r1 - p[1][q];
      }
#pragma unroll
      for (int j = 0; j < 3; ++j)
        st16(s.out + ((g * 2 + j) * s.rows + row) * s.pitch + (i - row * nv) * 8, pack(p[j]));
    }
  }
}

// bf16 rows [rows][cols] copied to rows `pitch` apart.
__global__ void __launch_bounds__(256) repitch_kernel(const __nv_bfloat16* __restrict__ in, int64_t rows, int64_t cols,
                                                      int64_t pitch, __nv_bfloat16* __restrict__ out) {
  chain_wait();
  const int64_t nv = cols / 8, total = rows * nv;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / nv;
    st16(out + r * pitch + (i - r * nv) * 8, ld_stream16(in + i * 8));
  }
}

// out = the sum of `parts` arrays of n floats (a multiple of 4), in order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ part, int parts, int64_t n,
                                                        float* __restrict__ out) {
  chain_wait();
  const int64_t step = (int64_t)gridDim.x * blockDim.x * 4;
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4; i < n; i += step) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < parts; ++s) {
      float f[4];
      unpack(ld_stream16(part + s * n + i), f);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] += f[q];
    }
    st16(out + i, pack(acc));
  }
}

// The products' parts [parts][R][NP] added in order, with the epilogue of lrm_linear (DX: none): a CTA per row,
// 8 columns a thread.
template <typename TI, typename TO>
__global__ void __launch_bounds__(128) finish_parts_kernel(const int32_t* __restrict__ seg, int E, int64_t R, int N,
                                                           const float* __restrict__ part, int parts, int act,
                                                           const TI* __restrict__ bias, const TO* __restrict__ residual,
                                                           TO* __restrict__ y, TI* __restrict__ z) {
  chain_wait();
  const bool glu = act == LRM_ACT_SWIGLU;
  const int NP = glu ? 2 * N : N;
  const int64_t row = blockIdx.x;
  int e = 0;
  if (seg != nullptr) {
    if (!rows_valid(seg, E, R, nullptr) || row >= seg[E]) return;  // (recorded by the products)
    int lo = 0, hi = E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seg[mid] <= row) lo = mid; else hi = mid;
    }
    e = lo;
  }
  auto sum8 = [&](int col, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float* at = part + ((int64_t)s * R + row) * NP + col;
      float a[4], b[4];
      unpack(ldg16(at), a);
      unpack(ldg16(at + 4), b);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[q] += a[q];
        v[4 + q] += b[q];
      }
    }
    if (bias != nullptr)
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += to_f(bias[(int64_t)e * NP + col + q]);
    if (z != nullptr)
#pragma unroll
      for (int q = 0; q < 8; ++q) z[row * NP + col + q] = from_f<TI>(v[q]);
  };
  for (int c = threadIdx.x * 8; c < N; c += blockDim.x * 8) {
    float v[8], u[8];
    sum8(c, v);
    if (glu) sum8(N + c, u);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (glu) {
        v[q] = act_value<LRM_ACT_SWIGLU>(v[q]) * u[q];
      } else {
        switch (act) {
          case LRM_ACT_RELU: v[q] = act_value<LRM_ACT_RELU>(v[q]); break;
          case LRM_ACT_GELU: v[q] = act_value<LRM_ACT_GELU>(v[q]); break;
          case LRM_ACT_SILU: v[q] = act_value<LRM_ACT_SILU>(v[q]); break;
          default: break;
        }
      }
      if (residual != nullptr) v[q] += to_f(residual[row * N + c + q]);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) y[row * N + c + q] = from_f<TO>(v[q]);
  }
}

// ---------------------------------------------------------------- host side ----------
// [d2][d1][d0] of 2- or 4-byte elements, d0 contiguous (a multiple of 16 bytes), with a {b0, b1, 1} box.
bool make_map(CUtensorMap* m, const void* base, bool f32, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1,
              uint64_t stride2, uint32_t b0, uint32_t b1, bool operand) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {b0, b1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     operand ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     operand ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A bf16 operand [planes][rows][cols], its rows `pitch` apart.
bool operand_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t pitch, uint64_t rows, uint64_t planes,
                 uint32_t box_rows) {
  return make_map(m, base, false, cols, rows, planes, pitch * 2, rows * pitch * 2, 64, box_rows, true);
}
// The same seen as [planes][pitch / 64][rows][64], `blocks` blocks of 64 columns and 64 rows a box; the plain
// form with one block where the pitch does not divide (*one_box tells).
bool column_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t pitch, uint64_t rows, uint64_t planes,
                uint32_t blocks, bool* one_box) {
  *one_box = pitch % 64 == 0 && pitch >= 64 * blocks;
  if (!*one_box) return operand_map(m, base, cols, pitch, rows, planes, 64);
  const cuuint64_t dims[4] = {64, rows, pitch / 64, planes};
  const cuuint64_t strides[3] = {pitch * 2, 128, rows * pitch * 2};
  const cuuint32_t box[4] = {64, 64, blocks, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// An output [groups][rows][cols] in 32-row boxes of 64 bytes; halves: [rows][2][cols] seen as two groups.
bool output_map(CUtensorMap* m, const void* base, bool f32, uint64_t cols, uint64_t rows, uint64_t groups,
                bool halves = false) {
  const uint64_t b = f32 ? 4 : 2, line = cols * b * (halves ? 2 : 1);
  return make_map(m, base, f32, cols, rows, groups, line, halves ? cols * b : rows * line, f32 ? 16 : 32, 32, false);
}

template <int KIND, int BN, bool GLU, bool PROMOTE, typename TI, typename TO>
lrm_status launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& y, const CUtensorMap& z,
                  const Params& p, int64_t tiles_bound, cudaStream_t s) {
  constexpr auto kernel = linear_tc_kernel<KIND, BN, GLU, PROMOTE, TI, TO>;
  using C = Cfg<KIND, BN>;
  const size_t smem = C::smem();
  if (ensure_max_smem<kernel>((int)smem) != cudaSuccess) return LRM_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;  // the occupancy query sees the cluster shape only
  static int resident[kDeviceSlots] = {};  // CTA pairs, per device
  const int slot = current_device_slot();
  int pairs = slot >= 0 ? resident[slot] : 0;
  if (pairs == 0) {
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs <= 0) pairs = sm_count() / 2;
    if (slot >= 0) resident[slot] = pairs;
  }
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(2 * (tiles_bound < pairs ? tiles_bound : pairs)));
  if (cudaLaunchKernelEx(&cfg, kernel, a, b, y, z, p) != cudaSuccess) return LRM_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? LRM_OK : LRM_ERR_CUDA;
}

uint64_t plane_pitch(uint64_t cols) { return (cols + 63) / 64 * 64; }

void add_split(Splits& a, const void* x, int64_t groups, int64_t rows, int64_t cols, void* out) {
  a.t[a.count++] = Split{static_cast<const float*>(x), groups, rows, cols, (int64_t)plane_pitch((uint64_t)cols),
                         static_cast<__nv_bfloat16*>(out)};
}
void launch_splits(const Splits& a, cudaStream_t s) {
  int64_t blocks = 1;
  for (int k = 0; k < a.count; ++k) {
    const int64_t n = (a.t[k].groups * a.t[k].rows * a.t[k].cols / 8 + 255) / 256;
    blocks = n > blocks ? n : blocks;
  }
  launch_chained(split_planes_kernel, dim3((unsigned)(blocks < 1216 ? blocks : 1216)), dim3(256), 0, s, a);
}

// K slices per accumulator where the result is fp32: 256 products for split fp32 inputs (2.4e-7 off against
// 64 bits, as fp32 arithmetic itself), 512 for bf16 inputs (4.7e-7; 1024 products: 9.9e-7).
constexpr int kSlicesF32 = 4, kSlicesBf16 = 8;
// bf16 results of longer sums leave TMEM like fp32 ones: sums of one sign are 4e-4 off after 65536 products and 1.6e-3
// after 262144, near half a bf16 unit (8192 x 4096 x 65600: 2291 us, 2220 us in one accumulator).
constexpr int kLongSum = 65536;

// Most row tiles there can be, and about how many (every segment ends in half a tile).
int64_t row_tiles(const int32_t* seg, int64_t R, int E) {
  return (R + 2 * kBM - 1) / (2 * kBM) + (seg != nullptr ? E : 0);
}
int64_t likely_row_tiles(const int32_t* seg, int64_t R, int E) {
  return (R + 2 * kBM - 1) / (2 * kBM) + (seg != nullptr ? (R < E ? R : E) / 2 : 0);
}

// How a product is cut where its tiles are few and its reduction long (with fp32 inputs six terms make it six
// times as long): tile width and parts of the reduction by the least time, in units of 0.05 us.  A
// slice takes 3 units (5 in the 256-column tile); adding the parts up, by a launch and a pass, is worth 130
// (fp32 128 x 128 x 2048 12.8 us in parts, 37 us without; bf16 64 x 4096 x 4096 22.9 us in parts, 15.9 us
// without, and left whole by this).
struct Cut {
  int bn, parts, len;
};
Cut cut_product(int64_t R, int32_t E, int64_t cols, int total, int least) {
  const int64_t tm = (R + 2 * kBM - 1) / (2 * kBM) + (E > 1 ? (R < E ? R : E) / 2 : 0);
  Cut best{least, 1, total};
  if (R <= 0) return best;  // no tiles at all (the size functions ask)
  int64_t best_time = INT64_MAX;
  for (int bn = least; bn <= 256; bn *= 2) {
    const int64_t base = tm * ((cols + bn - 1) / bn);
    int64_t parts = kPairs / base;
    if (parts > total / 16) parts = total / 16;
    for (int64_t n : {(int64_t)1, parts}) {
      if (n < 1) continue;
      const int64_t len = ((total + n - 1) / n + 7) / 8 * 8, used = (total + len - 1) / len;
      const int64_t waves = (base * used + kPairs - 1) / kPairs;
      const int64_t time = waves * (n == 1 ? total : len) * (bn == 256 ? 5 : 3) + (used > 1 ? 130 : 0);
      if (time < best_time) {
        best_time = time;
        best = Cut{bn, (int)used, used > 1 ? (int)len : total};
      }
    }
  }
  return best;
}
// bf16 weights whose rows start off the 32-byte sectors (K an odd multiple of 8) are copied to 128-byte rows
// first where they serve many rows: with x off the sectors too, TMA reads five sectors for four of both
// operands.  32768 x 4096 x 4072: 615 us with the copy, 780 us without; 8192 x 2048 x 2040: 49 and 58 us.
// (x copied as well: 686 and 57 us.)
bool repitch_weights(int64_t R, int32_t E, int32_t K, lrm_dtype dt) {
  return dt == LRM_BF16 && K % 16 != 0 && R >= 4096 * (int64_t)E;
}
int slices_of(int64_t red, lrm_dtype dt) { return (int)((red + kBK - 1) / kBK) * (dt == LRM_F32 ? 6 : 1); }

// Runs of rows for the weight gradient per expert where a popular expert's tiles would run long after the others
// (taken to have three times its share of the rows): run length and the most runs there can be, 0 for none.
// Times in us: a slice 0.155, the rows' products over all CTA pairs; 12 for two launches and the adding up.
struct Runs {
  int chunk, count;
};
Runs cut_rows(int64_t R, int32_t E, int64_t N, int64_t K, lrm_dtype dt) {
  const double slice = 0.155 * (dt == LRM_F32 ? 6 : 1) / kBK;  // per row
  const double tiles = (double)((N + 255) / 256) * (double)((K + 127) / 128);
  const double longest = slice * (double)(3 * R / E < R ? 3 * R / E : R), even = slice * (double)R * tiles / kPairs;
  double want = (even > 8 ? even / 2 : 4) / slice;  // rows of a run
  if (want < 256) want = 256;
  const int chunk = (int)(((int64_t)want + kBK - 1) / kBK * kBK);
  const int64_t count = (R + chunk - 1) / chunk + E;
  const double adding = 12 + 8.0 * (double)count * (double)N * (double)K / 6.8e6;
  if (count > LRM_MAX_EXPERTS || longest < even + adding) return Runs{0, 0};
  return Runs{chunk, (int)count};
}

// Tile width by the waves of tiles over the CTA pairs: a K slice of a 256-column tile takes 0.26 us (its
// products), one of a 128- or 64-column tile 0.155 us (the operands' way in).  On a tie the narrower: more
// SMs then share the reading of the weights.
template <typename F>
lrm_status with_width(int64_t tiles_m, int N, int least, F&& f) {
  const int64_t pairs = sm_count() / 2;
  auto cost = [&](int bn, int slice) { return (tiles_m * ((N + bn - 1) / bn) + pairs - 1) / pairs * slice; };
  const int64_t c256 = cost(256, 5), c128 = cost(128, 3), c64 = least > 64 ? INT64_MAX : cost(64, 3);
  if (c64 <= c128 && c64 <= c256) return f(IntTag<64>{});
  return c128 <= c256 ? f(IntTag<128>{}) : f(IntTag<256>{});
}

}  // namespace

size_t linear_planes_bytes(int64_t rows, int64_t cols) { return (size_t)rows * plane_pitch((uint64_t)cols) * 6; }

lrm_status launch_linear_tc(const LinearArgs& a, lrm_dtype dt, lrm_dtype out_dt, void* ws, cudaStream_t s) {
  if (!device_ok() || encode_fn() == nullptr) return LRM_ERR_UNSUPPORTED;
  using B16 = __nv_bfloat16;
  const bool f32 = dt == LRM_F32, glu = a.act == LRM_ACT_SWIGLU;
  const int NP = glu ? 2 * a.N : a.N;
  const void *xs = a.x, *wsrc = a.w;
  void* parts_ws = ws;
  if (f32) {
    char* b = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 127) & ~uintptr_t(127));
    Splits sp{};
    add_split(sp, a.x, 1, a.R, a.K, b);
    xs = b;
    b += (linear_planes_bytes(a.R, a.K) + 255) / 256 * 256;
    add_split(sp, a.w, a.E, NP, a.K, b);
    wsrc = b;
    parts_ws = b + (linear_planes_bytes((int64_t)a.E * NP, a.K) + 255) / 256 * 256;
    launch_splits(sp, s);
  }
  Params p{};
  p.E = a.E;
  p.R = a.R;
  p.N = a.N;
  p.red = a.K;
  p.terms = f32 ? 6 : 1;
  p.pk = f32 ? kSlicesF32 : kSlicesBf16;
  p.seg = a.seg_offsets;
  p.act = a.act;
  p.bias = a.bias;
  p.residual = a.residual;
  p.y = a.y;
  p.z = a.z;
  p.status = a.status;
  const int planes = f32 ? 3 : 1;
  uint64_t pitch = f32 ? plane_pitch(a.K) : a.K, pitch_w = pitch;
  const bool y32 = out_dt == LRM_F32;
  CUtensorMap mA, mB, mY, mZ;
  if (!operand_map(&mA, xs, a.K, pitch, a.R, planes, kBM) || !output_map(&mY, a.y, y32, a.N, a.R, 1))
    return LRM_ERR_CUDA;
  mZ = mY;
  if (a.z != nullptr && y32 == f32 && !output_map(&mZ, a.z, f32, a.N, a.R, glu ? 2 : 1, glu)) return LRM_ERR_CUDA;
  const int64_t tm = row_tiles(a.seg_offsets, a.R, a.E);
  auto go = [&](auto bn, auto glu_tag) {
    constexpr int BN = decltype(bn)::value;
    constexpr bool GLU = decltype(glu_tag)::value != 0;
    if constexpr (GLU && BN < 128) {
      return LRM_ERR_UNSUPPORTED;
    } else {
      constexpr int cols = GLU ? BN / 2 : BN;
      p.tiles_n = (a.N + cols - 1) / cols;
      if (!operand_map(&mB, wsrc, a.K, pitch_w, NP, (uint64_t)a.E * planes, BN / 2)) return LRM_ERR_CUDA;
      if (f32) return launch<FWD, BN, GLU, true, float, float>(mA, mB, mY, mZ, p, tm * p.tiles_n, s);
      if (y32) return launch<FWD, BN, GLU, true, B16, float>(mA, mB, mY, mZ, p, tm * p.tiles_n, s);
      if (a.K > kLongSum) return launch<FWD, BN, GLU, true, B16, B16>(mA, mB, mY, mZ, p, tm * p.tiles_n, s);
      return launch<FWD, BN, GLU, false, B16, B16>(mA, mB, mY, mZ, p, tm * p.tiles_n, s);
    }
  };
  p.parts = 1;
  p.part_len = slices_of(a.K, dt);
  const Cut cut = parts_ws != nullptr ? cut_product(a.R, a.E, NP, p.part_len, 64) : Cut{0, 1, p.part_len};
  if (cut.parts > 1) {
    float* part = static_cast<float*>(parts_ws);
    Params raw = p;  // the products alone, over all columns of w
    raw.N = NP;
    raw.act = LRM_ACT_NONE;
    raw.bias = raw.residual = raw.z = nullptr;
    raw.y = part;
    raw.parts = cut.parts;
    raw.part_len = cut.len;
    raw.tiles_n = (NP + cut.bn - 1) / cut.bn;
    if (!operand_map(&mB, wsrc, a.K, pitch_w, NP, (uint64_t)a.E * planes, cut.bn / 2) ||
        !output_map(&mY, part, true, NP, a.R, cut.parts))
      return LRM_ERR_CUDA;
    const int64_t tiles = tm * raw.tiles_n * cut.parts;
    auto products = [&](auto bn) {
      constexpr int BN = decltype(bn)::value;
      return f32 ? launch<FWD, BN, false, true, float, float>(mA, mB, mY, mY, raw, tiles, s)
                 : launch<FWD, BN, false, true, B16, float>(mA, mB, mY, mY, raw, tiles, s);
    };
    const lrm_status st = cut.bn == 256   ? products(IntTag<256>{})
                          : cut.bn == 128 ? products(IntTag<128>{})
                                          : products(IntTag<64>{});
    if (st) return st;
    auto finish = [&](auto kernel, auto* y, auto* z) {
      using TO = std::remove_pointer_t<decltype(y)>;
      using TI = std::remove_pointer_t<decltype(z)>;
      launch_chained(kernel, dim3((unsigned)a.R), dim3(128), 0, s, a.seg_offsets, a.E, a.R, a.N, (const float*)part,
                     cut.parts, (int)a.act, (const TI*)a.bias, (const TO*)a.residual, y, z);
    };
    if (f32)
      finish(finish_parts_kernel<float, float>, static_cast<float*>(a.y), static_cast<float*>(a.z));
    else if (y32)
      finish(finish_parts_kernel<B16, float>, static_cast<float*>(a.y), static_cast<B16*>(a.z));
    else
      finish(finish_parts_kernel<B16, B16>, static_cast<B16*>(a.y), static_cast<B16*>(a.z));
    return cudaGetLastError() == cudaSuccess ? LRM_OK : LRM_ERR_CUDA;
  }
  if (parts_ws != nullptr && repitch_weights(a.R, a.E, a.K, dt)) {
    B16* wp = static_cast<B16*>(parts_ws);
    pitch_w = plane_pitch(a.K);
    const int64_t rows = (int64_t)a.E * NP, blocks = (rows * (a.K / 8) + 255) / 256;
    launch_chained(repitch_kernel, dim3((unsigned)(blocks < 1216 ? blocks : 1216)), dim3(256), 0, s,
                   static_cast<const B16*>(a.w), rows, (int64_t)a.K, (int64_t)pitch_w, wp);
    wsrc = wp;
  }
  const int64_t likely = likely_row_tiles(a.seg_offsets, a.R, a.E);
  if (glu) return with_width(likely, NP, 128, [&](auto bn) { return go(bn, IntTag<1>{}); });
  return with_width(likely, NP, 64, [&](auto bn) { return go(bn, IntTag<0>{}); });
}

lrm_status launch_linear_backward_tc(const LinearGradArgs& a, lrm_dtype dt, void* ws, cudaStream_t s) {
  if (!device_ok() || encode_fn() == nullptr) return LRM_ERR_UNSUPPORTED;
  using B16 = __nv_bfloat16;
  const bool f32 = dt == LRM_F32;
  const int planes = f32 ? 3 : 1;
  const void *dzs = a.dz, *xs = a.x, *wsrc = a.w;
  // scratch: the expert maps of DW (128-byte aligned) and its plan, then the planes
  char* b = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 127) & ~uintptr_t(127));
  const bool by_segment = a.dw != nullptr && a.seg_offsets != nullptr;
  const int segments = by_segment ? linear_grad_segments(a.R, a.E, a.N, a.K, dt) : 0;
  CUtensorMap* maps = reinterpret_cast<CUtensorMap*>(b);
  int32_t* plan = reinterpret_cast<int32_t*>(b + 2 * sizeof(CUtensorMap) * (size_t)segments);
  b += linear_plan_bytes(segments);
  Splits sp{};
  auto split = [&](const void* src, int64_t groups, int64_t rows, int64_t cols) {
    add_split(sp, src, groups, rows, cols, b);
    const void* at = b;
    b += (linear_planes_bytes(groups * rows, cols) + 255) / 256 * 256;
    return at;
  };
  if (f32) {
    dzs = split(a.dz, 1, a.R, a.N);
    if (a.dx != nullptr) wsrc = split(a.w, a.E, a.N, a.K);
    if (a.dw != nullptr) xs = split(a.x, 1, a.R, a.K);
    launch_splits(sp, s);
  }
  const uint64_t pitch_n = f32 ? plane_pitch(a.N) : a.N, pitch_k = f32 ? plane_pitch(a.K) : a.K;
  Params p{};
  p.E = a.E;
  p.R = a.R;
  p.N = a.K;
  p.terms = f32 ? 6 : 1;
  p.pk = f32 ? kSlicesF32 : kSlicesBf16;
  p.seg = a.seg_offsets;
  p.status = a.status;
  CUtensorMap mA, mB, mY;
  if (a.dw != nullptr) {
    p.M = a.N;
    p.parts = 1;
    p.tiles_m = (a.N + 2 * kBM - 1) / (2 * kBM);
    const int parts = a.seg_offsets == nullptr ? linear_grad_parts(a.R, a.N, a.K) : 1;
    const Runs runs = a.seg_offsets == nullptr ? Runs{0, 0} : cut_rows(a.R, a.E, a.N, a.K, dt);
    const int32_t* seg = a.seg_offsets;
    int32_t *vseg = nullptr, *first_run = nullptr;
    if (runs.count > 0) {
      vseg = reinterpret_cast<int32_t*>(b);
      first_run = vseg + runs.count + 1;
      b += (sizeof(int32_t) * ((size_t)runs.count + a.E + 2) + 255) / 256 * 256;
      launch_chained(cut_segments_kernel, dim3(1), dim3(1024), 0, s, a.seg_offsets, a.E, a.R, runs.chunk, runs.count,
                     vseg, first_run, a.status);
      seg = vseg;
      p.seg = vseg;
      p.E = runs.count;
    }
    float* sums = parts > 1 || runs.count > 0 ? reinterpret_cast<float*>(b) : a.dw;
    p.y = sums;
    if (a.seg_offsets == nullptr) {
      p.E = parts;
      p.part_rows = (int)((a.R + (int64_t)parts * kBK - 1) / ((int64_t)parts * kBK) * kBK);
    }
    if (!column_map(&mA, dzs, a.N, pitch_n, a.R, planes, 2, &p.one_box_a) ||
        !output_map(&mY, sums, true, a.K, a.N, p.E))
      return LRM_ERR_CUDA;
    const int64_t tm = (int64_t)p.E * p.tiles_m;
    const lrm_status st = with_width(tm, a.K, 128, [&](auto bn) {
      constexpr int BN = decltype(bn)::value;
      if constexpr (BN < 128) {
        return LRM_ERR_UNSUPPORTED;
      } else {
        p.tiles_n = (a.K + BN - 1) / BN;
        if (!column_map(&mB, xs, a.K, pitch_k, a.R, planes, BN / 128, &p.one_box_b)) return LRM_ERR_CUDA;
        if (a.seg_offsets != nullptr) {
          const MapPair tpl{{mA, mB}};
          launch_chained(linear_plan_kernel, dim3(1), dim3(1024), 0, s, seg, p.E, a.R, plan, maps, tpl, a.status);
          p.plan = plan;
          p.maps = maps;
        }
        return launch<DW, BN, false, true, B16, float>(mA, mB, mY, mY, p, tm * p.tiles_n, s);
      }
    });
    if (st) return st;
    if (runs.count > 0) {
      b += (sizeof(float) * (size_t)runs.count * a.N * a.K + 255) / 256 * 256;
      const int64_t n = (int64_t)a.N * a.K, blocks = (n / 4 + 255) / 256;
      launch_chained(sum_runs_kernel, dim3((unsigned)(blocks < 304 ? blocks : 304), (unsigned)a.E), dim3(256), 0, s,
                     (const int32_t*)vseg, (const int32_t*)first_run, (const float*)sums, n, a.dw);
    }
    if (parts > 1) {
      b += (sizeof(float) * (size_t)parts * a.N * a.K + 255) / 256 * 256;
      const int64_t n = (int64_t)a.N * a.K, blocks = (n / 4 + 255) / 256;
      launch_chained(sum_parts_kernel, dim3((unsigned)(blocks < 1216 ? blocks : 1216)), dim3(256), 0, s,
                     (const float*)sums, parts, n, a.dw);
    }
  }
  if (a.dx != nullptr) {
    p.E = a.E;
    p.seg = a.seg_offsets;
    p.red = a.N;
    const Cut cut = cut_product(a.R, a.E, a.K, slices_of(a.N, dt), 128);
    p.parts = cut.parts;
    p.part_len = cut.len;
    float* part = reinterpret_cast<float*>(b);
    p.y = cut.parts > 1 ? part : a.dx;
    if (!operand_map(&mA, dzs, a.N, pitch_n, a.R, planes, kBM) ||
        !output_map(&mY, p.y, f32 || cut.parts > 1, a.K, a.R, cut.parts))
      return LRM_ERR_CUDA;
    const int64_t tm = row_tiles(a.seg_offsets, a.R, a.E);
    if (cut.parts > 1) {
      p.tiles_n = (a.K + cut.bn - 1) / cut.bn;
      if (!column_map(&mB, wsrc, a.K, pitch_k, a.N, (uint64_t)a.E * planes, cut.bn / 128, &p.one_box_b))
        return LRM_ERR_CUDA;
      const int64_t tiles = tm * p.tiles_n * cut.parts;
      const lrm_status st =
          f32 ? (cut.bn == 256 ? launch<DX, 256, false, true, float, float>(mA, mB, mY, mY, p, tiles, s)
                               : launch<DX, 128, false, true, float, float>(mA, mB, mY, mY, p, tiles, s))
              : (cut.bn == 256 ? launch<DX, 256, false, true, B16, float>(mA, mB, mY, mY, p, tiles, s)
                               : launch<DX, 128, false, true, B16, float>(mA, mB, mY, mY, p, tiles, s));
      if (st) return st;
      auto finish = [&](auto kernel, auto* out) {
        using T = std::remove_pointer_t<decltype(out)>;
        launch_chained(kernel, dim3((unsigned)a.R), dim3(128), 0, s, a.seg_offsets, a.E, a.R, a.K, (const float*)part,
                       cut.parts, (int)LRM_ACT_NONE, (const T*)nullptr, (const T*)nullptr, out, (T*)nullptr);
      };
      if (f32)
        finish(finish_parts_kernel<float, float>, static_cast<float*>(a.dx));
      else
        finish(finish_parts_kernel<B16, B16>, static_cast<B16*>(a.dx));
      return cudaGetLastError() == cudaSuccess ? LRM_OK : LRM_ERR_CUDA;
    }
    return with_width(likely_row_tiles(a.seg_offsets, a.R, a.E), a.K, 128, [&](auto bn) {
      constexpr int BN = decltype(bn)::value;
      if constexpr (BN < 128) {
        return LRM_ERR_UNSUPPORTED;
      } else {
        p.tiles_n = (a.K + BN - 1) / BN;
        if (!column_map(&mB, wsrc, a.K, pitch_k, a.N, (uint64_t)a.E * planes, BN / 128, &p.one_box_b))
          return LRM_ERR_CUDA;
        if (f32) return launch<DX, BN, false, true, float, float>(mA, mB, mY, mY, p, tm * p.tiles_n, s);
        if (a.N > kLongSum) return launch<DX, BN, false, true, B16, B16>(mA, mB, mY, mY, p, tm * p.tiles_n, s);
        return launch<DX, BN, false, false, B16, B16>(mA, mB, mY, mY, p, tm * p.tiles_n, s);
      }
    });
  }
  return LRM_OK;
}

// Parts of the rows that the dense weight gradient sums apart where its tiles alone would leave most of the
// 76 CTA pairs idle; at least 1024 rows each.
int linear_grad_parts(int64_t R, int32_t N, int32_t K) {
  const int64_t tiles = (int64_t)((N + 255) / 256) * ((K + 127) / 128);
  int64_t parts = 76 / tiles;
  if (parts > R / 1024) parts = R / 1024;
  return parts < 1 ? 1 : (int)parts;
}

size_t linear_extra_bytes(int64_t R, int32_t E, int32_t NP, int32_t K, lrm_dtype dt) {
  const int parts = cut_product(R, E, NP, slices_of(K, dt), 64).parts;
  if (parts > 1) return sizeof(float) * (size_t)parts * R * NP;
  return repitch_weights(R, E, K, dt) ? 2 * (size_t)E * NP * plane_pitch((uint64_t)K) : 0;
}
size_t linear_grad_parts_bytes(int64_t R, int32_t E, int32_t N, int32_t K, lrm_dtype dt) {
  const int parts = cut_product(R, E, K, slices_of(N, dt), 128).parts;
  return parts > 1 ? sizeof(float) * (size_t)parts * R * K : 0;
}

int linear_grad_segments(int64_t R, int32_t E, int32_t N, int32_t K, lrm_dtype dt) {
  const int runs = cut_rows(R, E, N, K, dt).count;
  return runs > E ? runs : E;
}
size_t linear_grad_runs_bytes(int64_t R, int32_t E, int32_t N, int32_t K, lrm_dtype dt) {
  const int runs = cut_rows(R, E, N, K, dt).count;
  return runs > 0 ? 512 + sizeof(int32_t) * ((size_t)runs + E + 2) + sizeof(float) * (size_t)runs * N * K : 0;
}

size_t linear_plan_bytes(int32_t E) {
  return (2 * sizeof(CUtensorMap) * (size_t)E + sizeof(int32_t) * ((size_t)E + 1) + 255) / 256 * 256;
}

}  // namespace lrm
