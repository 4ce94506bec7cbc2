// lrm_fp8_linear and lrm_fp8_linear_backward on the tensor cores of sm_103a (tcgen05 kind::f8f6f4, TMEM, TMA).
//
//   FWD  y  = act(sum over blocks b of 128 k: sx[r,b] sw[n/128,b] (x_b w_b^T) + bias) + residual
//   DX   dx = sum over blocks b of 128 n: sz[r,b] sw[b,k/128] (dz_b w_b)
//
// The scales change with every 128 steps of the reduction, so the products of a block are a sum of their own: each K
// slice of 128 (one stage of operands, four MMAs of K = 32) goes to the next of the accumulators that TMEM holds, and
// the epilogue warps take it out, scale it by row and block and add it up in fp32 registers while the tensor core is
// at the next.
//
// CTA pairs and tiles are those of linear_tc.cu: 256 x BN tiles over a persistent grid.  Warp 0 issues the TMA loads,
// warp 1 of the leader the MMAs, warps 2 and 3 bring the tile's place and its scales to shared memory (segment bounds
// and scales are trips to memory that the epilogue would wait for), the rest are the epilogue: each has a 32-row
// quarter of TMEM by 64 columns (SwiGLU: 32 gate columns and the 32 up columns that go with them), which lie in one
// block of 128 columns of W.
//
// A 256-column slice costs the tensor core 557 cycles and the 16 epilogue warps' loads and sums 300 (one multiply-add
// an element and slice, two an instruction), but 830 in all: TMEM holds two accumulators, so that a slice's products
// wait until all 32 warps of the pair have taken out the one before the last, and the signals both ways are as long as
// the sums.  Four accumulators of 128 columns each bring half as many products for three quarters of the operands
// (bound by L2: 0.25 us a slice, 256 columns 0.43 us); eight epilogue warps of 128 columns hide less.
// GB300: 32768 x 4096 x 4096 412 us (2.7 PFLOP/s), with bias, GELU and residual 514 us; 65536 rows over 128 experts to
// 2 x 768, K = 2048, SwiGLU 244 us (with z 281 us), its rows' gradient 266 us, 768 to 2048 180 us.
//
// W stays as it was quantised: FWD reads its rows K-major, DX the same bytes with the columns contiguous (MN-major).
#include "fp8.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "tc_host.h"
#include "tc_ptx.cuh"
#include "tc_tile.cuh"

#include <math.h>
#include <stddef.h>

namespace lrm {

namespace {

using B16 = __nv_bfloat16;

constexpr int kBM = 128;  // rows per CTA; a pair tile has 256
constexpr int kBK = 128;  // bytes, and elements, of a K slice

enum Kind { FWD = 0, DX = 1 };

// The scales of a tile's rows and columns for the next kRun K slices, two of them in turn.
constexpr int kRun = 8;
struct Scales {
  // a row's scale times that of each of the tile's two blocks of columns; SwiGLU: of the gate's, then of the up's
  // (the pad keeps the writing lanes' eight slices of four rows off each other's banks)
  float xw[2][kRun][kBM + 4];
  int tile[4];  // e, row0, row_end, n0 of the tile
};

// RES: 0 without a residual, 1 with one, 2 with one and outputs that go straight to memory.
template <int BN, bool GLU, int RES>
struct Cfg {
  static constexpr int kABytes = kBM * kBK;
  static constexpr int kBBytes = BN / 2 * kBK;  // this CTA's half of the columns
  static constexpr int kStage = kABytes + kBBytes;
  // SwiGLU's 32 columns a warp leave room for a fifth stage (65536 rows over 128 experts to 2 x 768, K = 2048: 246 us,
  // with four and a second box 250 us; with z 280 and 290 us)
  static constexpr bool kOneBox = BN == 256 && GLU && !RES;
  static constexpr int kStages = BN == 256 ? (kOneBox ? 5 : 4) : 6;
  static constexpr int kEpiBytes = kOneBox ? kBoxBytes : 2 * kBoxBytes;  // of an epilogue warp
  static constexpr int kEpiWarps = BN / 16;
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kAccs = 512 / BN;  // all of TMEM
  static constexpr uint32_t kEpi = kStages * kStage;
  static constexpr uint32_t kScales = kEpi + kEpiWarps * kEpiBytes;
  static constexpr uint32_t kBars = kScales + 2 * sizeof(Scales);
  // full, empty; accumulator full, empty; scales full[2], empty[2]; drain; residual of each epilogue warp
  static constexpr int kNBars = 2 * kStages + 2 * kAccs + 5 + kEpiWarps;
  static constexpr int kPrefix = LRM_MAX_EXPERTS + 2;
  static constexpr size_t smem() { return 1024 + kBars + kNBars * 8 + 16 + 4 * (kPrefix + kThreads / 32); }
  static_assert(1024 + kBars + kNBars * 8 + 16 + 4 * (kPrefix + kThreads / 32) <= 232448, "shared memory");
};

struct Params {
  int E;
  int64_t R;
  int N;        // columns of the output
  int tiles_n;
  int slices;   // K slices of the whole reduction
  int half_slices;  // DX: K slices of one half of dz's columns (SwiGLU: gate, then up); else as slices
  int halves;   // matrices of W an expert has: 2 for SwiGLU
  int w_rows;   // FWD: blocks of rows of one matrix of W; DX: blocks of its columns
  const float *x_scale, *w_scale;
  const int32_t* seg;  // NULL: one dense problem
  int act;
  const void* bias;
  void *y, *z;
  int32_t* status;
};

template <int BN>
__host__ __device__ constexpr uint32_t instr_desc(uint32_t b_mn) {  // D fp32, A and B e4m3, M = 256
  return (1u << 4) | (b_mn << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)((2 * kBM) >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 columns of this warp's quarter of TMEM.
__device__ __forceinline__ void tmem_take16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
// acc += s * v, two sums at a time
__device__ __forceinline__ void add_scaled(float* acc, const float (&v)[16], float s) {
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 r = __ffma2_rn(make_float2(v[i], v[i + 1]), s2, make_float2(acc[i], acc[i + 1]));
    acc[i] = r.x;
    acc[i + 1] = r.y;
  }
}
__device__ __forceinline__ float lds(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival, in either CTA of the pair, for the converged warp.
__device__ __forceinline__ void mbar_arrive_one(uint32_t cbar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cbar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_one_cta(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// Polls by a whole warp with one answer.
__device__ __forceinline__ bool mbar_try_all(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred q, p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The waits of the MMA warp and the epilogue: no call (what they hold in registers stays there), and no clock read
// before the first 256 polls.  The epilogue does not test the answer: a wait that gives up raises the abort flag, which
// it looks at once a run of slices; later waits then return at once.
__device__ __forceinline__ bool mbar_wait_here(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               int32_t* status) {
  if (mbar_try_all(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 0; it < (1u << 30); ++it) {
    if (mbar_try_all(bar, parity)) return true;
    if ((it & 255u) == 255u) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, now - t0 > kWaitNs)) break;
    }
  }
  *abort_flag = 1;
  set_status(status, LRM_ERR_TIMEOUT);
  return false;
}

// v += 8 bf16 values
__device__ __forceinline__ void add8(float* v, uint4 r) {
  float f[8];
  unpack(r, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += f[i];
}

__device__ __forceinline__ void st32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// A warp's 32 rows of bf16 output, a row per lane: whole 32-row blocks go through shared memory and TMA (which clips
// columns past the tensor), others by each live lane.  WIDE: in one box of 64 columns, else in boxes of 32.
template <bool WIDE, bool SECTORS>
struct Boxes {
  uint8_t* box;
  int lane;
  // 128-byte swizzle: piece j of row r sits at j ^ (r & 7); 64-byte swizzle: at j ^ ((r >> 1) & 3)
  __device__ __forceinline__ uint4* piece(int c, int j) const {
    return WIDE ? reinterpret_cast<uint4*>(box + lane * 128 + (((4 * c + j) ^ (lane & 7)) << 4))
                : reinterpret_cast<uint4*>(box + c * kBoxBytes + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
  }
  __device__ __forceinline__ void free() const {  // the last stores have read the boxes
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
  // 32 columns into chunk c, or to memory (SECTORS: always, in whole sectors)
  __device__ __forceinline__ void put(const float (&v)[32], int c, int n, int cols, bool whole, bool live,
                                      B16* at) const {
    uint4 last;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = v[8 * j + i];
      const uint4 q = pack(f);
      if constexpr (SECTORS) {
        if ((j & 1) && live && n + 8 * j < cols) st32(at + 8 * j - 8, last, q);
        last = q;
      } else if (whole) {  // warp-uniform
        *piece(c, j) = q;
      } else if (live && n + 8 * j < cols) {
        st16(at + 8 * j, q);
      }
    }
  }
  __device__ __forceinline__ void send(const CUtensorMap* map, int c, int n, int row, int half) const {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_3d(map, smem_u32(box + c * kBoxBytes), n, row, half);
  }
};

template <int ACT>
__device__ __forceinline__ void act_all(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    if (ACT == LRM_ACT_GELU || ACT == LRM_ACT_SILU) {
      const float2 z = make_float2(v[i], v[i + 1]), r = ACT == LRM_ACT_GELU ? gelu2(z) : silu2(z);
      v[i] = r.x;
      v[i + 1] = r.y;
    } else {
      v[i] = act_value<ACT>(v[i]);
      v[i + 1] = act_value<ACT>(v[i + 1]);
    }
  }
}

struct Tile {
  int e;
  int row0, row_end;  // this CTA's output rows
  int n0;             // first output column
  bool has_rows;
};

template <int BN, bool GLU>
__device__ __forceinline__ Tile decode(const Params& p, const int* prefix, int t, int rank) {
  Tile d;
  const int mg = t / p.tiles_n, nt = t - mg * p.tiles_n;
  d.n0 = nt * (GLU ? BN / 2 : BN);
  d.e = 0;
  int end = (int)p.R;
  if (p.seg != nullptr) {
    d.e = last_at_most(prefix, p.E, mg);
    end = __ldg(p.seg + d.e + 1);
    d.row0 = __ldg(p.seg + d.e) + (mg - prefix[d.e]) * (2 * kBM) + rank * kBM;
  } else {
    d.row0 = mg * (2 * kBM) + rank * kBM;
  }
  d.row_end = min(end, d.row0 + kBM);
  d.has_rows = d.row0 < end;
  return d;
}

template <int KIND, int BN, bool GLU, int RES>
__global__ void __launch_bounds__(Cfg<BN, GLU, RES>::kThreads, 1)
    fp8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ,
                  const __grid_constant__ CUtensorMap tmR, const Params p) {
  using C = Cfg<BN, GLU, RES>;
  constexpr int S = C::kStages, ACCS = C::kAccs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kNBars);
  int* abort_flag = reinterpret_cast<int*>(tmem_holder + 1);
  int* prefix = abort_flag + 3;     // [E + 1] row tiles before each expert
  int* scan = prefix + C::kPrefix;  // [kThreads / 32]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * S;
  const uint32_t accf0 = empty0 + 8 * S, acce0 = accf0 + 8 * ACCS;
  const uint32_t sf0 = acce0 + 8 * ACCS, se0 = sf0 + 16, drain = se0 + 16, res0 = drain + 8;
  Scales* scales = reinterpret_cast<Scales*>(smem + C::kScales);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 2);   // leader's: both producers arrive with their byte counts
      mbar_init(empty0 + 8 * s, 1);  // the leader's commit, multicast to the pair
    }
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(accf0 + 8 * i, 1);
      mbar_init(acce0 + 8 * i, 2 * C::kEpiWarps);  // leader's: the epilogue warps of both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sf0 + 8 * i, 2);             // both scale warps
      mbar_init(se0 + 8 * i, C::kEpiWarps);  // the epilogue warps
    }
    mbar_init(drain, 1);
    for (int i = 0; i < C::kEpiWarps; ++i) mbar_init(res0 + 8 * i, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_holder), 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any remote operation targets them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  chain_wait();  // the set-up above touches no global memory

  int n_tiles;
  if (p.seg == nullptr)
    n_tiles = (int)((p.R + 2 * kBM - 1) / (2 * kBM)) * p.tiles_n;
  else
    n_tiles = segment_tiles<C::kThreads>(p.seg, p.E, p.R, 2 * kBM, prefix, scan, p.status) * p.tiles_n;
  const int rounds = (n_tiles + n_pairs - 1) / n_pairs;
  volatile int* abortv = abort_flag;
  const uint32_t full_lead = cluster_addr(full0, 0), acce_lead = cluster_addr(acce0, 0);

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer ----
    uint32_t it = 0, st = 0, sph = 0;
    bool ok = true;
    for (int i = 0, t; i < rounds && ok; ++i) {
      t = nth_tile(i, pair, n_pairs);
      if (t >= n_tiles) continue;  // (a last round may leave some pairs without one)
      const Tile d = decode<BN, GLU>(p, prefix, t, rank);
      const uint32_t bytes = C::kBBytes + (d.has_rows ? C::kABytes : 0);
      for (int kb = 0; kb < p.slices; ++kb, ++it) {
        const uint32_t s = st, ph = sph;
        if (++st == (uint32_t)S) { st = 0; sph ^= 1u; }
        if (!mbar_wait_ahead(empty0 + 8 * s, ph ^ 1u, abortv, p.status, false)) { ok = false; break; }
        const uint32_t fb = full_lead + 8 * s, a_dst = smem_u32(smem + s * C::kStage), b_dst = a_dst + C::kABytes;
        const int half = KIND == DX && kb >= p.half_slices ? 1 : 0, k = (kb - half * p.half_slices) * kBK;
        if (elect_one()) {
          mbar_expect_tx_cluster(fb, bytes);
          if (d.has_rows) tma_load_3d_pair(a_dst, &tmA, k, half, d.row0, fb);
          if (KIND == DX)
            tma_load_3d_pair(b_dst, &tmB, d.n0 + rank * (BN / 2), k, d.e * p.halves + half, fb);
          else if (GLU)  // the leader stages the gate rows, the other CTA the up rows
            tma_load_3d_pair(b_dst, &tmB, k, d.n0, d.e * 2 + rank, fb);
          else
            tma_load_3d_pair(b_dst, &tmB, k, d.n0 + rank * (BN / 2), d.e, fb);
        }
        __syncwarp();
      }
    }
    // drain: every stage this warp filled has been consumed (so its data landed)
    const uint32_t first = it > (uint32_t)S ? it - S : 0u;
    for (uint32_t i = first; i < it; ++i) mbar_wait(empty0 + 8 * (i % S), (i / S) & 1u, abortv, p.status, false);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer ------
    if (leader) {
      constexpr uint32_t idesc = instr_desc<BN>(KIND == DX ? 1u : 0u);
      const uint32_t a0 = smem_u32(smem), b0 = a0 + C::kABytes;
      // a row of the swizzle is 128 bytes: of K (rows of x and W), or of columns (DX: W's rows below one another)
      const uint64_t adesc0 = smem_desc(a0, 16, 1024), bdesc0 = smem_desc(b0, 16, 1024);
      constexpr uint64_t a_step = 32 >> 4, b_step = KIND == FWD ? (32 >> 4) : (32 * 128 >> 4);
      uint32_t st = 0, sph = 0, aph = ~0u;  // operand stage and its phase; phases of the accumulators, a bit each
      bool ok = true;
      for (int i = 0, t; i < rounds && ok; ++i) {
        t = nth_tile(i, pair, n_pairs);
        if (t >= n_tiles) continue;
        for (int kb = 0; kb < p.slices; ++kb) {
          const uint32_t acc = kb % ACCS;
          if (!mbar_wait_here(full0 + 8 * st, sph, abortv, p.status) ||
              !mbar_wait_here(acce0 + 8 * acc, (aph >> acc) & 1u, abortv, p.status)) {
            ok = false;
            break;
          }
          aph ^= 1u << acc;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t soff = (uint64_t)((st * C::kStage) >> 4);
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)
              mma_e4m3(tmem_base + acc * BN, adesc0 + soff + kk * a_step, bdesc0 + soff + kk * b_step, idesc,
                       kk != 0 ? 1u : 0u);
            mma_commit_pair(empty0 + 8 * st);
            mma_commit_pair(accf0 + 8 * acc);
          }
          __syncwarp();
          if (++st == (uint32_t)S) { st = 0; sph ^= 1u; }
        }
      }
      if (elect_one()) mma_commit_pair(drain);
    }
    __syncwarp();
    mbar_wait_ahead(drain, 0, abortv, p.status, true);  // all MMAs into this CTA's TMEM are done before it is freed
  } else if (warp < 4) {
    // ---------------------------------------------------------------- scales ----------
    // each of the two warps loads 64 rows, eight slices of four rows at a time (whole sectors where rows allow)
    const int part = warp - 2, lk = lane & 7, lr = lane >> 3;
    uint32_t b = 0, bph = 0;
    bool ok = true;
    for (int i = 0, t; i < rounds && ok; ++i) {
      t = nth_tile(i, pair, n_pairs);
      if (t >= n_tiles) continue;
      const Tile d = decode<BN, GLU>(p, prefix, t, rank);
      // the tile's blocks of W's columns (columns past the last have any)
      const int blk0 = d.n0 / kQBlock, blk1 = min(blk0 + 1, p.w_rows - 1);
      for (int k0 = 0; k0 < p.slices; k0 += kRun) {
        if (!mbar_wait_ahead(se0 + 8 * b, bph ^ 1u, abortv, p.status, false)) { ok = false; break; }
        const int k = k0 + lk;
        float v[kBM / 8], w0 = 0.f, w1 = 0.f;
        const float* sx = p.x_scale + (int64_t)(d.row0 + part * (kBM / 2) + lr) * p.slices + k;
#pragma unroll
        for (int j = 0; j < kBM / 8; ++j) {
          const int row = d.row0 + part * (kBM / 2) + lr + 4 * j;
          v[j] = k < p.slices && row < d.row_end ? __ldg(sx + (int64_t)(4 * j) * p.slices) : 0.f;
        }
        if (k < p.slices) {
          if (KIND == DX) {
            const float* w = p.w_scale + ((int64_t)d.e * p.slices + k) * p.w_rows;
            w0 = __ldg(w + blk0);
            w1 = __ldg(w + blk1);
          } else {
            const float* w = p.w_scale + (int64_t)(GLU ? d.e * 2 : d.e) * p.w_rows * p.slices + k;
            w0 = __ldg(w + (int64_t)blk0 * p.slices);
            w1 = __ldg(w + (int64_t)(GLU ? p.w_rows + blk0 : blk1) * p.slices);
          }
        }
        Scales& to = scales[b];
#pragma unroll
        for (int j = 0; j < kBM / 8; ++j) {
          to.xw[0][lk][part * (kBM / 2) + lr + 4 * j] = v[j] * w0;
          to.xw[1][lk][part * (kBM / 2) + lr + 4 * j] = v[j] * w1;
        }
        if (part == 1 && lane == 0)
          *reinterpret_cast<int4*>(to.tile) = make_int4(d.e, d.has_rows ? d.row0 : d.row_end, d.row_end, d.n0);
        __syncwarp();
        if (lane == 0) mbar_arrive(sf0 + 8 * b);
        b ^= 1u;
        if (b == 0) bph ^= 1u;
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue --------
    constexpr int NO = GLU ? 1 : 2;  // 32-column chunks of output of a warp
    constexpr int kBlock = (int)sizeof(scales[0].xw[0]);
    const int ew = warp - 4, q = warp & 3, group = ew >> 2;
    uint8_t* boxes = smem + C::kEpi + ew * C::kEpiBytes;
    const uint32_t res_bar = res0 + 8 * ew;
    // TMEM columns of the warp's two chunks (SwiGLU: gate, up)
    const uint32_t col0 = group * NO * 32, col1 = GLU ? BN / 2 + group * 32 : col0 + 32;
    const uint32_t quarter = tmem_base + ((uint32_t)(q * 32) << 16);
    const int NP = GLU ? 2 * p.N : p.N;
    const uint32_t scales_s = smem_u32(scales);
    uint32_t aph = 0, b = 0, bph = 0, rph = 0;  // phases of the accumulators (a bit each), the scales and the residual
    for (int i = 0; i < rounds; ++i) {
      if (nth_tile(i, pair, n_pairs) >= n_tiles) continue;
      float acc[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c][j] = 0.f;
      // the tile comes with its first scales (segment bounds are a trip to memory, which the scale warps make ahead)
      if (!mbar_wait_here(sf0 + 8 * b, bph, abortv, p.status)) break;
      const int4 d = *reinterpret_cast<const int4*>(scales[b].tile);  // expert, first and last row, first column
      const int row_base = d.y + q * 32, n_first = d.w + group * NO * 32;
      // (the check, where it is on, covers what this warp's stores address: the expert, and its first and last row)
      const int nrows = LRM_DCHECK(d.x >= 0 && d.x < p.E && row_base >= 0 && d.z <= p.R, p.status, LRM_ERR_BAD_INDEX)
                            ? min(32, d.z - row_base)
                            : 0;
      const bool mine = nrows > 0 && n_first < p.N;  // warp-uniform: this warp has output
      if (RES && mine && lane == 0) {  // the residual comes into the boxes meanwhile
        bulk_wait_read<0>();
        mbar_expect_tx(res_bar, NO * kBoxBytes);
        tma_load_3d_cta(smem_u32(boxes), &tmR, n_first, row_base, 0, res_bar);
      }
      const B16* bias = KIND == FWD && p.bias != nullptr
                            ? static_cast<const B16*>(p.bias) + (int64_t)d.x * NP + n_first
                            : nullptr;
      if (bias != nullptr && mine) {  // on its way meanwhile
        prefetch_l1(bias);
        if (GLU) prefetch_l1(bias + p.N);
      }
      const int blk = n_first / kQBlock - d.w / kQBlock;  // 0 or 1
      bool ok = true;
      for (int k0 = 0; k0 < p.slices; k0 += kRun) {
        if (k0 > 0) mbar_wait_here(sf0 + 8 * b, bph, abortv, p.status);
        const uint32_t xa = scales_s + b * (uint32_t)sizeof(Scales) + (GLU ? 0 : blk * kBlock) + (q * 32 + lane) * 4;
#pragma unroll 2  // (eight at a time spill)
        for (int kr = 0; kr < min(kRun, p.slices - k0); ++kr) {
          constexpr int kPitch = (int)sizeof(scales[0].xw[0][0]);
          const int a = kr % ACCS;  // (a tile starts at the first accumulator)
          const float s0 = lds(xa + kr * kPitch), s1 = GLU ? lds(xa + kBlock + kr * kPitch) : s0;
          mbar_wait_here(accf0 + 8 * a, (aph >> a) & 1u, abortv, p.status);
          aph ^= 1u << a;
          tc_fence_after();
          const uint32_t tbase = quarter + a * BN;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float r[16];
            tmem_take16(tbase + (c < 2 ? col0 : col1) + (c & 1) * 16, r);
            if (c == 3) {  // the accumulator goes back before its last columns are added
              tc_fence_before();
              mbar_arrive_one(acce_lead + 8 * a);
            }
            add_scaled(acc[c >> 1] + (c & 1) * 16, r, c < 2 ? s0 : s1);
          }
        }
        mbar_arrive_one_cta(se0 + 8 * b);
        b ^= 1u;
        if (b == 0) bph ^= 1u;
        if (__any_sync(0xffffffffu, *abortv != 0)) {
          ok = false;
          break;
        }
      }
      if (!ok) {  // (the residual's copy lands before the CTA exits)
        if (RES && mine) mbar_wait(res_bar, rph, abortv, p.status, false);
        break;
      }
      if (!mine) continue;
      // without segments the output map ends where the rows end, so TMA clips a partial block
      const bool whole = RES != 2 && (nrows == 32 || p.seg == nullptr);
      const bool live = lane < nrows;
      const int64_t row = row_base + lane;
      if (RES) {
        mbar_wait_here(res_bar, rph, abortv, p.status);
        rph ^= 1u;
      }
      const Boxes<!GLU, RES == 2> out{boxes, lane};
      if (KIND == FWD && bias != nullptr) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n_first + (GLU ? 0 : c * 32) + 8 * j < p.N)
              add8(acc[c] + 8 * j, ldg16(bias + (GLU ? c * p.N : c * 32) + 8 * j));
      }
      if (KIND == FWD && p.z != nullptr) {  // (where the boxes hold the residual, from the registers)
        const bool boxed = whole && !RES;
        const bool z_live = live || (whole && row < d.z);
        B16* z_row = static_cast<B16*>(p.z) + row * NP + n_first;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int at = C::kOneBox ? 0 : c;
          if (boxed && (c == 0 || C::kOneBox)) out.free();
          out.put(acc[c], at, n_first + (GLU ? 0 : c * 32), p.N, boxed, z_live, z_row + (GLU ? c * p.N : c * 32));
          if (boxed && (c == 1 || GLU)) out.send(&tmZ, GLU ? at : 0, n_first, row_base, GLU ? c : 0);
        }
      }
      if (whole && !RES) out.free();
#pragma unroll
      for (int c = 0; c < NO; ++c) {
        float(&v)[32] = acc[c];
        if (KIND == FWD) {
          if (GLU) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 r = __fmul2_rn(silu2(make_float2(v[j], v[j + 1])), make_float2(acc[1][j], acc[1][j + 1]));
              v[j] = r.x;
              v[j + 1] = r.y;
            }
          } else {
            switch (p.act) {
              case LRM_ACT_RELU: act_all<LRM_ACT_RELU>(v); break;
              case LRM_ACT_GELU: act_all<LRM_ACT_GELU>(v); break;
              case LRM_ACT_SILU: act_all<LRM_ACT_SILU>(v); break;
              default: break;
            }
          }
          if (RES)
#pragma unroll
            for (int j = 0; j < 4; ++j) add8(v + 8 * j, *out.piece(c, j));
        }
        out.put(v, c, n_first + c * 32, p.N, whole, live, static_cast<B16*>(p.y) + row * p.N + n_first + c * 32);
      }
      if (whole) out.send(&tmY, 0, n_first, row_base, 0);
      if (RES == 2) __syncwarp();  // every lane has read its residual: the next may come
    }
    if (lane == 0) bulk_wait_all();  // stores complete before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no remote arrive may target a CTA that has exited
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- host side ----------
// 8-bit operands [d2][d1][d0], d0 contiguous and a multiple of 16, with a {128, b1, b2} box.
bool fp8_map(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t b1, uint32_t b2) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {d0, d0 * d1};
  const cuuint32_t box[3] = {128, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// bf16 rows [rows][halves][cols] in boxes of 32 rows and `wide` (32 or 64) columns of one half.
bool rows_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t halves, uint32_t wide) {
  const cuuint64_t dims[3] = {cols, rows, halves};
  const cuuint64_t strides[2] = {cols * halves * 2, halves > 1 ? cols * 2 : cols * rows * 2};
  const cuuint32_t box[3] = {wide, 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     wide == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// About how many row tiles there are: every expert with rows ends in half a tile, and has one at least.
double likely_tiles(bool grouped, int64_t R, int E) {
  const double whole = (double)((R + kTileRows - 1) / kTileRows);
  if (!grouped) return whole;
  const double active = E * (1. - exp(-(double)R / E));
  return active > (double)R / kTileRows + active / 2 ? active : (double)R / kTileRows + active / 2;
}

int blocks_of(int n) { return (n + kQBlock - 1) / kQBlock; }

}  // namespace

lrm_status launch_fp8_tc(const Fp8Args& a, cudaStream_t s) {
  if (!device_ok() || encode_fn() == nullptr) return LRM_ERR_UNSUPPORTED;
  const bool glu = a.act == LRM_ACT_SWIGLU;
  const uint32_t wide = glu ? 32 : 64;
  Params p{};
  p.E = a.E;
  p.R = a.R;
  p.N = a.N;
  p.slices = p.half_slices = blocks_of(a.K);
  p.halves = glu ? 2 : 1;
  p.w_rows = blocks_of(a.N);
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.seg = a.seg_offsets;
  p.act = a.act;
  p.bias = a.bias;
  p.y = a.y;
  p.z = a.z;
  p.status = a.status;
  CUtensorMap mA, mB, mY, mZ, mR;
  if (!fp8_map(&mA, a.x, a.K, 1, a.R, 1, kBM) || !rows_map(&mY, a.y, a.N, a.R, 1, wide)) return LRM_ERR_CUDA;
  mZ = mR = mY;
  if (a.z != nullptr && !rows_map(&mZ, a.z, a.N, a.R, p.halves, wide)) return LRM_ERR_CUDA;
  if (a.residual != nullptr && !rows_map(&mR, a.residual, a.N, a.R, 1, wide)) return LRM_ERR_CUDA;
  auto tiles = [&](auto bn, auto glu_tag, auto res_tag) {
    constexpr int BN = decltype(bn)::value;
    constexpr bool GLU = decltype(glu_tag)::value != 0;
    constexpr int RES = decltype(res_tag)::value;
    constexpr int cols = GLU ? BN / 2 : BN;
    using C = Cfg<BN, GLU, RES>;
    p.tiles_n = (a.N + cols - 1) / cols;
    if (!fp8_map(&mB, a.w, a.K, a.N, (uint64_t)a.E * p.halves, BN / 2, 1)) return LRM_ERR_CUDA;
    return launch_pairs<fp8_tc_kernel<FWD, BN, GLU, RES>>(
        C::smem(), C::kThreads, row_tiles(a.seg_offsets, a.R, a.E) * p.tiles_n, s, mA, mB, mY, mZ, mR, p);
  };
  // Where the boxes hold the residual and pieces of 32 bytes are aligned, outputs go straight to memory (32768 x 4096 x
  // 4096 with bias, GELU and residual 514 us, through the boxes 521; without a residual the boxes are faster, 768 to
  // 2048 180 us and 190).
  const uintptr_t starts = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.z);
  const bool sectors = a.N % 16 == 0 && (starts & 31) == 0;
  auto go = [&](auto bn, auto glu_tag) {
    if (a.residual == nullptr) return tiles(bn, glu_tag, IntTag<0>{});
    return sectors ? tiles(bn, glu_tag, IntTag<2>{}) : tiles(bn, glu_tag, IntTag<1>{});
  };
  // Tile width by the waves of tiles over the CTA pairs; a K slice of a 256-column tile takes 0.43 us (its sums out of
  // TMEM), of a 128-column one 0.25 us, of a 64-column one 0.22 us.  E.g. 256 rows over 8 experts to 2 x 1408, K =
  // 4096: 88, 176 or 352 tiles, 35, 31 and 44 us; 8192 x 4096 x 4096 110, 123 and 211 us; 32 rows, 17, 12 and 11 us.
  const double rows = likely_tiles(a.seg_offsets != nullptr, a.R, a.E);
  const int pairs = sm_count() / 2, per = glu ? 2 : 1;
  auto cost = [&](int bn, double slice) { return ceil(rows * ((a.N * per + bn - 1) / bn) / pairs) * slice; };
  const double c256 = cost(256, 0.43), c128 = cost(128, 0.25), c64 = cost(64, 0.22);
  auto width = [&](auto glu_tag) {
    if (c64 <= c128 && c64 <= c256) return go(IntTag<64>{}, glu_tag);
    return c128 <= c256 ? go(IntTag<128>{}, glu_tag) : go(IntTag<256>{}, glu_tag);
  };
  return glu ? width(IntTag<1>{}) : width(IntTag<0>{});
}

// One tile width: whatever the size, tiles of 256 columns (1222 rows over 7 experts, 2 x 208 to 1040, 8.4 us, of which
// few CTA pairs are busy; narrower tiles were not measured here).
lrm_status launch_fp8_dx(const Fp8GradArgs& a, cudaStream_t s) {
  if (!device_ok() || encode_fn() == nullptr) return LRM_ERR_UNSUPPORTED;
  using C = Cfg<256, false, 0>;
  Params p{};
  p.E = a.E;
  p.R = a.R;
  p.N = a.K;
  p.tiles_n = (a.K + 255) / 256;
  p.halves = a.glu ? 2 : 1;
  p.half_slices = blocks_of(a.N);
  p.slices = p.halves * p.half_slices;
  p.w_rows = blocks_of(a.K);
  p.x_scale = a.dz_scale;
  p.w_scale = a.w_scale;
  p.seg = a.seg_offsets;
  p.y = a.dx;
  p.status = a.status;
  CUtensorMap mA, mB, mY;
  if (!fp8_map(&mA, a.dz, a.N, p.halves, a.R, 1, kBM) ||
      !fp8_map(&mB, a.w, a.K, a.N, (uint64_t)a.E * p.halves, kBK, 1) || !rows_map(&mY, a.dx, a.K, a.R, 1, 64))
    return LRM_ERR_CUDA;
  return launch_pairs<fp8_tc_kernel<DX, 256, false, 0>>(
      C::smem(), C::kThreads, row_tiles(a.seg_offsets, a.R, a.E) * p.tiles_n, s, mA, mB, mY, mY, mY, p);
}

}  // namespace lrm
