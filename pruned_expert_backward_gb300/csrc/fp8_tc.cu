// lrm_fp8_linear and lrm_fp8_linear_backward on the tensor cores of sm_103a (tcgen05 kind::f8f6f4, TMEM, TMA).
//
//   FWD  y  = act(sum over blocks b of 128 k: sx[r,b] sw[n/128,b] (x_b w_b^T) + bias) + residual
//   DX   dx = sum over blocks b of 128 n: sz[r,b] sw[b,k/128] (dz_b w_b)
//
// The scales change with every 128 steps of the reduction, so the products of a block are a sum of their own: each K
// slice of 128 (one stage of operands, four MMAs of K = 32) goes to the next of the accumulators that TMEM holds, and
// the epilogue warps take it out, scale it by row and block and add it up in fp32 registers while the tensor core is
// at the next.  A slice's products are exact to fp32's last bits, so the result errs like a sum of K / 128 fp32 numbers.
//
// CTA pairs, roles and tiles are those of linear_tc.cu: 256 x BN tiles over a persistent grid, warp 0 the TMA
// producer, warp 1 of the leader the MMA issuer.  BN / 16 epilogue warps each hold a 32-row quarter of TMEM by 64
// columns (64 registers of sums); SwiGLU: 32 gate columns and the 32 up columns that go with them.  They lie within
// one block of 128 columns, so that a warp has one weight scale a slice (two for SwiGLU).
//
// W stays as it was quantised: FWD reads its rows K-major, DX the same bytes with the columns contiguous (MN-major).
#include "fp8.cuh"
#include "kernels.h"
#include "linear.cuh"
#include "tc_host.h"
#include "tc_ptx.cuh"
#include "tc_tile.cuh"

namespace lrm {

namespace {

using B16 = __nv_bfloat16;

constexpr int kBM = 128;  // rows per CTA; a pair tile has 256
constexpr int kBK = 128;  // bytes, and elements, of a K slice

enum Kind { FWD = 0, DX = 1 };

template <int BN>
struct Cfg {
  static constexpr int kABytes = kBM * kBK;
  static constexpr int kBBytes = BN / 2 * kBK;  // this CTA's half of the columns
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 5 : 7;
  static constexpr int kEpiWarps = BN / 16;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kAccs = 512 / BN;  // accumulators: all of TMEM
  static constexpr uint32_t kEpi = kStages * kStage;
  static constexpr uint32_t kBars = kEpi + kEpiWarps * kBoxBytes;
  static constexpr int kNBars = 2 * kStages + 2 * kAccs + 1;  // full, empty; accumulator full, empty; drain
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
  const void *bias, *residual;
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

// 16 columns of TMEM on their way: the values are there after tmem_wait16 of the same registers.
__device__ __forceinline__ void tmem_start16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
// acc[16 i ..] += s * v, two at a time
__device__ __forceinline__ void add_scaled16(float (&acc)[32], int at, const uint32_t (&v)[16], float s) {
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), s2,
                                make_float2(acc[at + i], acc[at + i + 1]));
    acc[at + i] = r.x;
    acc[at + i + 1] = r.y;
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

template <int KIND, int BN, bool GLU>
__global__ void __launch_bounds__(Cfg<BN>::kThreads, 1)
    fp8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ, const Params p) {
  using C = Cfg<BN>;
  constexpr int S = C::kStages, ACCS = C::kAccs;
  static_assert(KIND == FWD || BN == 256, "DX stages 128 columns a CTA, one row of the 128-byte swizzle");
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
  const uint32_t accf0 = empty0 + 8 * S, acce0 = accf0 + 8 * ACCS, drain = acce0 + 8 * ACCS;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 2);   // leader's: both producers arrive with their byte counts
      mbar_init(empty0 + 8 * s, 1);  // the leader's commit, multicast to the pair
    }
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(accf0 + 8 * i, 1);
      mbar_init(acce0 + 8 * i, 2 * C::kEpiWarps);  // leader's: the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
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
        if (!mbar_wait_warp(empty0 + 8 * s, ph ^ 1u, abortv, p.status)) { ok = false; break; }
        const uint32_t fb = full_lead + 8 * s, a_dst = smem_u32(smem + s * C::kStage), b_dst = a_dst + C::kABytes;
        const int half = KIND == DX && kb >= p.half_slices ? 1 : 0, k = (kb - half * p.half_slices) * kBK;
        if (elect_one()) {
          mbar_expect_tx_cluster(fb, bytes);
          if (d.has_rows) tma_load_3d_pair(a_dst, &tmA, k, half, d.row0, fb);
          if (KIND == DX)
            tma_load_3d_pair(b_dst, &tmB, d.n0 + rank * 128, k, d.e * p.halves + half, fb);
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
      // a row of the swizzle is 128 bytes: of K (rows of x and W), or of columns (DX: 128 rows of W below one another)
      const uint64_t adesc0 = smem_desc(a0, 16, 1024);
      const uint64_t bdesc0 = KIND == FWD ? smem_desc(b0, 16, 1024) : smem_desc(b0, 16384, 1024);
      constexpr uint64_t a_step = 32 >> 4, b_step = KIND == FWD ? (32 >> 4) : (4096 >> 4);
      uint32_t st = 0, sph = 0, acc = 0, aph = 0;  // operand stage and accumulator, with their phases
      bool ok = true;
      for (int i = 0, t; i < rounds && ok; ++i) {
        t = nth_tile(i, pair, n_pairs);
        if (t >= n_tiles) continue;
        for (int kb = 0; kb < p.slices; ++kb) {
          if (!mbar_wait_warp(acce0 + 8 * acc, aph ^ 1u, abortv, p.status) ||
              !mbar_wait_warp(full0 + 8 * st, sph, abortv, p.status)) {
            ok = false;
            break;
          }
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
          if (++acc == (uint32_t)ACCS) { acc = 0; aph ^= 1u; }
        }
      }
      if (elect_one()) mma_commit_pair(drain);
    }
    __syncwarp();
    mbar_wait(drain, 0, abortv, p.status, false);  // all MMAs into this CTA's TMEM are done before it is freed
  } else {
    // ---------------------------------------------------------------- epilogue --------
    constexpr int NO = GLU ? 1 : 2;  // 32-column chunks of output of a warp
    const int ew = warp - 2, q = warp & 3, group = ew >> 2;
    uint8_t* boxes = smem + C::kEpi + ew * kBoxBytes;
    Out<1> out{boxes, smem_u32(boxes), 0};
    // TMEM column of the warp's chunk c (SwiGLU: gate, up)
    const uint32_t col0 = GLU ? group * 32 : group * 64, col1 = GLU ? BN / 2 + group * 32 : group * 64 + 32;
    const int NP = GLU ? 2 * p.N : p.N;
    uint32_t a = 0, aph = 0;
    bool ok = true;
    for (int i = 0, t; i < rounds && ok; ++i) {
      t = nth_tile(i, pair, n_pairs);
      if (t >= n_tiles) continue;
      const Tile d = decode<BN, GLU>(p, prefix, t, rank);
      const int row_base = d.row0 + q * 32;
      // (the check, where it is on, covers what this warp's stores address: the expert, and its first and last row)
      const int nrows = d.has_rows && LRM_DCHECK(d.e >= 0 && d.e < p.E && row_base >= 0 && d.row_end <= p.R, p.status,
                                                 LRM_ERR_BAD_INDEX)
                            ? min(32, d.row_end - row_base)
                            : 0;
      // without segments the output map ends where the rows end, so TMA clips a partial block
      const bool whole = nrows == 32 || (nrows > 0 && p.seg == nullptr);
      const bool live = lane < nrows;
      const int64_t row = row_base + lane;
      const int n_first = d.n0 + group * NO * 32;
      // this row's scales, and those of the warp's block of columns (rows and columns past the last have any)
      const float* sx = p.x_scale + (live ? row : 0) * p.slices;
      const int blk = min(n_first / kQBlock, p.w_rows - 1);
      const float *sw0, *sw1 = nullptr;
      int64_t w_step = 1;
      if (KIND == DX) {
        sw0 = p.w_scale + (int64_t)d.e * p.slices * p.w_rows + blk;
        w_step = p.w_rows;
      } else {
        sw0 = p.w_scale + ((int64_t)d.e * p.halves * p.w_rows + blk) * p.slices;
        if (GLU) sw1 = sw0 + (int64_t)p.w_rows * p.slices;
      }
      float acc[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c][j] = 0.f;
      // scales one slice ahead
      float nx = __ldg(sx), n0 = __ldg(sw0), n1 = GLU ? __ldg(sw1) : 0.f;
      for (int kb = 0; kb < p.slices; ++kb) {
        const float s0 = nx * n0, s1 = GLU ? nx * n1 : s0;
        if (kb + 1 < p.slices) {
          nx = __ldg(sx + kb + 1);
          n0 = __ldg(sw0 + (kb + 1) * w_step);
          if (GLU) n1 = __ldg(sw1 + kb + 1);
        }
        if (!mbar_wait(accf0 + 8 * a, aph, abortv, p.status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tbase = tmem_base + a * BN + ((uint32_t)(q * 32) << 16);
        uint32_t r0[16], r1[16];
        __syncwarp();
        tmem_start16(tbase + col0, r0);
        tmem_wait16(r0);
        tmem_start16(tbase + col0 + 16, r1);
        add_scaled16(acc[0], 0, r0, s0);
        tmem_wait16(r1);
        tmem_start16(tbase + col1, r0);
        add_scaled16(acc[0], 16, r1, s0);
        tmem_wait16(r0);
        tmem_start16(tbase + col1 + 16, r1);
        add_scaled16(acc[1], 0, r0, s1);
        tmem_wait16(r1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acce_lead + 8 * a);
        add_scaled16(acc[1], 16, r1, s1);
        if (++a == (uint32_t)ACCS) { a = 0; aph ^= 1u; }
      }
      if (!ok) break;
      __syncwarp();
      const B16* res =
          KIND == FWD && p.residual != nullptr && live ? static_cast<const B16*>(p.residual) + row * p.N : nullptr;
      B16* y_row = static_cast<B16*>(p.y) + row * p.N;
#pragma unroll
      for (int c = 0; c < NO; ++c) {
        const int n = n_first + c * 32;
        if (nrows <= 0 || n >= p.N) continue;  // warp-uniform
        float(&v)[32] = acc[c];
        if (KIND == FWD) {
          if (p.bias != nullptr) {
            const B16* b = static_cast<const B16*>(p.bias) + (int64_t)d.e * NP;
            add_row(v, b, n, p.N);
            if (GLU) add_row(acc[1], b + p.N, n, p.N);
          }
          if (p.z != nullptr) {
            B16* z_row = static_cast<B16*>(p.z) + row * NP;
            out.put(v, &tmZ, lane, n, p.N, row_base, 0, whole, live, z_row);
            if (GLU) out.put(acc[1], &tmZ, lane, n, p.N, row_base, 1, whole, live, z_row + p.N);
          }
          if (GLU) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = act_value<LRM_ACT_SWIGLU>(v[j]) * acc[1][j];
          } else {
            switch (p.act) {
              case LRM_ACT_RELU: act32<LRM_ACT_RELU>(v); break;
              case LRM_ACT_GELU: act32<LRM_ACT_GELU>(v); break;
              case LRM_ACT_SILU: act32<LRM_ACT_SILU>(v); break;
              default: break;
            }
          }
          if (res != nullptr) add_row(v, res, n, p.N);
        }
        out.put(v, &tmY, lane, n, p.N, row_base, 0, whole, live, y_row);
      }
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
  const cuuint32_t box[3] = {kBK, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int blocks_of(int n) { return (n + kQBlock - 1) / kQBlock; }

}  // namespace

lrm_status launch_fp8_tc(const Fp8Args& a, cudaStream_t s) {
  if (!device_ok() || encode_fn() == nullptr) return LRM_ERR_UNSUPPORTED;
  const bool glu = a.act == LRM_ACT_SWIGLU;
  const int NP = glu ? 2 * a.N : a.N;
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
  p.residual = a.residual;
  p.y = a.y;
  p.z = a.z;
  p.status = a.status;
  CUtensorMap mA, mB, mY, mZ;
  if (!fp8_map(&mA, a.x, a.K, 1, a.R, 1, kBM) || !output_map(&mY, a.y, false, a.N, a.R, 1)) return LRM_ERR_CUDA;
  mZ = mY;
  if (a.z != nullptr && !output_map(&mZ, a.z, false, a.N, a.R, glu ? 2 : 1, glu)) return LRM_ERR_CUDA;
  auto go = [&](auto bn, auto glu_tag) {
    constexpr int BN = decltype(bn)::value;
    constexpr bool GLU = decltype(glu_tag)::value != 0;
    constexpr int cols = GLU ? BN / 2 : BN;
    p.tiles_n = (a.N + cols - 1) / cols;
    if (!fp8_map(&mB, a.w, a.K, a.N, (uint64_t)a.E * p.halves, BN / 2, 1)) return LRM_ERR_CUDA;
    return launch_pairs<fp8_tc_kernel<FWD, BN, GLU>>(Cfg<BN>::smem(), Cfg<BN>::kThreads,
                                                     row_tiles(a.seg_offsets, a.R, a.E) * p.tiles_n, s, mA, mB, mY, mZ,
                                                     p);
  };
  const int64_t likely = likely_row_tiles(a.seg_offsets, a.R, a.E);
  if (glu) return with_width(likely, NP, 64, [&](auto bn) { return go(bn, IntTag<1>{}); });
  return with_width(likely, NP, 64, [&](auto bn) { return go(bn, IntTag<0>{}); });
}

lrm_status launch_fp8_dx(const Fp8GradArgs& a, cudaStream_t s) {
  if (!device_ok() || encode_fn() == nullptr) return LRM_ERR_UNSUPPORTED;
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
      !fp8_map(&mB, a.w, a.K, a.N, (uint64_t)a.E * p.halves, 128, 1) || !output_map(&mY, a.dx, false, a.K, a.R, 1))
    return LRM_ERR_CUDA;
  return launch_pairs<fp8_tc_kernel<DX, 256, false>>(Cfg<256>::smem(), Cfg<256>::kThreads,
                                                     row_tiles(a.seg_offsets, a.R, a.E) * p.tiles_n, s, mA, mB, mY, mY,
                                                     p);
}

}  // namespace lrm
