// Internal launchers of the LRM-pruned expert backward kernels.  abi.cu validates the
// arguments of the public entry points and calls these; they only launch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "lrm.h"

namespace lrm {

// Selection works on chunks of this many consecutive pairs (one CTA, one pair per thread).
constexpr int kSelChunk = 256;

struct SelectWs {
  int32_t* counts;        // [n_chunks][E]  per-chunk expert counts, then exclusive bases
  int32_t* bucket_start;  // [E+1]          start of each expert's bucket in sorted_u
  int32_t* keep;          // [E]            min(max(quota,0), load), or 0 on capacity overflow
  int32_t* loads;         // [E]            pairs routed to each expert
  int32_t* sorted_u;      // [P]            pairs grouped by expert, u ascending
  uint32_t* sorted_key;   // [P]            score bits in the same order
  int64_t n_chunks;
};

// Scratch of the tensor-core grouped GEMMs: tile tables, then 6*E per-expert TMA tensor maps
// (128 bytes each, 128-byte aligned) built on the device from seg_offsets.
struct GemmWs {
  int32_t* plan;  // [2E+3+kTileCounters]
  void* maps;     // [6][E] CUtensorMap
};
// var-K launches of one grouped call whose tile counters sit in the plan region
constexpr int kTileCounters = 2;
size_t gemm_plan_bytes(int32_t E);  // plan[2E+3+kTileCounters]: tile tables, checks, tile counters
size_t gemm_ws_bytes(int32_t E);

struct WsLayout {
  size_t counts, bucket_start, keep, loads, sorted_u, sorted_key, gemm, total;
};
WsLayout workspace_layout(int64_t P, int32_t E);

void launch_plan_quotas(const int32_t* topk_idx, int64_t P, int32_t E, int kind, int32_t num, int32_t den,
                        int32_t cap, const int32_t* explicit_q, int32_t* loads, int32_t* quotas, int32_t* status,
                        cudaStream_t s);

void launch_score(const float* alpha, const void* g, const void* phi, int64_t T, int32_t k, int32_t H, int32_t I,
                  lrm_dtype dt, float* scores, int32_t* status, cudaStream_t s);

void launch_score_norms(const float* alpha, const void* g, const float* phi_sq, int64_t T, int32_t k, int32_t H,
                        lrm_dtype dt, float* scores, int32_t* status, cudaStream_t s);

lrm_status launch_route(const float* logits, int64_t T, int32_t E, int32_t k, int kind, int32_t num, int32_t den,
                        int32_t cap, const int32_t* explicit_q, int32_t* topk_idx, float* alpha, int32_t* loads,
                        int32_t* quotas, uint32_t* done, int32_t* status, cudaStream_t s);

void launch_swiglu_forward(const void* h, int64_t P, int32_t I, lrm_dtype dt, void* phi, float* phi_sq,
                           cudaStream_t s);

void launch_grad_score(const void* g, int64_t T, int32_t k, int32_t H, lrm_dtype dt, bool abs_mode, float* scores,
                       int32_t* status, cudaStream_t s);

void launch_select(const int32_t* topk_idx, const float* scores, const int32_t* quotas, int64_t P, int32_t E,
                   int64_t cap, int32_t* seg_offsets, int32_t* kept_pair, int32_t* row_of_pair, const SelectWs& ws,
                   int32_t* status, cudaStream_t s);

void launch_compact(const int32_t* row_of_pair, const float* alpha, const void* g, const void* x, const void* h,
                    const void* phi, int64_t T, int32_t k, int32_t H, int32_t I, lrm_dtype dt, int64_t cap,
                    void* dy_c, void* x_c, void* h_c, void* phi_c, int32_t* status, cudaStream_t s);

void launch_scatter_dx(const int32_t* row_of_pair, const void* dx_c, int64_t T, int32_t k, int32_t H, lrm_dtype dt,
                       int64_t cap, void* dx, int32_t* status, cudaStream_t s);

struct GroupedArgs {
  const int32_t* seg_offsets;
  const void *dy_c, *x_c, *h_c, *phi_c, *w_gate_up, *w_down;
  int32_t E, H, I;
  int64_t cap;
  float *dw_gate_up, *dw_down;
  void *dh_c, *dx_c;
  int32_t* status;
  float* row_dot;   // optional [cap]: dphi . phi per retained row
  float* dot_part;  // scratch for row_dot: [cap][dot_parts_max(I)]
  // Compaction-free variant (kept_pair non-null): x_c, h_c, phi_c are not used; their rows are
  // read from x [T,H] (token u / k), h [P,2I] and phi [P,I] (pair u = kept_pair[r]).
  const int32_t* kept_pair;
  int32_t k;
  const void *x, *h, *phi;
  int64_t n_pairs;  // T*k: rows of h and phi; a kept_pair entry outside [0, n_pairs) is not followed
};

// Parts of the dphi . phi row sums: one per 128 output columns (tensor-core path) or per 64
// (CUDA-core path); scratch is sized for the larger count.
inline int dot_parts_max(int32_t I) { return (I + 63) / 64; }
void launch_row_dot(const float* part, int n_part, const int32_t* seg_offsets, int32_t E, int64_t cap,
                    float* row_dot, cudaStream_t s);
void launch_router_grad(const int32_t* row_of_pair, const float* alpha, const float* row_dot, int64_t P,
                        int64_t cap, float* dalpha, cudaStream_t s);

void launch_grouped_simt(const GroupedArgs& a, lrm_dtype dt, cudaStream_t s);

// The saved forward state of the retained rows, recomputed from x_c (lrm_recompute_forward).
struct RecomputeArgs {
  const int32_t* seg_offsets;
  const void *x_c, *w_gate_up;
  int32_t E, H, I;
  int64_t cap;
  void *h_c, *phi_c;
  int32_t* status;
};
lrm_status launch_recompute_tc(const RecomputeArgs& a, const GemmWs& ws, cudaStream_t s);
void launch_recompute_simt(const RecomputeArgs& a, lrm_dtype dt, cudaStream_t s);
// Returns LRM_OK, or LRM_ERR_UNSUPPORTED / LRM_ERR_CUDA when the tensor-core path cannot run.
lrm_status launch_grouped_tc(const GroupedArgs& a, const GemmWs& ws, cudaStream_t s);
lrm_status launch_wait_selftest(int32_t* status, int64_t limit_ns, cudaStream_t s);

// Tokens sorted by expert (lrm_sort_tokens), and the weighted way back with its gradient.
struct SortArgs {
  const int32_t* topk_idx;
  const void* x;
  int64_t T;
  int32_t k, E, H;
  int32_t *seg_offsets, *pair_of_row, *row_of_pair;
  void* x_s;        // optional
  int32_t* counts;  // scratch [chunks][E + 1]
  int32_t* loads;   // scratch [E + 1]
  int32_t* status;
};
bool sort_in_one_launch(int64_t T, int32_t k, int32_t E);
bool sort_self_counted(int64_t T, int32_t k);  // up to so many pairs the ranking counts them itself
bool sort_needs_scratch(int64_t T, int32_t k, int32_t E);
int sort_chunk_tokens(int32_t k);  // tokens of a chunk of the multi-launch form
lrm_status launch_sort_tokens(const SortArgs& a, lrm_dtype dt, cudaStream_t s);
void launch_combine(const int32_t* row_of_pair, const float* alpha, const void* y_s, const void* residual, int64_t T,
                    int32_t k, int32_t H, lrm_dtype dt, int64_t cap, void* y, int32_t* status, cudaStream_t s);
void launch_combine_backward(const int32_t* row_of_pair, const float* alpha, const void* dy, const void* y_s, int64_t T,
                             int32_t k, int32_t H, lrm_dtype dt, int64_t cap, void* dy_s, float* dalpha,
                             int32_t* status, cudaStream_t s);

// lrm_linear and its gradients.  seg_offsets is NULL for one dense product (E = 1).
struct LinearArgs {
  const int32_t* seg_offsets;
  const void *x, *w, *bias, *residual;  // bias, residual optional
  int64_t R;
  int32_t E, N, K;  // N: columns of y (w has 2N rows per expert for SwiGLU)
  lrm_act act;
  void *y, *z;  // z optional: the pre-activation
  int32_t* status;
};
void launch_linear_simt(const LinearArgs& a, lrm_dtype dt, lrm_dtype out_dt, cudaStream_t s);
// Whether one pass over the weights by plain loads takes a product of so few rows, not the tensor cores' tiles
// of 256 rows.  GB300, us, rows kernel : tiles.
// Dense, up to 32 rows (fp32 24).  bf16, weights 1408+1408 x 4096 (SwiGLU), 4096 x 4096, 768+768 x 2048: 12.4 : 17.4,
// 12.8 : 15.6, 6.5 : 10.3 at 32 rows, 20.7 : 17.4, 22.1 : 15.6, 9.2 : 10.3 at 64; fp32 the same at 24 rows 52 : 50,
// 53 : 70, 21 : 23.
// Per expert, bf16, up to 64 rows in all: 128 experts of 768+768 x 2048, popularity even and zipf 1, 65 : 66 and
// 36 : 42 at 64 rows, 101 : 92 and 51 : 46 at 128; 42 experts of 232 x 1472 8.8 : 11 and 9.2 : 10.4 at 84.
// Per expert, fp32, up to 8 rows a mean expert (the tiles split every expert's weights first): 128 experts
// 502 : 1599 and 532 : 1238 at 1024 rows, 42 experts 32 : 69 and 58 : 68 at 336, 46 : 71 and 99 : 70 at 672.
inline bool linear_few_rows(int64_t R, int32_t E, bool grouped, lrm_dtype dt) {
  if (!grouped) return R <= (dt == LRM_F32 ? 24 : 32);
  return R <= 32 || (dt == LRM_F32 ? R <= 8 * (int64_t)E : R <= 64);
}
void launch_linear_rows(const LinearArgs& a, lrm_dtype dt, lrm_dtype out_dt, cudaStream_t s);
// ws: for bf16 inputs NULL, or room for linear_extra_bytes.
lrm_status launch_linear_tc(const LinearArgs& a, lrm_dtype dt, lrm_dtype out_dt, void* ws, cudaStream_t s);
size_t linear_planes_bytes(int64_t rows, int64_t cols);  // an fp32 operand as three bf16 planes
size_t linear_plan_bytes(int32_t E);                     // plan and expert maps of the weights' gradient
// scratch beside the planes: parts of a long reduction, or weights copied to aligned rows (forward); parts (dx)
size_t linear_extra_bytes(int64_t R, int32_t E, int32_t NP, int32_t K, lrm_dtype dt);
size_t linear_grad_parts_bytes(int64_t R, int32_t E, int32_t N, int32_t K, lrm_dtype dt);
// weight gradients per expert cut into runs of rows: segments in the plan, and bytes of the runs
int linear_grad_segments(int64_t R, int32_t E, int32_t N, int32_t K, lrm_dtype dt);
size_t linear_grad_runs_bytes(int64_t R, int32_t E, int32_t N, int32_t K, lrm_dtype dt);
int linear_grad_parts(int64_t R, int32_t N, int32_t K);  // parts of the dense weights' gradient, summed apart
struct LinearGradArgs {
  const int32_t* seg_offsets;
  const void *dz, *x, *w;
  int64_t R;
  int32_t E, N, K;  // N: columns of dz (rows of w)
  void* dx;         // optional
  float* dw;        // optional
  int32_t* status;
};
void launch_linear_backward_simt(const LinearGradArgs& a, lrm_dtype dt, cudaStream_t s);
lrm_status launch_linear_backward_tc(const LinearGradArgs& a, lrm_dtype dt, void* ws, cudaStream_t s);
struct ActGradArgs {
  const int32_t* seg_offsets;
  const void *dy, *z;
  int64_t R;
  int32_t E, N;
  lrm_act act;
  void* dz;
  float* db;    // optional
  float* part;  // scratch [act_backward_part_rows][columns of dz], only with db
  int32_t* status;
};
size_t act_backward_part_rows(int64_t R, int32_t E);
void launch_act_backward(const ActGradArgs& a, lrm_dtype dt, cudaStream_t s);

}  // namespace lrm
