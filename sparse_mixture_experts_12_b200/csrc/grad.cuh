// Internal launch interface of the layer's gradients (see the files named below).
#pragma once

#include "kernels.cuh"

namespace moe {

// ------------------------------------------------------------- token_grad.cu
struct CombineBwdArgs {
  const void *dy;        // [T, d] dtype
  const void *y_perm;    // [R, d] dtype (read when dgate is given)
  const int32_t *inv;    // [T*k]
  const float *gate;     // [T*k] (read when dy_perm is given)
  void *dy_perm;         // [R, d] dtype or nullptr
  float *dgate;          // [T*k] or nullptr
  int T, d, k, R;
  int32_t *err;
};
cudaError_t launch_combine_bwd(const CombineBwdArgs &a, int dtype, cudaStream_t st);

struct PermuteBwdArgs {
  const void *dx_perm;   // [R, d]: dtype, or fp32 when dx_perm_f32
  int dx_perm_f32;
  const int32_t *inv;    // [T*k]
  const float *add0;     // [T, d] fp32 or nullptr
  const float *add1;     // [T, d] fp32 or nullptr
  void *dx;              // [T, d] dtype
  int T, d, k, R;
  int32_t *err;
};
cudaError_t launch_permute_bwd(const PermuteBwdArgs &a, int dtype, cudaStream_t st);

// x and dy rows to every kept slot's row, and the slot's gate to row_w [R]
struct GatherRowsArgs {
  const void *x, *dy;    // [T, d] dtype
  const int32_t *inv;    // [T*k]
  const float *gate;     // [T*k]
  void *x_perm, *dy_perm;  // [R, d] dtype
  float *row_w;          // [R]
  int T, k, R, row_bytes;
  int32_t *err;
};
cudaError_t launch_gather_rows(const GatherRowsArgs &a, cudaStream_t st);

// ------------------------------------------------------------- route_grad.cu
struct RouteBwdArgs {
  const void *x;             // [T, d] dtype
  const void *w;             // [E, d] dtype
  const float *logits;       // [T, E]
  const int32_t *topk_idx;   // [T, k]
  const int32_t *counts;     // [E] (read when d_losses is given)
  const float *dgate;        // [T, k] or nullptr
  const float *row_dot;      // [R] or nullptr: dgate[t,s] = row_dot[inv[t,s]]
  const int32_t *inv;        // [T*k] (with row_dot)
  const float *d_losses;     // [2] or nullptr
  float *dlogits;            // [T, E]
  float *dx;                 // [T, d] fp32 or nullptr
  void *dw;                  // [E, d] dtype or nullptr
  float *db;                 // [E] or nullptr
  void *part;                // scratch of route_bwd_scratch_bytes()
  int T, d, E, k, gate_mode, R;
  float alpha;
  int32_t *err;
};
size_t route_bwd_scratch_bytes(int T, int d, int E, int dtype);
cudaError_t launch_route_bwd(const RouteBwdArgs &a, int dtype, cudaStream_t st);

// --------------------------------------------------------------- ffn_grad.cu
// Gradient of the grouped expert FFN (see GroupedFfnArgs). The pre-activations are
// recomputed. With row_w the rows' output is weighted: dy is the gradient of
// w_r E(x_r), and row_dot[r] = <dy_r, E(x_r)> is the gradient of w_r.
struct FfnGradArgs {
  const void *x, *dy;        // [rows, d] dtype
  int rows;                  // rows allocated in x, dy, dx and the scratch
  const int32_t *offsets;    // [G+1] checked (all zero when the caller's were invalid)
  const int32_t *mprefix;    // [G+1]
  int G, m_tiles_ub, d, F, act;
  const void *w1, *w3, *w2;
  const float *b1, *b2;
  const float *row_w;        // [rows] or nullptr
  float *row_dot;            // [rows] or nullptr
  float *dot_part;           // [ceil(F / 64), rows] scratch (with row_dot)
  void *h, *dg, *du;         // [rows, F] dtype scratch: w h, w dg, w du
  void *dx;                  // [rows, d] or nullptr
  int dx_f32;
  void *dw1, *dw3, *dw2;     // [G, F, d], [G, F, d], [G, d, F] dtype, or nullptr
  float *db1, *db2;          // [G, F], [G, d] fp32, or nullptr
  float *col_part;           // [m_tiles_ub, max(F, d)] scratch (with db1 or db2)
  int32_t *err;
};
cudaError_t launch_ffn_bwd(const FfnGradArgs &a, int dtype, cudaStream_t st);
// offsets -> checked copy and tile prefix
cudaError_t launch_grad_tables(const int32_t *offsets, int G, int max_rows, int32_t *checked,
                               int32_t *mprefix, int32_t *err, cudaStream_t st);
// one group of n rows: offsets {0, n} and its tile prefix
cudaError_t launch_one_group(int n, int32_t *offsets, int32_t *mprefix, cudaStream_t st);

}  // namespace moe
