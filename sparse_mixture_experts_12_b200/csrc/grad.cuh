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

// The experts' rows of x and dy in the padded layout of the experts' gradients: expert
// g's rows begin at poff[g], rows up to poff[g+1] are zero (see launch_grad_tables).
struct PadRowsArgs {
  const void *x, *dy;      // [R, d] expert-contiguous rows, or [T, d] with inv
  const int32_t *inv;      // [T*k] or nullptr; with it also:
  const float *gate;       //   [T*k]
  float *row_w;            //   [poff[G]] each row's gate, 0 for a padding row
  int32_t *inv_pad;        //   [T*k] inv in the padded layout (-1: no row)
  int T, k;
  int R;                   // rows that offsets may name
  const int32_t *offsets, *poff;  // [G+1] checked
  int G, rows;             // rows: bound of poff[G]
  void *x_pad, *dy_pad;    // [rows, d]
  int row_bytes;
  int32_t *err;
};
cudaError_t launch_pad_rows(const PadRowsArgs &a, cudaStream_t st);

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
  float *dlogits;            // [T, E]; nullptr unless route_bwd_reads_dlogits()
  float *dx;                 // [T, d] fp32 or nullptr
  void *dw;                  // [E, d] dtype or nullptr
  float *db;                 // [E] or nullptr
  void *part;                // scratch of route_bwd_scratch_bytes()
  int T, d, E, k, gate_mode, R;
  float alpha;
  int32_t *err;
};
// The projection's gradients on the tensor cores (bf16), in ffn_grad_tc.cu: dz as a sum of
// bf16 terms, rounded one after another. dx takes three (dz to its last bit: the result
// stays fp32), dW two (2^-16 of dz, far below the rounding of the result to bf16).
constexpr int kSplit = 3, kSplitDw = 2;
struct RouteTcArgs {
  const void *x, *w;           // [T, d], [E, d]
  __nv_bfloat16 *terms;        // [T, kSplit, Ep], Ep = E rounded up to 64 (zeros behind E)
  int32_t *all, *all_rows, *all_tiles;  // {0, T rounded up to 64}, {0, T}, {0, 256-row tiles}
  int32_t *piece;              // [pieces + 1] first tokens (multiples of 64) of the pieces of dW
  float *dx, *dw_part;         // [T, d]; [pieces, kSplitDw, Ep, d]: a sum for each term; either
                               // may be nullptr
  int T, d, E, Ep, pieces;
  int32_t *err;
};
cudaError_t launch_route_tc(const RouteTcArgs &a, cudaStream_t st);
// whether the launch needs RouteBwdArgs::dlogits (else it may be nullptr: the tensor cores
// read dz from its terms)
bool route_bwd_reads_dlogits(int E, int dtype);
size_t route_bwd_scratch_bytes(int T, int d, int E, int dtype);
cudaError_t launch_route_bwd(const RouteBwdArgs &a, int dtype, cudaStream_t st);

// -------------------------------------------- ffn_grad.cu, ffn_grad_tc.cu
// Gradient of the grouped expert FFN (see GroupedFfnArgs). The pre-activations are
// recomputed. With row_w the rows' output is weighted: dy is the gradient of
// w_r E(x_r), and row_dot[r] = <dy_r, E(x_r)> is the gradient of w_r.
struct FfnGradArgs {
  const void *x, *dy;        // [x_rows, d] dtype
  int x_rows;                // rows allocated in x and dy (rows past the experts' are zero
                             // up to the padding, or not allocated)
  int rows;                  // rows allocated in the scratch, row_w and row_dot
  long long row_bound;       // rows the experts may have in all
  const int32_t *offsets;    // [G+1] checked (all zero when the caller's were invalid):
                             // expert g has offsets[g+1] - offsets[g] rows
  const int32_t *poff;       // [G+1] its first row in all arrays but dx
  const int32_t *dx_off;     // [G+1] its first row in dx: offsets or poff
  const int32_t *mprefix;    // [G+1] prefix of the experts' tile_rows-row tiles
  const int32_t *pre256;     // [G+1] prefix of their 256-row tiles
  int tile_rows;             // 8, 32 or 128, see grad_tile_rows()
  int G, m_tiles_ub, pair_tiles_ub;  // bounds of those tiles and of the 256-row tiles
  int d, F, act;
  const void *w1, *w3, *w2;
  const float *b1, *b2;
  const float *row_w;        // [rows] or nullptr
  float *row_dot;            // [rows] or nullptr
  float *dot_part;           // [ceil(F / 32), rows] scratch (with row_dot)
  void *h, *dg, *du;         // [rows, F] dtype scratch: w h, w dg, w du
  void *dx;                  // [dx_rows, d] or nullptr
  float *dx_part;            // [dx_splits() or dx_splits_tc(), rows, d] scratch
  int dx_f32, dx_rows;
  void *dw1, *dw3, *dw2;     // [G, F, d], [G, F, d], [G, d, F] dtype, or nullptr
  float *db1, *db2;          // [G, F], [G, d] fp32, or nullptr
  float *col_part, *part2;   // scratch of col_part_rows() x F (with db1), m_tiles_ub x d (db2)
  int32_t *err;
};
cudaError_t launch_ffn_bwd(const FfnGradArgs &a, int dtype, cudaStream_t st);
// its steps on the tensor cores (bf16)
cudaError_t launch_act_grad_tc(const FfnGradArgs &a, cudaStream_t st);
// splits > 1: dx in parts (fp32, the padded rows) to dx_part [splits, rows, d]
cudaError_t launch_products_tc(const FfnGradArgs &a, int splits, cudaStream_t st);

// Rows to which each expert's are padded: the K slice of the tensor-core products of the
// weights' gradients (bf16), none on CUDA cores.
inline int row_pad(int dtype) { return dtype == MOE_DTYPE_F32 ? 1 : 64; }
// bound of the padded rows of at most R rows of G experts
inline long long padded_rows_ub(long long R, int G, int pad) {
  const long long r = R + (long long)(pad - 1) * (R < G ? R : G);
  return (r + pad - 1) / pad * pad;
}
// Rows of a tile of the CUDA-core products (and of a partial of db2): fewer where experts
// average fewer rows, so that small experts do not pay for empty ones.
inline int grad_tile_rows(long long rows, int G) {
  return rows <= 8LL * G ? 8 : (rows < 64LL * G ? 32 : 128);
}
// Pieces of F that dx's tiles on CUDA cores are split into: two blocks an SM, with a
// reduction of at least 256 each; and at most 1024 products in one running sum (two for
// each index with SwiGLU), whose fp32 error grows with the root of their number (2.3e-6 of
// the result after 13008 of them, where sums of 1024 keep it near 5e-7) while the parts take
// no more than 256 MB.
inline int dx_splits(long long rows, int m_tiles, int d, int F, bool glu) {
  const long long tiles = (long long)m_tiles * ceil_div(d, 64);
  const int most = F / 256 > 1 ? F / 256 : 1;
  const long long fill = tiles > 0 ? (296 + tiles - 1) / tiles : 1;
  const int s = fill < most ? (int)fill : most;
  const long long fit = (256ll << 20) / (4 * (rows > 0 ? rows : 1) * d);
  const long long exact = ceil_div(F, glu ? 512 : 1024);
  const long long more = exact < fit ? exact : fit;
  return s > more ? s : (int)more;
}
// ... and its CTA-pair tiles (bf16): where they leave half of the pairs without one, into as
// many as fill them, of sixteen 64-wide slices at least. (Two rows of two experts of 64 x
// 7104: 222 slices one after another took 78 of 88 us.)
inline int dx_splits_tc(int pair_tiles, int d, int F, bool glu) {
  const long long tiles = (long long)pair_tiles * ceil_div(d, 256);
  const int slices = (glu ? 2 : 1) * ceil_div(F, 64);
  if (tiles == 0 || 2 * tiles > 74 || slices < 32) return 1;
  const int fill = (int)(74 / tiles), s = fill < slices / 16 ? fill : slices / 16;
  return ceil_div(slices, ceil_div(slices, s));  // none of them empty
}
inline int grad_tiles_ub(long long rows, int G, int unit) {
  return (int)(rows / unit + (rows < G ? rows : G));
}
// partials of db1: one per row tile, or (bf16) one per 32 padded rows
inline long long col_part_rows(long long rows, int m_tiles, int dtype) {
  return dtype == MOE_DTYPE_F32 ? m_tiles : rows / 32;
}
// offsets -> checked copy, tile prefix and the padded first rows
cudaError_t launch_grad_tables(const int32_t *offsets, int G, int max_rows, int unit, int pad,
                               int32_t *checked, int32_t *mprefix, int32_t *pre256, int32_t *poff,
                               int32_t *err, cudaStream_t st);
// the tables of one group of n rows
cudaError_t launch_one_group(int n, int unit, int pad, int32_t *offsets, int32_t *mprefix,
                             int32_t *pre256, int32_t *poff, cudaStream_t st);

}  // namespace moe
