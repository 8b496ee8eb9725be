// C ABI of the layer's gradients: host-side validation, workspace layout and the
// launch sequences.
#include "api.cuh"
#include "grad.cuh"

namespace moe {

namespace {

enum Buf {
  G_ERR, G_OFFSETS, G_MPREFIX, G_PRE256, G_POFF, G_SH, G_H, G_DG, G_DU,
  G_COL, G_COL2, G_DLOGITS, G_ROUTE, G_X, G_DY, G_INV, G_DX, G_DX_PART, G_ROW_W, G_ROW_DOT,
  G_DOT_PART, G_DX_ROUTER, G_DX_SHARED, G_NBUF
};

struct Layout {
  size_t off[G_NBUF];
  size_t total;
};

size_t elem_bytes(const moe_cfg_t &c) { return c.dtype == MOE_DTYPE_F32 ? 4 : 2; }

// rows of the experts' padded buffers
long long scratch_rows(const moe_cfg_t &c) {
  return padded_rows_ub(expert_rows(c), c.n_experts, row_pad(c.dtype));
}

int tile_rows(const moe_cfg_t &c) { return grad_tile_rows(expert_rows(c), c.n_experts); }

size_t larger(size_t a, size_t b) { return a > b ? a : b; }

Layout layout_for(const moe_cfg_t &c) {
  const size_t T = (size_t)c.n_tokens, E = (size_t)c.n_experts;
  const size_t d = (size_t)c.d_model, F = (size_t)c.d_ff;
  const size_t eb = elem_bytes(c);
  const size_t Fs = (size_t)c.n_shared * (size_t)c.d_ff_shared;
  const bool glu = c.act == MOE_ACT_SWIGLU;
  const bool tc = !expert_choice(c);  // moe_backward's own buffers: token choice
  // the experts' rows, padded; the shared experts run after the routed ones, in the same
  // h / dg / du
  const size_t R = (size_t)scratch_rows(c), Ts = (size_t)padded_rows_ub(c.n_tokens, 1, row_pad(c.dtype));
  const size_t act = larger(R * F, Ts * Fs);
  const int tiles = grad_tiles_ub(expert_rows(c), c.n_experts, tile_rows(c));
  const bool copies = c.dtype != MOE_DTYPE_F32 || tc;  // of x and dy rows
  size_t sz[G_NBUF];
  sz[G_ERR] = 4 * sizeof(int32_t);
  sz[G_OFFSETS] = sz[G_MPREFIX] = sz[G_PRE256] = sz[G_POFF] = (E + 1) * 4;
  sz[G_SH] = 4 * 2 * 4;  // the same tables of the shared experts' one group
  sz[G_H] = act * eb;
  sz[G_DG] = act * eb;
  sz[G_DU] = (glu || Fs ? act : 0) * eb;
  sz[G_COL] = glu ? 0 : (size_t)col_part_rows((long long)R, tiles, c.dtype) * F * 4;
  sz[G_COL2] = glu ? 0 : (size_t)tiles * d * 4;
  sz[G_DLOGITS] = tc && route_bwd_reads_dlogits(c.n_experts, c.dtype) ? T * E * 4 : 0;
  sz[G_ROUTE] = tc ? route_bwd_scratch_bytes(c.n_tokens, c.d_model, c.n_experts, c.dtype) : 0;
  sz[G_X] = copies ? R * d * eb : 0;
  sz[G_DY] = copies ? R * d * eb : 0;
  sz[G_INV] = tc ? T * (size_t)c.top_k * 4 : 0;
  sz[G_DX] = tc ? R * d * 4 : 0;
  const int us = grad_tile_rows(c.n_tokens, 1);
  const int pt = grad_tiles_ub(expert_rows(c), c.n_experts, 2 * kRowTile);
  const int pt_sh = ceil_div(c.n_tokens, 2 * kRowTile);
  size_t parts, parts_sh;  // of dx: the routed experts', the shared experts'
  if (c.dtype == MOE_DTYPE_F32) {
    parts = (size_t)dx_splits((long long)R, tiles, c.d_model, c.d_ff, glu);
    parts_sh = (size_t)dx_splits(c.n_tokens, ceil_div(c.n_tokens, us), c.d_model, (int)Fs, true);
  } else {
    parts = (size_t)dx_splits_tc(pt, c.d_model, c.d_ff, glu);
    parts_sh = (size_t)dx_splits_tc(pt_sh, c.d_model, (int)Fs, true);
  }
  sz[G_DX_PART] = larger(parts > 1 ? parts * R : 0, Fs && parts_sh > 1 ? parts_sh * Ts : 0) * d * 4;
  sz[G_ROW_W] = tc ? R * 4 : 0;
  sz[G_ROW_DOT] = tc ? R * 4 : 0;
  sz[G_DOT_PART] = tc ? R * (size_t)ceil_div(c.d_ff, 32) * 4 : 0;
  sz[G_DX_ROUTER] = tc ? T * d * 4 : 0;
  sz[G_DX_SHARED] = Fs ? T * d * 4 : 0;
  Layout L;
  size_t o = 0;
  for (int i = 0; i < G_NBUF; ++i) {
    L.off[i] = o;
    o += align256(sz[i]);
  }
  L.total = o;
  return L;
}

template <typename P>
P *at(void *ws, const Layout &L, Buf b) {
  return reinterpret_cast<P *>(static_cast<char *>(ws) + L.off[b]);
}

moe_status_t check_ws(const moe_cfg_t *c, const void *ws, size_t ws_bytes) {
  if (ws == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
  if (ws_bytes < layout_for(*c).total) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// what every gradient of the token movement and the routing starts with
moe_status_t check_token_choice(const moe_cfg_t *cfg, const void *ws, size_t ws_bytes) {
  MOE_TRY(check_cfg(cfg));
  MOE_TRY(check_ws(cfg, ws, ws_bytes));
  return expert_choice(*cfg) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

moe_status_t check_expert_grads(const moe_cfg_t &c, const moe_weights_t *w, const moe_grads_t &g) {
  const bool glu = c.act == MOE_ACT_SWIGLU;
  if (!glu && g.w3) return MOE_ERR_INVALID_ARG;
  if ((g.b1 && !w->b1) || (g.b2 && !w->b2)) return MOE_ERR_INVALID_ARG;
  return check_ptrs({{g.w1, false}, {g.w3, false}, {g.w2, false}, {g.b1, false}, {g.b2, false}});
}

moe_status_t zero(void *p, size_t bytes, cudaStream_t st) {
  return p ? cuda_status(cudaMemsetAsync(p, 0, bytes, st)) : MOE_OK;
}

// gradients over no tokens
moe_status_t zero_router_grads(const moe_cfg_t &c, const moe_grads_t &g, cudaStream_t st) {
  MOE_TRY(zero(g.w_router, (size_t)c.n_experts * c.d_model * elem_bytes(c), st));
  return zero(g.b_router, (size_t)c.n_experts * 4, st);
}
moe_status_t zero_expert_grads(const moe_cfg_t &c, const moe_grads_t &g, cudaStream_t st) {
  const size_t E = (size_t)c.n_experts, d = (size_t)c.d_model, F = (size_t)c.d_ff;
  MOE_TRY(zero(g.w1, E * F * d * elem_bytes(c), st));
  MOE_TRY(zero(g.w3, E * F * d * elem_bytes(c), st));
  MOE_TRY(zero(g.w2, E * F * d * elem_bytes(c), st));
  MOE_TRY(zero(g.b1, E * F * 4, st));
  return zero(g.b2, E * d * 4, st);
}

FfnGradArgs expert_args(const moe_cfg_t &c, const moe_weights_t &w, const moe_grads_t &g, void *ws,
                        const Layout &L) {
  FfnGradArgs a{};
  a.rows = a.x_rows = (int)scratch_rows(c);
  a.row_bound = expert_rows(c);
  a.offsets = at<int32_t>(ws, L, G_OFFSETS);
  a.mprefix = at<int32_t>(ws, L, G_MPREFIX);
  a.pre256 = at<int32_t>(ws, L, G_PRE256);
  a.poff = at<int32_t>(ws, L, G_POFF);
  a.G = c.n_experts;
  a.tile_rows = tile_rows(c);
  a.m_tiles_ub = grad_tiles_ub(expert_rows(c), c.n_experts, a.tile_rows);
  a.pair_tiles_ub = grad_tiles_ub(expert_rows(c), c.n_experts, 2 * kRowTile);
  a.d = c.d_model;
  a.F = c.d_ff;
  a.act = c.act;
  a.w1 = w.w1;
  a.w3 = w.w3;
  a.w2 = w.w2;
  a.b1 = w.b1;
  a.b2 = w.b2;
  a.h = at<void>(ws, L, G_H);
  a.dg = at<void>(ws, L, G_DG);
  a.du = at<void>(ws, L, G_DU);
  a.col_part = at<float>(ws, L, G_COL);
  a.part2 = at<float>(ws, L, G_COL2);
  a.dx_part = at<float>(ws, L, G_DX_PART);
  a.dw1 = g.w1;
  a.dw3 = g.w3;
  a.dw2 = g.w2;
  a.db1 = g.b1;
  a.db2 = g.b2;
  a.err = at<int32_t>(ws, L, G_ERR);
  return a;
}

moe_status_t expert_tables(const moe_cfg_t &c, const int32_t *offsets, void *ws, const Layout &L,
                           cudaStream_t st) {
  return cuda_status(launch_grad_tables(
      offsets, c.n_experts, (int)expert_rows(c), tile_rows(c), row_pad(c.dtype),
      at<int32_t>(ws, L, G_OFFSETS), at<int32_t>(ws, L, G_MPREFIX), at<int32_t>(ws, L, G_PRE256),
      at<int32_t>(ws, L, G_POFF), at<int32_t>(ws, L, G_ERR), st));
}

// copies of the experts' rows of x and dy, padded
PadRowsArgs pad_args(const moe_cfg_t &c, const void *x, const void *dy, void *ws, const Layout &L) {
  PadRowsArgs a{};
  a.x = x;
  a.dy = dy;
  a.R = (int)expert_rows(c);
  a.offsets = at<int32_t>(ws, L, G_OFFSETS);
  a.poff = at<int32_t>(ws, L, G_POFF);
  a.G = c.n_experts;
  a.rows = (int)scratch_rows(c);
  a.x_pad = at<void>(ws, L, G_X);
  a.dy_pad = at<void>(ws, L, G_DY);
  a.row_bytes = (int)(c.d_model * elem_bytes(c));
  a.err = at<int32_t>(ws, L, G_ERR);
  return a;
}

RouteBwdArgs route_args(const moe_cfg_t &c, void *ws, const Layout &L) {
  RouteBwdArgs a{};
  a.T = c.n_tokens;
  a.d = c.d_model;
  a.E = c.n_experts;
  a.k = c.top_k;
  a.R = c.n_tokens * c.top_k;
  a.gate_mode = c.gate_mode;
  a.alpha = c.aux_alpha;
  if (route_bwd_reads_dlogits(c.n_experts, c.dtype)) a.dlogits = at<float>(ws, L, G_DLOGITS);
  a.part = at<void>(ws, L, G_ROUTE);
  a.err = at<int32_t>(ws, L, G_ERR);
  return a;
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status_t moe_backward_workspace_size(const moe_cfg_t *cfg, size_t *bytes) {
  MOE_TRY(check_cfg(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = layout_for(*cfg).total;
  return MOE_OK;
}

MOE_API moe_status_t moe_combine_backward(const moe_cfg_t *cfg, const void *dy,
                                          const void *y_perm, const int32_t *inv,
                                          const float *topk_gate, void *dy_perm, float *dgate,
                                          void *ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(check_token_choice(cfg, ws, ws_bytes));
  if (cfg->n_tokens == 0) return MOE_OK;
  MOE_TRY(check_ptrs({{dy, true}, {inv, true}, {y_perm, dgate != nullptr},
                      {topk_gate, dy_perm != nullptr}, {dy_perm, false}, {dgate, false}}));
  const moe_cfg_t &c = *cfg;
  CombineBwdArgs a{};
  a.dy = dy;
  a.y_perm = y_perm;
  a.inv = inv;
  a.gate = topk_gate;
  a.dy_perm = dy_perm;
  a.dgate = dgate;
  a.T = c.n_tokens;
  a.d = c.d_model;
  a.k = c.top_k;
  a.R = c.n_tokens * c.top_k;
  a.err = at<int32_t>(ws, layout_for(c), G_ERR);
  return cuda_status(launch_combine_bwd(a, c.dtype, stream));
}

MOE_API moe_status_t moe_permute_backward(const moe_cfg_t *cfg, const void *dx_perm,
                                          const int32_t *inv, const float *dx_add, void *dx,
                                          void *ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(check_token_choice(cfg, ws, ws_bytes));
  if (cfg->n_tokens == 0) return MOE_OK;
  MOE_TRY(check_ptrs({{dx_perm, true}, {inv, true}, {dx_add, false}, {dx, true}}));
  const moe_cfg_t &c = *cfg;
  PermuteBwdArgs a{};
  a.dx_perm = dx_perm;
  a.inv = inv;
  a.add0 = dx_add;
  a.dx = dx;
  a.T = c.n_tokens;
  a.d = c.d_model;
  a.k = c.top_k;
  a.R = c.n_tokens * c.top_k;
  a.err = at<int32_t>(ws, layout_for(c), G_ERR);
  return cuda_status(launch_permute_bwd(a, c.dtype, stream));
}

MOE_API moe_status_t moe_route_backward(const moe_cfg_t *cfg, const moe_weights_t *w,
                                        const void *x, const float *logits,
                                        const int32_t *topk_idx, const int32_t *counts,
                                        const float *dgate, const float *d_losses,
                                        float *dlogits, float *dx, const moe_grads_t *grads,
                                        void *ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(check_token_choice(cfg, ws, ws_bytes));
  moe_grads_t g{};
  if (grads) g = *grads;
  MOE_TRY(check_ptrs({{g.w_router, false}, {g.b_router, false}, {dlogits, false}, {dx, false}}));
  if (cfg->n_tokens == 0) return zero_router_grads(*cfg, g, stream);
  if (dx != nullptr && w == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ptrs({{logits, true}, {topk_idx, true}, {dgate, false},
                      {counts, d_losses != nullptr}, {x, g.w_router != nullptr},
                      {w ? w->w_router : nullptr, dx != nullptr}}));
  if (!aligned(d_losses, 4)) return MOE_ERR_MISALIGNED;
  const moe_cfg_t &c = *cfg;
  RouteBwdArgs a = route_args(c, ws, layout_for(c));
  a.x = x;
  a.w = w ? w->w_router : nullptr;
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.counts = counts;
  a.dgate = dgate;
  a.d_losses = d_losses;
  if (dlogits) a.dlogits = dlogits;
  a.dx = dx;
  a.dw = g.w_router;
  a.db = g.b_router;
  return cuda_status(launch_route_bwd(a, c.dtype, stream));
}

MOE_API moe_status_t moe_expert_ffn_backward(const moe_cfg_t *cfg, const moe_weights_t *w,
                                             const void *x_perm, const int32_t *offsets,
                                             const void *dy_perm, void *dx_perm,
                                             const moe_grads_t *grads, void *ws,
                                             size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(check_cfg(cfg));
  MOE_TRY(check_ws(cfg, ws, ws_bytes));
  MOE_TRY(check_expert_weights(cfg, w));
  const moe_cfg_t &c = *cfg;
  moe_grads_t g{};
  if (grads) g = *grads;
  MOE_TRY(check_expert_grads(c, w, g));
  if (expert_rows(c) == 0) return zero_expert_grads(c, g, stream);
  MOE_TRY(check_ptrs({{x_perm, true}, {offsets, true}, {dy_perm, true}, {dx_perm, false}}));
  const Layout L = layout_for(c);
  FfnGradArgs a = expert_args(c, *w, g, ws, L);
  MOE_TRY(expert_tables(c, offsets, ws, L, stream));
  if (row_pad(c.dtype) == 1) {
    a.x = x_perm;
    a.dy = dy_perm;
  } else {
    const PadRowsArgs p = pad_args(c, x_perm, dy_perm, ws, L);
    MOE_CUDA(launch_pad_rows(p, stream));
    a.x = p.x_pad;
    a.dy = p.dy_pad;
  }
  a.dx = dx_perm;
  a.dx_off = a.offsets;
  a.dx_rows = (int)expert_rows(c);
  return cuda_status(launch_ffn_bwd(a, c.dtype, stream));
}

MOE_API moe_status_t moe_backward(const moe_cfg_t *cfg, const moe_weights_t *w, const void *x,
                                  const moe_taps_t *taps, const void *dy, const float *d_losses,
                                  void *dx, const moe_grads_t *grads, void *ws, size_t ws_bytes,
                                  moe_stream_t stream) {
  MOE_TRY(check_token_choice(cfg, ws, ws_bytes));
  const moe_cfg_t &c = *cfg;
  MOE_TRY(check_expert_weights(cfg, w));
  MOE_TRY(check_shared_weights(cfg, w));
  moe_grads_t g{};
  if (grads) g = *grads;
  MOE_TRY(check_expert_grads(c, w, g));
  if (c.n_shared == 0 && (g.ws_gate || g.ws_up || g.ws_down)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ptrs({{g.w_router, false}, {g.b_router, false}, {g.ws_gate, false},
                      {g.ws_up, false}, {g.ws_down, false}, {dx, false}}));
  const size_t fs = (size_t)c.n_shared * c.d_ff_shared * c.d_model * elem_bytes(c);
  if (c.n_tokens == 0) {
    MOE_TRY(zero_router_grads(c, g, stream));
    MOE_TRY(zero_expert_grads(c, g, stream));
    MOE_TRY(zero(g.ws_gate, fs, stream));
    MOE_TRY(zero(g.ws_up, fs, stream));
    return zero(g.ws_down, fs, stream);
  }
  if (taps == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ptrs({{x, true}, {dy, true}, {w->w_router, dx != nullptr}, {taps->logits, true},
                      {taps->topk_idx, true}, {taps->topk_gate, true}, {taps->offsets, true},
                      {taps->inv, true}, {taps->counts, d_losses != nullptr}}));
  if (!aligned(d_losses, 4)) return MOE_ERR_MISALIGNED;
  const Layout L = layout_for(c);
  // 1. the experts' rows of x and dy, and each row's gate
  FfnGradArgs a = expert_args(c, *w, g, ws, L);
  MOE_TRY(expert_tables(c, taps->offsets, ws, L, stream));
  PadRowsArgs gr = pad_args(c, x, dy, ws, L);
  gr.inv = taps->inv;
  gr.gate = taps->topk_gate;
  gr.row_w = at<float>(ws, L, G_ROW_W);
  gr.inv_pad = at<int32_t>(ws, L, G_INV);
  gr.T = c.n_tokens;
  gr.k = c.top_k;
  MOE_CUDA(launch_pad_rows(gr, stream));
  // 2. the routed experts; the gates' gradient comes from their rows
  const bool router = dx || g.w_router || g.b_router;
  a.x = gr.x_pad;
  a.dy = gr.dy_pad;
  a.row_w = gr.row_w;
  a.row_dot = router ? at<float>(ws, L, G_ROW_DOT) : nullptr;
  a.dot_part = at<float>(ws, L, G_DOT_PART);
  a.dx = dx ? at<void>(ws, L, G_DX) : nullptr;
  a.dx_f32 = 1;
  a.dx_off = a.poff;
  a.dx_rows = a.rows;
  MOE_CUDA(launch_ffn_bwd(a, c.dtype, stream));
  // 3. the router
  if (router) {
    RouteBwdArgs r = route_args(c, ws, L);
    r.x = x;
    r.w = w->w_router;
    r.logits = taps->logits;
    r.topk_idx = taps->topk_idx;
    r.counts = taps->counts;
    r.row_dot = a.row_dot;
    r.inv = gr.inv_pad;
    r.R = a.rows;
    r.d_losses = d_losses;
    r.dx = dx ? at<float>(ws, L, G_DX_ROUTER) : nullptr;
    r.dw = g.w_router;
    r.db = g.b_router;
    MOE_CUDA(launch_route_bwd(r, c.dtype, stream));
  }
  // 4. the always-on shared experts: one group of all tokens, F concatenated
  float *dx_shared = nullptr;
  if (c.n_shared > 0 && (dx || g.ws_gate || g.ws_up || g.ws_down)) {
    FfnGradArgs s{};
    s.tile_rows = grad_tile_rows(c.n_tokens, 1);
    int32_t *tab = at<int32_t>(ws, L, G_SH);
    MOE_CUDA(launch_one_group(c.n_tokens, s.tile_rows, row_pad(c.dtype), tab, tab + 2, tab + 4,
                              tab + 6, stream));
    s.x = x;
    s.dy = dy;
    s.x_rows = c.n_tokens;  // the padding rows lie past the operands' bounds: read as zero
    s.rows = (int)padded_rows_ub(c.n_tokens, 1, row_pad(c.dtype));
    s.row_bound = c.n_tokens;
    s.offsets = tab;
    s.mprefix = tab + 2;
    s.pre256 = tab + 4;
    s.poff = s.dx_off = tab + 6;
    s.G = 1;
    s.m_tiles_ub = ceil_div(c.n_tokens, s.tile_rows);
    s.pair_tiles_ub = ceil_div(c.n_tokens, 2 * kRowTile);
    s.d = c.d_model;
    s.F = c.n_shared * c.d_ff_shared;
    s.act = MOE_ACT_SWIGLU;
    s.w1 = w->ws_gate;
    s.w3 = w->ws_up;
    s.w2 = w->ws_down;
    s.h = at<void>(ws, L, G_H);
    s.dg = at<void>(ws, L, G_DG);
    s.du = at<void>(ws, L, G_DU);
    s.dx = dx_shared = dx ? at<float>(ws, L, G_DX_SHARED) : nullptr;
    s.dx_part = at<float>(ws, L, G_DX_PART);
    s.dx_f32 = 1;
    s.dx_rows = c.n_tokens;
    s.dw1 = g.ws_gate;
    s.dw3 = g.ws_up;
    s.dw2 = g.ws_down;
    s.err = a.err;
    MOE_CUDA(launch_ffn_bwd(s, c.dtype, stream));
  }
  // 5. the tokens' gradient: their experts' rows, the router's and the shared share
  if (dx) {
    PermuteBwdArgs p{};
    p.dx_perm = a.dx;
    p.dx_perm_f32 = 1;
    p.inv = gr.inv_pad;
    p.add0 = at<float>(ws, L, G_DX_ROUTER);
    p.add1 = dx_shared;
    p.dx = dx;
    p.T = c.n_tokens;
    p.d = c.d_model;
    p.k = c.top_k;
    p.R = a.rows;
    p.err = a.err;
    MOE_CUDA(launch_permute_bwd(p, c.dtype, stream));
  }
  return MOE_OK;
}
