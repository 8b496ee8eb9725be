// Gradient of the router: gates, load-balancing loss and z-loss, and the projection.
//
// With z [T, E] the logits, S_t the selected experts, p = softmax(z_t), dg the gates'
// gradients and c = (c0, c1) the upstream gradients of the two losses:
//   gates over the selected logits (MOE_GATE_TOPK_SOFTMAX; the renormalised mode is the
//   same function of z: p_s / sum_S p = softmax over S):
//       dz_s = g_s (dg_s - sum_j g_j dg_j)                        for s in S_t
//   raw gates g_s = p_s:  dz_i = p_i ([i in S_t] dg_i - sum_s p_s dg_s)
//   aux = alpha E sum_i f_i P_i, f held fixed:
//       dz_i += c0 alpha E / T p_i (f_i - sum_j f_j p_j)
//   z_loss = mean_t lse_t^2:  dz_i += c1 2 / T lse_t p_i
//   dW = dz^T x, db = sum_t dz (also the logit bias's), dx = dz W.
// dz is fp32; the two products run on CUDA cores (fp32 layers) or, with dz split into bf16
// terms, on the tensor cores. The sums over tokens are split into pieces whose partial
// sums a second kernel adds in a fixed order.
#include "grad.cuh"
#include "grad_simt.cuh"

namespace moe {

namespace {

constexpr int kMaxBlocks = 1184;  // of k_dlogits: eight per SM

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// dz as bf16 terms: each the rounding of what the ones before it leave
__device__ __forceinline__ void split_terms(float v, __nv_bfloat16 (&t)[kSplit]) {
#pragma unroll
  for (int i = 0; i < kSplit; ++i) {
    t[i] = __float2bfloat16_rn(v);
    const float r = __bfloat162float(t[i]);
    v = isinf(r) ? 0.f : v - r;  // an infinite value has no remainder
  }
}

// A warp per token (blocks stride over the tokens): lane l holds experts l + 32 j, j <
// kEpl. With TC dz also goes out as bf16 terms, and the first block writes the tables of
// the tensor-core products.
template <int kEpl, bool TC>
__global__ void __launch_bounds__(256) k_dlogits(RouteBwdArgs a, float *db_part, RouteTcArgs tc) {
  __shared__ float red[8][32 * kEpl];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int E = a.E, k = a.k;
  if (TC && blockIdx.x == 0) {
    const int slices = ceil_div(a.T, 64), per = ceil_div(slices, tc.pieces);
    for (int i = threadIdx.x; i <= tc.pieces; i += 256) tc.piece[i] = 64 * min(slices, i * per);
    if (threadIdx.x == 0) {
      tc.all[0] = tc.all_rows[0] = 0;
      tc.all[1] = 64 * slices;
      tc.all_rows[1] = a.T;
    }
  }
  const bool losses = a.d_losses != nullptr;
  const bool need_p = losses || a.gate_mode == MOE_GATE_SOFTMAX_TOPK_RAW;
  const float c0 = losses ? a.d_losses[0] * a.alpha * (float)E / (float)a.T : 0.f;
  const float c1 = losses ? a.d_losses[1] * 2.f / (float)a.T : 0.f;
  float f[kEpl], db[kEpl];
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
    const int e = lane + 32 * j;
    db[j] = 0.f;
    f[j] = (losses && e < E) ? (float)a.counts[e] / ((float)a.T * (float)k) : 0.f;
  }
  for (int t = blockIdx.x * 8 + warp; t < a.T; t += gridDim.x * 8) {
    const float *zt = a.logits + (size_t)t * E;
    // the slots: lane s < k
    int idx = -1;
    float dg = 0.f, zs = neg_inf();
    if (lane < k) {
      const size_t q = (size_t)t * k + lane;
      idx = a.topk_idx[q];
      if (idx < 0 || idx >= E) {
        report_error(a.err, MOE_DEVERR_EXPERT_INDEX, (int32_t)q);
        idx = -1;
      }
      if (idx >= 0) {
        zs = zt[idx];
        if (a.row_dot) {
          const int r = a.inv[q];
          dg = (r >= 0 && r < a.R) ? a.row_dot[r] : 0.f;
        } else if (a.dgate) {
          dg = a.dgate[q];
        }
      }
    }
    float p[kEpl], dz[kEpl];
#pragma unroll
    for (int j = 0; j < kEpl; ++j) p[j] = dz[j] = 0.f;
    float ds = 0.f;  // this lane's slot: what its expert's logit gets
    if (need_p) {
      float m = neg_inf();
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        const int e = lane + 32 * j;
        p[j] = e < E ? zt[e] : neg_inf();
        m = fmaxf(m, p[j]);
      }
      m = warp_max(m);
      if (m > neg_inf()) {  // a token whose logits are all -inf has no probabilities
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
          p[j] = lane + 32 * j < E ? expf(p[j] - m) : 0.f;
          sum += p[j];
        }
        sum = warp_sum(sum);
        const float inv = 1.f / sum, lse = m + logf(sum);
        float pf = 0.f;
#pragma unroll
        for (int j = 0; j < kEpl; ++j) {
          p[j] *= inv;
          pf = fmaf(p[j], f[j], pf);
        }
        if (losses) {
          pf = warp_sum(pf);
#pragma unroll
          for (int j = 0; j < kEpl; ++j) dz[j] = p[j] * (c0 * (f[j] - pf) + c1 * lse);
        }
        if (a.gate_mode == MOE_GATE_SOFTMAX_TOPK_RAW) {
          const float ps = idx >= 0 ? expf(zs - m) * inv : 0.f;
          ds = ps * dg;
          const float sd = warp_sum(ds);
#pragma unroll
          for (int j = 0; j < kEpl; ++j) dz[j] = fmaf(-p[j], sd, dz[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kEpl; ++j) p[j] = 0.f;
      }
    }
    if (a.gate_mode != MOE_GATE_SOFTMAX_TOPK_RAW) {
      const float m = warp_max(zs);
      const float ex = (idx >= 0 && m > neg_inf()) ? expf(zs - m) : 0.f;
      const float sum = warp_sum(ex);
      const float gt = sum > 0.f ? ex / sum : ex;  // a NaN logit stays one
      const float gd = warp_sum(gt * dg);
      ds = gt * (dg - gd);
    }
    for (int s = 0; s < k; ++s) {
      const int e = __shfl_sync(0xffffffffu, idx, s);
      const float v = __shfl_sync(0xffffffffu, ds, s);
#pragma unroll
      for (int j = 0; j < kEpl; ++j)
        if (e == lane + 32 * j) dz[j] += v;
    }
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
      const int e = lane + 32 * j;
      if (e < E && a.dlogits) a.dlogits[(size_t)t * E + e] = dz[j];
      db[j] += dz[j];
      if (TC && e < tc.Ep) {
        __nv_bfloat16 part[kSplit];
        split_terms(e < E ? dz[j] : 0.f, part);
#pragma unroll
        for (int i = 0; i < kSplit; ++i)
          if (tc.term[i]) tc.term[i][(size_t)t * tc.Ep + e] = part[i];
      }
    }
  }
  if (db_part == nullptr) return;
#pragma unroll
  for (int j = 0; j < kEpl; ++j) red[warp][lane + 32 * j] = db[j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][e];
    db_part[(size_t)blockIdx.x * E + e] = v;
  }
}

// Few experts (EP >= E, at most kFewExperts): both products on CUDA cores in one pass over
// x. A thread owns VC columns and keeps their EP rows of W and of dW in registers; the
// block walks over its piece of the tokens with dz broadcast from shared memory. 4 E flops
// per element of x: up to E = 16 the reads of x and the writes of dx bound it.
constexpr int kFewExperts = 32;
constexpr int kProjThreads = 128, kProjTokens = 32;

template <typename T, int VC>
__device__ __forceinline__ void load_cols(const T *p, float (&f)[VC]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (VC == 4) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
      f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
      const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
      f[0] = v.x; f[1] = v.y;
    }
  } else {
    uint32_t u[VC / 2];
    if constexpr (VC == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
      u[0] = v.x; u[1] = v.y;
    } else {
      u[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
#pragma unroll
    for (int i = 0; i < VC / 2; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <typename T, int EP, int VC>
__global__ void __launch_bounds__(kProjThreads) k_route_proj(const T *x, const T *w,
                                                             const float *dz, float *dx,
                                                             float *dw_part, int n_tok, int d,
                                                             int E, int per) {
  __shared__ __align__(16) float zs[kProjTokens][EP];
  const int tid = threadIdx.x;
  const int col = (blockIdx.x * kProjThreads + tid) * VC;
  const bool live = col < d;
  pdl_wait();
  pdl_trigger();
  float wr[EP][VC], acc[EP][VC];
#pragma unroll
  for (int e = 0; e < EP; ++e) {
#pragma unroll
    for (int c = 0; c < VC; ++c) wr[e][c] = acc[e][c] = 0.f;
    if (dx && live && e < E) load_cols<T, VC>(w + (size_t)e * d + col, wr[e]);
  }
  const int t0 = blockIdx.y * per, t1 = min(n_tok, t0 + per);
  for (int tb = t0; tb < t1; tb += kProjTokens) {
    const int n = min(kProjTokens, t1 - tb);
    __syncthreads();
    for (int i = tid; i < kProjTokens * EP; i += kProjThreads) {
      const int u = i / EP, e = i % EP;
      zs[u][e] = (u < n && e < E) ? dz[(size_t)(tb + u) * E + e] : 0.f;
    }
    __syncthreads();
    if (!live) continue;
    constexpr int NB = 4;  // tokens requested before any is used
    for (int u0 = 0; u0 < n; u0 += NB) {
      float xv[NB][VC];
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (dw_part && u0 + i < n) load_cols<T, VC>(x + (size_t)(tb + u0 + i) * d + col, xv[i]);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (u0 + i >= n) break;
        float o[VC], z[EP];
#pragma unroll
        for (int e = 0; e < EP; e += 4) {
          const float4 q = *reinterpret_cast<const float4 *>(&zs[u0 + i][e]);
          z[e] = q.x; z[e + 1] = q.y; z[e + 2] = q.z; z[e + 3] = q.w;
        }
        if (dx) {
#pragma unroll
          for (int c = 0; c < VC; ++c) {
            o[c] = 0.f;
#pragma unroll
            for (int e = 0; e < EP; ++e) o[c] = fmaf(z[e], wr[e][c], o[c]);
          }
          float *out = dx + (size_t)(tb + u0 + i) * d + col;
          if constexpr (VC == 4)
            *reinterpret_cast<float4 *>(out) = make_float4(o[0], o[1], o[2], o[3]);
          else
            *reinterpret_cast<float2 *>(out) = make_float2(o[0], o[1]);
        }
        if (dw_part) {
#pragma unroll
          for (int e = 0; e < EP; ++e)
#pragma unroll
            for (int c = 0; c < VC; ++c) acc[e][c] = fmaf(z[e], xv[i][c], acc[e][c]);
        }
      }
    }
  }
  if (dw_part && live) {
#pragma unroll
    for (int e = 0; e < EP; ++e)
      if (e < E) {
        float *out = dw_part + ((size_t)blockIdx.y * E + e) * d + col;
#pragma unroll
        for (int c = 0; c < VC; ++c) out[c] = acc[e][c];
      }
  }
}

// dw[i] = sum over the pieces of part [pieces, n], and (the last E blocks) db[e] = the
// sum of the blocks' partials, each in a fixed order
template <typename T>
__global__ void __launch_bounds__(128) k_route_sums(const float *part, int pieces, size_t n, T *dw,
                                                    int dw_blocks, const float *db_part, int blocks,
                                                    int E, float *db) {
  __shared__ float red[4];
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < dw_blocks) {  // n is a multiple of 4
    const size_t i = ((size_t)blockIdx.x * 128 + threadIdx.x) * 4;
    if (i >= n) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < pieces; ++s) {
      const float4 p = __ldg(reinterpret_cast<const float4 *>(part + (size_t)s * n + i));
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    dw[i] = Elem<T>::from_f(v.x);
    dw[i + 1] = Elem<T>::from_f(v.y);
    dw[i + 2] = Elem<T>::from_f(v.z);
    dw[i + 3] = Elem<T>::from_f(v.w);
    return;
  }
  const int e = blockIdx.x - dw_blocks;
  float v = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < blocks; i += 128) v += db_part[(size_t)i * E + e];
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) db[e] = (red[0] + red[1]) + (red[2] + red[3]);
}

int dlogits_blocks(int T) {
  const int b = ceil_div(T, 8);
  return b < kMaxBlocks ? b : kMaxBlocks;
}

// pieces of the tokens for dW: enough tiles for two per SM
int dw_pieces(int T, int d, int E) {
  const int tiles = ceil_div(E, simt::BM) * ceil_div(d, simt::BN);
  int s = 296 / tiles;
  if (s < 1) s = 1;
  const int most = ceil_div(T, 64);
  return s < most ? s : most;
}

// ... with the CTA-pair tiles: one per pair, K long enough to pay for the reduction
int dw_pieces_tc(int T, int d) {
  const int s = 74 / ceil_div(d, 256), most = ceil_div(T, 256);
  return s < 1 ? 1 : (s < most ? s : most);
}

// ... of k_route_proj: three blocks per SM (as many as its registers let it hold), at
// least sixteen tokens each
int proj_cols(int E) { return E <= 16 ? 4 : 2; }
int proj_pieces(int T, int d, int E) {
  const int s = 148 * 3 / ceil_div(d, kProjThreads * proj_cols(E)), most = ceil_div(T, 16);
  return s < 1 ? 1 : (s < most ? s : most);
}

int e_padded(int E) { return (E + 63) / 64 * 64; }

template <bool TC>
cudaError_t dlogits(const RouteBwdArgs &a, float *db_part, const RouteTcArgs &tc, cudaStream_t st) {
  const dim3 g(dlogits_blocks(a.T)), b(256);
  const int cols = TC ? tc.Ep : a.E;
  if (cols <= 32) return launch_pdl(k_dlogits<1, TC>, g, b, 0, st, a, db_part, tc);
  if (cols <= 64) return launch_pdl(k_dlogits<2, TC>, g, b, 0, st, a, db_part, tc);
  if (cols <= 128) return launch_pdl(k_dlogits<4, TC>, g, b, 0, st, a, db_part, tc);
  return launch_pdl(k_dlogits<8, TC>, g, b, 0, st, a, db_part, tc);
}

template <typename T>
cudaError_t sums(const RouteBwdArgs &a, const float *dw_part, int pieces, const float *db_part,
                 cudaStream_t st) {
  const size_t n = a.dw ? (size_t)a.E * a.d : 0;
  const int dw_blocks = (int)((n / 4 + 127) / 128), db_blocks = a.db ? a.E : 0;
  if (dw_blocks + db_blocks == 0) return cudaSuccess;
  return launch_pdl(k_route_sums<T>, dim3(dw_blocks + db_blocks), dim3(128), 0, st, dw_part, pieces,
                    n, static_cast<T *>(a.dw), dw_blocks, db_part, dlogits_blocks(a.T), a.E, a.db);
}

template <typename T>
cudaError_t route_bwd_few(const RouteBwdArgs &a, cudaStream_t st) {
  float *db_part = static_cast<float *>(a.part);
  cudaError_t e = dlogits<false>(a, a.db ? db_part : nullptr, RouteTcArgs{}, st);
  if (e != cudaSuccess) return e;
  const int pieces = proj_pieces(a.T, a.d, a.E);
  float *dw_part = db_part + (size_t)kMaxBlocks * a.E;
  if (a.dx || a.dw) {
    const dim3 g(ceil_div(a.d, kProjThreads * proj_cols(a.E)), pieces), b(kProjThreads);
    const T *x = static_cast<const T *>(a.x), *w = static_cast<const T *>(a.w);
    auto run = [&](auto kernel) {
      return launch_pdl(kernel, g, b, 0, st, x, w, (const float *)a.dlogits, a.dx,
                        a.dw ? dw_part : static_cast<float *>(nullptr), a.T, a.d, a.E,
                        ceil_div(a.T, pieces));
    };
    e = a.E <= 8 ? run(k_route_proj<T, 8, 4>)
                 : (a.E <= 16 ? run(k_route_proj<T, 16, 4>) : run(k_route_proj<T, 32, 2>));
    if (e != cudaSuccess) return e;
  }
  return sums<T>(a, dw_part, pieces, db_part, st);
}

// fp32, more experts: tiles on CUDA cores
cudaError_t route_bwd_simt(const RouteBwdArgs &a, cudaStream_t st) {
  float *db_part = static_cast<float *>(a.part);
  const dim3 b(256);
  cudaError_t e = dlogits<false>(a, a.db ? db_part : nullptr, RouteTcArgs{}, st);
  if (e != cudaSuccess) return e;
  const float *x = static_cast<const float *>(a.x), *w = static_cast<const float *>(a.w);
  if (a.dx) {
    simt::Gemm<float, float, float> m{};
    m.a[0] = a.dlogits;
    m.b[0] = w;
    m.c[0] = a.dx;
    m.M[0] = a.T;
    m.N[0] = m.ldb[0] = a.d;
    m.lda[0] = a.E;
    m.nseg = 1;
    m.K = a.E;
    m.G = 1;
    e = launch_pdl(simt::k_gemm<float, float, float, false>,
                   dim3(ceil_div(a.d, simt::BN), ceil_div(a.T, simt::BM)), b, 0, st, m);
    if (e != cudaSuccess) return e;
  }
  const int pieces = dw_pieces(a.T, a.d, a.E);
  float *dw_part = db_part + (size_t)kMaxBlocks * a.E;
  if (a.dw) {
    simt::Gemm<float, float, float> m{};
    m.a[0] = a.dlogits;
    m.b[0] = x;
    m.c[0] = dw_part;
    m.M[0] = m.lda[0] = a.E;
    m.N[0] = m.ldb[0] = a.d;
    m.nseg = 1;
    m.K = a.T;
    m.chunk = ceil_div(a.T, pieces);
    m.G = pieces;
    e = launch_pdl(simt::k_gemm<float, float, float, true>,
                   dim3(ceil_div(a.d, simt::BN), ceil_div(a.E, simt::BM), pieces), b, 0, st, m);
    if (e != cudaSuccess) return e;
  }
  return sums<float>(a, dw_part, pieces, db_part, st);
}

// bf16 scratch: tables | db partials | dW partials | terms
struct TcScratch {
  size_t tables, db, dw, term, term_bytes, total;
};
TcScratch tc_scratch(int T, int d, int E) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  TcScratch s;
  s.tables = 0;
  s.db = up((kMaxExperts + 1 + 4) * 4);
  s.dw = s.db + up((size_t)kMaxBlocks * E * 4);
  s.term = s.dw + up((size_t)dw_pieces_tc(T, d) * E * d * 4);
  s.term_bytes = up((size_t)T * e_padded(E) * 2);
  s.total = s.term + kSplit * s.term_bytes;
  return s;
}

cudaError_t route_bwd_tc(const RouteBwdArgs &a, cudaStream_t st) {
  const TcScratch s = tc_scratch(a.T, a.d, a.E);
  char *base = static_cast<char *>(a.part);
  float *db_part = reinterpret_cast<float *>(base + s.db);
  RouteTcArgs tc{};
  tc.x = a.x;
  tc.w = a.w;
  const int terms = a.dx ? kSplit : (a.dw ? kSplitDw : 0);
  for (int i = 0; i < terms; ++i)
    tc.term[i] = reinterpret_cast<__nv_bfloat16 *>(base + s.term + i * s.term_bytes);
  tc.all = reinterpret_cast<int32_t *>(base);
  tc.all_rows = tc.all + 2;
  tc.piece = tc.all + 4;
  tc.dx = a.dx;
  tc.dw_part = reinterpret_cast<float *>(base + s.dw);
  tc.T = a.T;
  tc.d = a.d;
  tc.E = a.E;
  tc.Ep = e_padded(a.E);
  tc.pieces = dw_pieces_tc(a.T, a.d);
  tc.err = a.err;
  cudaError_t e = terms ? dlogits<true>(a, a.db ? db_part : nullptr, tc, st)
                        : dlogits<false>(a, a.db ? db_part : nullptr, tc, st);
  if (e != cudaSuccess) return e;
  if (a.dx) {
    e = launch_route_dx_tc(tc, st);
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    e = launch_route_dw_tc(tc, st);
    if (e != cudaSuccess) return e;
  }
  return sums<__nv_bfloat16>(a, tc.dw_part, tc.pieces, db_part, st);
}

}  // namespace

size_t route_bwd_scratch_bytes(int T, int d, int E, int dtype) {
  if (T < 1) T = 1;
  if (E > kFewExperts && dtype != MOE_DTYPE_F32) return tc_scratch(T, d, E).total;
  const int pieces = E <= kFewExperts ? proj_pieces(T, d, E) : dw_pieces(T, d, E);
  return sizeof(float) * ((size_t)kMaxBlocks * E + (size_t)pieces * E * d);
}

cudaError_t launch_route_bwd(const RouteBwdArgs &a, int dtype, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const bool f32 = dtype == MOE_DTYPE_F32;
  if (a.E <= kFewExperts) return f32 ? route_bwd_few<float>(a, st) : route_bwd_few<__nv_bfloat16>(a, st);
  return f32 ? route_bwd_simt(a, st) : route_bwd_tc(a, st);
}

}  // namespace moe
