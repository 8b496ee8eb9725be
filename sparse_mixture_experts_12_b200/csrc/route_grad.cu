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
// Everything is fp32. The sums over tokens are split into pieces whose partial sums a
// second kernel adds in a fixed order.
#include "grad.cuh"
#include "grad_simt.cuh"

namespace moe {

namespace {

constexpr int kMaxBlocks = 592;  // of k_dlogits: four per SM
constexpr int kEpl = kMaxExperts / 32;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// A warp per token (blocks stride over the tokens): lane l holds experts l + 32 j.
__global__ void __launch_bounds__(256) k_dlogits(RouteBwdArgs a, float *db_part) {
  __shared__ float red[8][kMaxExperts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int E = a.E, k = a.k;
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
      if (e < E) a.dlogits[(size_t)t * E + e] = dz[j];
      db[j] += dz[j];
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

// out[i] = sum over the pieces of part [pieces, n], in order
template <typename T>
__global__ void __launch_bounds__(256) k_sum_pieces(const float *part, int pieces, size_t n,
                                                    T *out) {
  pdl_wait();
  pdl_trigger();
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int s = 0; s < pieces; ++s) v += part[(size_t)s * n + i];
  out[i] = Elem<T>::from_f(v);
}

// db [E] from the blocks' sums: a block per expert
__global__ void __launch_bounds__(128) k_db(const float *part, int blocks, int E, float *db) {
  __shared__ float red[4];
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.x;
  float v = 0.f;
  for (int i = threadIdx.x; i < blocks; i += 128) v += part[(size_t)i * E + e];
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

template <typename T>
cudaError_t route_bwd(const RouteBwdArgs &a, cudaStream_t st) {
  float *db_part = static_cast<float *>(a.part);
  const int blocks = dlogits_blocks(a.T);
  const dim3 b(256);
  cudaError_t e = launch_pdl(k_dlogits, dim3(blocks), b, 0, st, a,
                             a.db ? db_part : static_cast<float *>(nullptr));
  if (e != cudaSuccess) return e;
  if (a.db) {
    e = launch_pdl(k_db, dim3(a.E), dim3(128), 0, st, (const float *)db_part, blocks, a.E, a.db);
    if (e != cudaSuccess) return e;
  }
  const T *x = static_cast<const T *>(a.x), *w = static_cast<const T *>(a.w);
  if (a.dx) {
    simt::Gemm<float, T, float> m{};
    m.a[0] = a.dlogits;
    m.b[0] = w;
    m.c[0] = a.dx;
    m.M[0] = a.T;
    m.N[0] = m.ldb[0] = a.d;
    m.lda[0] = a.E;
    m.nseg = 1;
    m.K = a.E;
    m.G = 1;
    e = launch_pdl(simt::k_gemm<float, T, float, false>,
                   dim3(ceil_div(a.d, simt::BN), ceil_div(a.T, simt::BM)), b, 0, st, m);
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    const int pieces = dw_pieces(a.T, a.d, a.E);
    const size_t n = (size_t)a.E * a.d;
    float *dw_part = db_part + (size_t)kMaxBlocks * a.E;
    simt::Gemm<float, T, float> m{};
    m.a[0] = a.dlogits;
    m.b[0] = x;
    m.c[0] = dw_part;
    m.M[0] = m.lda[0] = a.E;
    m.N[0] = m.ldb[0] = a.d;
    m.nseg = 1;
    m.K = a.T;
    m.chunk = ceil_div(a.T, pieces);
    m.G = pieces;
    e = launch_pdl(simt::k_gemm<float, T, float, true>,
                   dim3(ceil_div(a.d, simt::BN), ceil_div(a.E, simt::BM), pieces), b, 0, st, m);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_sum_pieces<T>, dim3((unsigned)((n + 255) / 256)), b, 0, st,
                   (const float *)dw_part, pieces, n, static_cast<T *>(a.dw));
  }
  return e;
}

}  // namespace

size_t route_bwd_scratch_bytes(int T, int d, int E, int dtype) {
  (void)dtype;
  return sizeof(float) * ((size_t)kMaxBlocks * E + (size_t)dw_pieces(T > 0 ? T : 1, d, E) * E * d);
}

cudaError_t launch_route_bwd(const RouteBwdArgs &a, int dtype, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  return dtype == MOE_DTYPE_F32 ? route_bwd<float>(a, st) : route_bwd<__nv_bfloat16>(a, st);
}

}  // namespace moe
