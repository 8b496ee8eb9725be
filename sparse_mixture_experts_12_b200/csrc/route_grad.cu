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

// LPT lanes per token, eight consecutive experts each: a warp works on 32 / LPT tokens at
// once, reductions over the experts take log2(LPT) exchanges, and rows move in 16-byte
// pieces (a warp per token took 17 us on 16384 tokens of 128 experts, this 13, bound by its
// instructions). Every lane goes through the token's slots by itself. With TC dz also goes out as
// bf16 terms, and the first block writes the tables of the tensor-core products.
constexpr int kDzThreads = 128, kEpl = 8;

template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int LPT, bool TC>
__global__ void __launch_bounds__(kDzThreads, 8) k_dlogits(RouteBwdArgs a, float *db_part,
                                                        RouteTcArgs tc) {
  constexpr int kTokens = kDzThreads / LPT, kWarps = kDzThreads / 32;
  __shared__ float red[kWarps][LPT * kEpl];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = threadIdx.x % LPT, e0 = sub * kEpl;
  pdl_wait();
  pdl_trigger();
  const int E = a.E, k = a.k;
  if (TC && blockIdx.x == 0) {
    const int slices = ceil_div(a.T, 64), per = ceil_div(slices, tc.pieces);
    for (int i = threadIdx.x; i <= tc.pieces; i += kDzThreads)
      tc.piece[i] = 64 * min(slices, i * per);
    if (threadIdx.x == 0) {
      tc.all[0] = tc.all_rows[0] = tc.all_tiles[0] = 0;
      tc.all[1] = 64 * slices;
      tc.all_rows[1] = a.T;
      tc.all_tiles[1] = ceil_div(a.T, 256);
    }
  }
  const bool losses = a.d_losses != nullptr, raw = a.gate_mode == MOE_GATE_SOFTMAX_TOPK_RAW;
  const bool need_p = losses || raw, vec = (E & 3) == 0;
  const float c0 = losses ? a.d_losses[0] * a.alpha * (float)E / (float)a.T : 0.f;
  const float c1 = losses ? a.d_losses[1] * 2.f / (float)a.T : 0.f;
  float f[kEpl], db[kEpl];
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
    db[j] = 0.f;
    f[j] = (losses && e0 + j < E) ? (float)a.counts[e0 + j] / ((float)a.T * (float)k) : 0.f;
  }
  for (int base = blockIdx.x * kTokens; base < a.T; base += gridDim.x * kTokens) {
    const int t = base + threadIdx.x / LPT;
    const bool live = t < a.T;
    const float *zt = a.logits + (size_t)(live ? t : 0) * E;
    float p[kEpl], dz[kEpl];
#pragma unroll
    for (int j = 0; j < kEpl; ++j) {
      p[j] = neg_inf();
      dz[j] = 0.f;
    }
    if (need_p && live) {
#pragma unroll
      for (int j = 0; j < kEpl; j += 4) {
        if (vec && e0 + j < E) {
          const float4 q = __ldg(reinterpret_cast<const float4 *>(zt + e0 + j));
          p[j] = q.x; p[j + 1] = q.y; p[j + 2] = q.z; p[j + 3] = q.w;
        } else if (!vec) {
#pragma unroll
          for (int i = j; i < j + 4; ++i)
            if (e0 + i < E) p[i] = __ldg(zt + e0 + i);
        }
      }
    }
    // the slots: expert, logit, and the gate's gradient
    int idx[kMaxTopK];
    float zs[kMaxTopK], ds[kMaxTopK];
#pragma unroll
    for (int s = 0; s < kMaxTopK; ++s) {
      idx[s] = -1;
      zs[s] = neg_inf();
      ds[s] = 0.f;
      if (s < k && live) {
        const size_t q = (size_t)t * k + s;
        idx[s] = __ldg(a.topk_idx + q);
        if (idx[s] < 0 || idx[s] >= E) {
          if (sub == 0) report_error(a.err, MOE_DEVERR_EXPERT_INDEX, (int32_t)q);
          idx[s] = -1;
        } else {
          zs[s] = __ldg(zt + idx[s]);
          if (a.row_dot) {
            const int r = a.inv[q];
            ds[s] = (r >= 0 && r < a.R) ? a.row_dot[r] : 0.f;
          } else if (a.dgate) {
            ds[s] = __ldg(a.dgate + q);
          }
        }
      }
    }
    float m = neg_inf(), inv = 0.f;  // of all experts
    if (need_p) {
#pragma unroll
      for (int j = 0; j < kEpl; ++j) m = fmaxf(m, p[j]);
      m = group_max<LPT>(m);
      // a token whose logits are all -inf has no probabilities
      const float top = m > neg_inf() ? m : 0.f;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        p[j] = e0 + j < E ? expf(p[j] - top) : 0.f;
        sum += p[j];
      }
      sum = group_sum<LPT>(sum);
      const bool some = m > neg_inf();
      inv = some ? 1.f / sum : 0.f;
      const float lse = some ? m + logf(sum) : 0.f;
      float pf = 0.f;
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        p[j] = some ? p[j] * inv : 0.f;
        pf = fmaf(p[j], f[j], pf);
      }
      if (losses) {
        pf = group_sum<LPT>(pf);
#pragma unroll
        for (int j = 0; j < kEpl; ++j) dz[j] = p[j] * (c0 * (f[j] - pf) + c1 * lse);
      }
    }
    if (raw) {
      float sd = 0.f;
#pragma unroll
      for (int s = 0; s < kMaxTopK; ++s)
        if (s < k) {
          const float ps = (idx[s] >= 0 && m > neg_inf()) ? expf(zs[s] - m) * inv : 0.f;
          ds[s] *= ps;
          sd += ds[s];
        }
#pragma unroll
      for (int j = 0; j < kEpl; ++j) dz[j] = fmaf(-p[j], sd, dz[j]);
    } else {
      float ms = neg_inf(), sum = 0.f, gd = 0.f;
#pragma unroll
      for (int s = 0; s < kMaxTopK; ++s)
        if (s < k) ms = fmaxf(ms, zs[s]);
#pragma unroll
      for (int s = 0; s < kMaxTopK; ++s)
        if (s < k) {
          zs[s] = (idx[s] >= 0 && ms > neg_inf()) ? expf(zs[s] - ms) : 0.f;
          sum += zs[s];
        }
      const float is = sum != 0.f ? 1.f / sum : 0.f;  // a NaN logit stays one
#pragma unroll
      for (int s = 0; s < kMaxTopK; ++s)
        if (s < k) {
          zs[s] *= is;
          gd = fmaf(zs[s], ds[s], gd);
        }
#pragma unroll
      for (int s = 0; s < kMaxTopK; ++s)
        if (s < k) ds[s] = zs[s] * (ds[s] - gd);
    }
#pragma unroll
    for (int s = 0; s < kMaxTopK; ++s)
      if (s < k) {
#pragma unroll
        for (int j = 0; j < kEpl; ++j)
          if (idx[s] == e0 + j) dz[j] += ds[s];
      }
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < kEpl; ++j) db[j] += dz[j];
    if (a.dlogits) {
      float *out = a.dlogits + (size_t)t * E + e0;
#pragma unroll
      for (int j = 0; j < kEpl; j += 4) {
        if (vec && e0 + j < E) {
          *reinterpret_cast<float4 *>(out + j) =
              make_float4(dz[j], dz[j + 1], dz[j + 2], dz[j + 3]);
        } else if (!vec) {
#pragma unroll
          for (int i = j; i < j + 4; ++i)
            if (e0 + i < E) out[i] = dz[i];
        }
      }
    }
    if (TC && e0 < tc.Ep) {
      __nv_bfloat16 part[kSplit][kEpl];
#pragma unroll
      for (int j = 0; j < kEpl; ++j) {
        __nv_bfloat16 q[kSplit];
        split_terms(e0 + j < E ? dz[j] : 0.f, q);
#pragma unroll
        for (int i = 0; i < kSplit; ++i) part[i][j] = q[i];
      }
#pragma unroll
      for (int i = 0; i < kSplit; ++i)
        *reinterpret_cast<uint4 *>(tc.terms + ((size_t)t * kSplit + i) * tc.Ep + e0) =
            *reinterpret_cast<const uint4 *>(part[i]);
    }
  }
  if (db_part == nullptr) return;
#pragma unroll
  for (int j = 0; j < kEpl; ++j) {
#pragma unroll
    for (int o = 16; o >= LPT; o >>= 1) db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
    if (lane < LPT) red[warp][e0 + j] = db[j];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kDzThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][e];
    db_part[(size_t)blockIdx.x * E + e] = v;
  }
}

// Few experts (EP >= E, see few_experts()): both products on CUDA cores in one pass over
// x. A thread owns VC columns and keeps their EP rows of W and of dW in registers; the
// block walks over its piece of the tokens with dz broadcast from shared memory: 100 MB in
// 25 us on 4096 tokens of 4096, bound by latency (four blocks an SM of 55 tokens each; two,
// three, eight and twelve were slower).
constexpr int kProjThreads = 128, kProjTokens = 128, kProjCols = 4;

// VC values of type T as they lie in memory, and unpacked
template <typename T, int VC>
struct Cols {
  uint32_t u[VC * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T *p) {
    constexpr int n = VC * sizeof(T) / 4;
    if constexpr (n == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
      u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    } else {
      static_assert(n == 2, "8 or 16 bytes");
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
      u[0] = v.x; u[1] = v.y;
    }
  }
  __device__ __forceinline__ float get(int c) const {
    if (sizeof(T) == 4) return __uint_as_float(u[c]);
    return __uint_as_float((c & 1) ? u[c / 2] & 0xffff0000u : u[c / 2] << 16);
  }
};

template <typename T, int EP>
__global__ void __launch_bounds__(kProjThreads) k_route_proj(const T *x, const T *w,
                                                             const float *dz, float *dx,
                                                             float *dw_part, int n_tok, int d,
                                                             int E, int per) {
  constexpr int VC = kProjCols;
  __shared__ __align__(16) float2 zs[kProjTokens][EP];  // each dz twice: operands of packed FMAs
  const int tid = threadIdx.x;
  const int col = (blockIdx.x * kProjThreads + tid) * VC;
  const bool live = col < d;
  // W and x do not come from the kernel ahead (the logits' gradient), which began its
  // successor after its own wait: they are read before this one's
  constexpr int VP = VC / 2;  // pairs of columns
  float2 wr[EP][VP], acc[EP][VP];
#pragma unroll
  for (int e = 0; e < EP; ++e) {
#pragma unroll
    for (int c = 0; c < VP; ++c) wr[e][c] = acc[e][c] = make_float2(0.f, 0.f);
    if (dx && live && e < E) {
      Cols<T, VC> r;
      r.load(w + (size_t)e * d + col);
#pragma unroll
      for (int c = 0; c < VP; ++c) wr[e][c] = make_float2(r.get(2 * c), r.get(2 * c + 1));
    }
  }
  const int t0 = blockIdx.y * per, t1 = min(n_tok, t0 + per);
  // 32 bytes of x per thread are requested while the 32 before are worked on
  constexpr int NB = 32 / (VC * (int)sizeof(T)) < 8 ? 32 / (VC * (int)sizeof(T)) : 8;
  Cols<T, VC> next[NB];
  auto request = [&](int t) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (dw_part && live && t + i < t1) next[i].load(x + (size_t)(t + i) * d + col);
  };
  request(t0);
  pdl_wait();
  pdl_trigger();
  for (int tb = t0; tb < t1; tb += kProjTokens) {  // a multiple of NB
    const int n = min(kProjTokens, t1 - tb);
    __syncthreads();
    for (int i = tid; i < kProjTokens * EP; i += kProjThreads) {
      const int u = i / EP, e = i % EP;
      if (u >= n) break;
      const float z = e < E ? dz[(size_t)(tb + u) * E + e] : 0.f;
      zs[u][e] = make_float2(z, z);
    }
    __syncthreads();
    if (!live) continue;
    for (int u0 = 0; u0 < n; u0 += NB) {
      Cols<T, VC> xv[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) xv[i] = next[i];
      request(tb + u0 + NB);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (u0 + i >= n) break;
        float2 o[VP], xp[VP];
#pragma unroll
        for (int c = 0; c < VP; ++c) {
          o[c] = make_float2(0.f, 0.f);
          xp[c] = make_float2(xv[i].get(2 * c), xv[i].get(2 * c + 1));
        }
#pragma unroll
        for (int e = 0; e < EP; e += 2) {
          const float4 q = *reinterpret_cast<const float4 *>(&zs[u0 + i][e]);
          const float2 z[2] = {make_float2(q.x, q.y), make_float2(q.z, q.w)};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < VP; ++c) {
              if (dx) o[c] = __ffma2_rn(z[h], wr[e + h][c], o[c]);
              if (dw_part) acc[e + h][c] = __ffma2_rn(z[h], xp[c], acc[e + h][c]);
            }
        }
        if (dx) {
          float *out = dx + (size_t)(tb + u0 + i) * d + col;
          *reinterpret_cast<float4 *>(out) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
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
        for (int c = 0; c < VP; ++c) reinterpret_cast<float2 *>(out)[c] = acc[e][c];
      }
  }
}

// dw [E, d] = the sum of the `parts` partials (each `rows` x d, its first E rows), and (the
// last blocks) db[e] = the sum of the blocks' partials. Eight (32) groups of threads take
// every eighth (32nd) partial, so that few loads follow one another (one thread for all of
// them: 14 us for 74 partials, this 4); the groups are added in order.
template <typename T>
__global__ void __launch_bounds__(256) k_route_sums(const float *part, int parts, int rows, int d,
                                                    T *dw, int dw_blocks, const float *db_part,
                                                    int blocks, int E, float *db) {
  __shared__ float4 red4[8][32];
  __shared__ float red[32][8];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < dw_blocks) {  // d is a multiple of 4
    const int x = tid & 31, g = tid >> 5;
    const size_t i = ((size_t)blockIdx.x * 32 + x) * 4;
    const bool in = i < (size_t)E * d;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
#pragma unroll 4
      for (int s = g; s < parts; s += 8) {
        const float4 p = __ldg(reinterpret_cast<const float4 *>(part + (size_t)s * rows * d + i));
        v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
      }
    }
    red4[g][x] = v;
    __syncthreads();
    if (g > 0 || !in) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) {
      const float4 p = red4[q][x];
      v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
    }
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4 *>(dw + i) = v;
    else
      *reinterpret_cast<uint2 *>(dw + i) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    return;
  }
  const int e = ((int)blockIdx.x - dw_blocks) * 8 + (tid & 7), g = tid >> 3;
  float v = 0.f;
  if (e < E) {
#pragma unroll 8
    for (int s = g; s < blocks; s += 32) v += db_part[(size_t)s * E + e];
  }
  red[g][tid & 7] = v;
  __syncthreads();
  if (tid >= 8 || e >= E) return;
#pragma unroll
  for (int q = 1; q < 32; ++q) v += red[q][tid];
  db[e] = v;
}

// lanes per token of k_dlogits: eight experts each, the tensor-core terms' padding too
int dz_lanes(int cols) {
  int l = 1;
  while (l * kEpl < cols) l *= 2;
  return l;
}
int dlogits_blocks(int T, int lanes) {
  const int b = ceil_div(T, kDzThreads / lanes);
  return b < kMaxBlocks ? b : kMaxBlocks;
}

// pieces of the tokens for dW: enough tiles for two per SM
int dw_pieces(int T, int d, int E) {
  const int tiles = ceil_div(E, 128) * ceil_div(d, simt::BN);
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

// ... of k_route_proj: as many blocks as the SMs hold (registers), at least sixteen tokens
// each
int proj_pieces(int T, int d, int E) {
  const int s = 148 * (E <= 8 ? 4 : 2) / ceil_div(d, kProjThreads * kProjCols), most = ceil_div(T, 16);
  return s < 1 ? 1 : (s < most ? s : most);
}

int e_padded(int E) { return (E + 63) / 64 * 64; }

template <bool TC>
cudaError_t dlogits(const RouteBwdArgs &a, float *db_part, const RouteTcArgs &tc, int lanes,
                    cudaStream_t st) {
  const dim3 g(dlogits_blocks(a.T, lanes)), b(kDzThreads);
  if constexpr (!TC) {  // the terms' rows are 64 experts at least
    if (lanes == 1) return launch_pdl(k_dlogits<1, TC>, g, b, 0, st, a, db_part, tc);
    if (lanes == 2) return launch_pdl(k_dlogits<2, TC>, g, b, 0, st, a, db_part, tc);
    if (lanes == 4) return launch_pdl(k_dlogits<4, TC>, g, b, 0, st, a, db_part, tc);
  }
  if (lanes == 8) return launch_pdl(k_dlogits<8, TC>, g, b, 0, st, a, db_part, tc);
  if (lanes == 16) return launch_pdl(k_dlogits<16, TC>, g, b, 0, st, a, db_part, tc);
  return launch_pdl(k_dlogits<32, TC>, g, b, 0, st, a, db_part, tc);
}

template <typename T>
cudaError_t sums(const RouteBwdArgs &a, const float *dw_part, int parts, int rows,
                 const float *db_part, int lanes, cudaStream_t st) {
  const int dw_blocks = a.dw ? (int)(((size_t)a.E * a.d / 4 + 31) / 32) : 0;
  const int db_blocks = a.db ? ceil_div(a.E, 8) : 0;
  if (dw_blocks + db_blocks == 0) return cudaSuccess;
  return launch_pdl(k_route_sums<T>, dim3(dw_blocks + db_blocks), dim3(256), 0, st, dw_part, parts,
                    rows, a.d, static_cast<T *>(a.dw), dw_blocks, db_part,
                    dlogits_blocks(a.T, lanes), a.E, a.db);
}

template <typename T>
cudaError_t route_bwd_few(const RouteBwdArgs &a, cudaStream_t st) {
  float *db_part = static_cast<float *>(a.part);
  cudaError_t e = dlogits<false>(a, a.db ? db_part : nullptr, RouteTcArgs{}, dz_lanes(a.E), st);
  if (e != cudaSuccess) return e;
  const int pieces = proj_pieces(a.T, a.d, a.E);
  float *dw_part = db_part + (size_t)kMaxBlocks * a.E;
  if (a.dx || a.dw) {
    const dim3 g(ceil_div(a.d, kProjThreads * kProjCols), pieces), b(kProjThreads);
    const T *x = static_cast<const T *>(a.x), *w = static_cast<const T *>(a.w);
    auto run = [&](auto kernel) {
      return launch_pdl(kernel, g, b, 0, st, x, w, (const float *)a.dlogits, a.dx,
                        a.dw ? dw_part : static_cast<float *>(nullptr), a.T, a.d, a.E,
                        ceil_div(a.T, pieces));
    };
    if constexpr (sizeof(T) == 2)
      e = run(k_route_proj<T, 8>);
    else
      e = a.E <= 8 ? run(k_route_proj<T, 8>) : run(k_route_proj<T, 16>);
    if (e != cudaSuccess) return e;
  }
  return sums<T>(a, dw_part, pieces, a.E, db_part, dz_lanes(a.E), st);
}

// fp32, more experts: tiles on CUDA cores, those of dx = dz W and of the pieces of dW =
// dz^T x in one launch. E need not be a multiple of 4.
using ProjTile = simt::Tile<128>;
template <bool VEC>
__global__ void __launch_bounds__(simt::kThreads) k_proj_tiles(RouteBwdArgs a, float *dw_part,
                                                               int dx_blocks, int per) {
  using T = ProjTile;
  __shared__ simt::GemmSmem<T> sm;
  pdl_wait();
  pdl_trigger();
  const float *x = static_cast<const float *>(a.x), *w = static_cast<const float *>(a.w);
  const int nt = ceil_div(a.d, simt::BN), E = a.E, d = a.d;
  int b = blockIdx.x;
  if (b < dx_blocks) {
    const int m0 = b / nt * T::BM, n0 = b % nt * simt::BN;
    float acc[T::TM][T::TN];
    simt::clear(acc);
    simt::mma_tile<T, false, VEC>(sm, acc, a.dlogits + (size_t)m0 * E, E, a.T - m0, w + n0, d,
                                  d - n0, E);
    simt::store_tile<T, true>(acc, a.dx + (size_t)m0 * d + n0, d, min(T::BM, a.T - m0),
                              min(simt::BN, d - n0));
    return;
  }
  b -= dx_blocks;
  const int mt = ceil_div(E, T::BM), piece = b / (mt * nt);
  b -= piece * mt * nt;
  const int m0 = b / nt * T::BM, n0 = b % nt * simt::BN;
  const int t0 = min(a.T, piece * per), n = min(a.T - t0, per);
  simt::sum_rows<T, VEC, true>(sm, a.dlogits + (size_t)t0 * E + m0, E, E - m0,
                               x + (size_t)t0 * d + n0, d, d - n0, n,
                               dw_part + ((size_t)piece * E + m0) * d + n0, d);
}

cudaError_t route_bwd_simt(const RouteBwdArgs &a, cudaStream_t st) {
  float *db_part = static_cast<float *>(a.part);
  cudaError_t e = dlogits<false>(a, a.db ? db_part : nullptr, RouteTcArgs{}, dz_lanes(a.E), st);
  if (e != cudaSuccess) return e;
  const int pieces = dw_pieces(a.T, a.d, a.E), nt = ceil_div(a.d, simt::BN);
  float *dw_part = db_part + (size_t)kMaxBlocks * a.E;
  const int dx = a.dx ? nt * ceil_div(a.T, ProjTile::BM) : 0;
  const int dw = a.dw ? nt * ceil_div(a.E, ProjTile::BM) * pieces : 0;
  if (dx + dw > 0) {
    e = launch_pdl(a.E % 4 ? k_proj_tiles<false> : k_proj_tiles<true>, dim3(dx + dw),
                   dim3(simt::kThreads), 0, st, a, dw_part, dx, ceil_div(a.T, pieces));
    if (e != cudaSuccess) return e;
  }
  return sums<float>(a, dw_part, pieces, a.E, db_part, dz_lanes(a.E), st);
}

// bf16 scratch: tables | db partials | dW partials | terms
struct TcScratch {
  size_t db, dw, terms, total;
};
TcScratch tc_scratch(int T, int d, int E) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  TcScratch s;
  s.db = up((kMaxExperts + 1 + 6) * 4);
  s.dw = s.db + up((size_t)kMaxBlocks * E * 4);
  s.terms = s.dw + up((size_t)dw_pieces_tc(T, d) * kSplitDw * e_padded(E) * d * 4);
  s.total = s.terms + up((size_t)T * kSplit * e_padded(E) * 2);
  return s;
}

cudaError_t route_bwd_tc(const RouteBwdArgs &a, cudaStream_t st) {
  const TcScratch s = tc_scratch(a.T, a.d, a.E);
  char *base = static_cast<char *>(a.part);
  float *db_part = reinterpret_cast<float *>(base + s.db);
  RouteTcArgs tc{};
  tc.x = a.x;
  tc.w = a.w;
  const bool terms = a.dx || a.dw;
  tc.terms = reinterpret_cast<__nv_bfloat16 *>(base + s.terms);
  tc.all = reinterpret_cast<int32_t *>(base);
  tc.all_rows = tc.all + 2;
  tc.all_tiles = tc.all + 4;
  tc.piece = tc.all + 6;
  tc.dx = a.dx;
  tc.dw_part = a.dw ? reinterpret_cast<float *>(base + s.dw) : nullptr;
  tc.T = a.T;
  tc.d = a.d;
  tc.E = a.E;
  tc.Ep = e_padded(a.E);
  tc.pieces = dw_pieces_tc(a.T, a.d);
  tc.err = a.err;
  const int lanes = dz_lanes(terms ? tc.Ep : a.E);
  cudaError_t e = terms ? dlogits<true>(a, a.db ? db_part : nullptr, tc, lanes, st)
                        : dlogits<false>(a, a.db ? db_part : nullptr, tc, lanes, st);
  if (e != cudaSuccess) return e;
  if (terms) {
    e = launch_route_tc(tc, st);
    if (e != cudaSuccess) return e;
  }
  return sums<__nv_bfloat16>(a, tc.dw_part, tc.pieces * kSplitDw, tc.Ep, db_part, lanes, st);
}

}  // namespace

// Whether the one pass of k_route_proj takes the products. Against the tensor cores (bf16,
// T = 4096, d = 4096): 36 us to 39 with 8 experts, 63 to 39 with 12, 167 to 40 with 32.
// Against the tiles on CUDA cores (fp32): 41 us with 8 and 60 with 16, where the tiles take 130
// (20 experts; 156 with 17, whose rows are not vectors), but 163 to 131 with 32, where a
// thread's registers hold half the columns.
static bool few_experts(int E, int dtype) { return E <= (dtype == MOE_DTYPE_F32 ? 16 : 8); }

bool route_bwd_reads_dlogits(int E, int dtype) {
  return few_experts(E, dtype) || dtype == MOE_DTYPE_F32;
}

size_t route_bwd_scratch_bytes(int T, int d, int E, int dtype) {
  if (T < 1) T = 1;
  if (!route_bwd_reads_dlogits(E, dtype)) return tc_scratch(T, d, E).total;
  const int pieces = few_experts(E, dtype) ? proj_pieces(T, d, E) : dw_pieces(T, d, E);
  return sizeof(float) * ((size_t)kMaxBlocks * E + (size_t)pieces * E * d);
}

cudaError_t launch_route_bwd(const RouteBwdArgs &a, int dtype, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const bool f32 = dtype == MOE_DTYPE_F32;
  if (few_experts(a.E, dtype))
    return f32 ? route_bwd_few<float>(a, st) : route_bwd_few<__nv_bfloat16>(a, st);
  return f32 ? route_bwd_simt(a, st) : route_bwd_tc(a, st);
}

}  // namespace moe
