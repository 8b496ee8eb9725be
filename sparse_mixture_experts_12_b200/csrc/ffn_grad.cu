// Gradient of the grouped expert FFN: the CUDA-core path (fp32 layers), and what both
// paths share (tables, bias gradients, the weights' row gradient).
//
// With x, dy the expert-contiguous rows of an expert and w_r an optional weight of
// row r's output (1 without), from recomputed pre-activations:
//   SwiGLU  a = x W1^T, u = x W3^T, q = dy W2, s = sigmoid(a)
//           h = a s u,  du = w q a s,  da = w q u s (1 + a (1 - s))
//   MLP     a = x W1^T + b1, q = dy W2;  h = act(a),  da = w q act'(a)
//   dx = da W1 (+ du W3);  dW1 = da^T x, dW3 = du^T x, dW2 = dy^T (w h)
//   db1 = sum_r da, db2 = sum_r w dy, and dw_r = <dy_r, E(x_r)> = <q_r, h_r> (+ <dy_r, b2>)
// The last identity gives the gate's gradient without a second down projection. The
// weight is applied once, in fp32, before the one rounding of h, da and du to the
// layer's type; the bias and row gradients are summed from the unrounded values.
//
// Sums over rows and over columns go through per-tile partials that a second
// kernel adds in tile order, so the results do not depend on the schedule.
#include "grad.cuh"
#include "grad_simt.cuh"

namespace moe {

namespace {

using namespace simt;

constexpr int kDBK = 16;  // K slice of the fused first step: three B tiles and two A tiles
constexpr int kDA = BM * kDBK / 256, kDB = BN * kDBK / 256;

// d act(v) / dv and act(v)
__device__ __forceinline__ void act_and_slope(int act, float v, float &h, float &s) {
  if (act == MOE_ACT_RELU) {
    h = fmaxf(v, 0.f);
    s = v > 0.f ? 1.f : 0.f;
  } else {
    const float c = 0.5f * (1.f + erff(v * 0.70710678118654752f));
    h = v * c;
    s = c + v * 0.39894228040143268f * expf(-0.5f * v * v);
  }
}

// Step 1: one 128-row x 64-column tile of h, da (and du) from the three products,
// all with reduction length d.
template <typename T, bool GLU>
__global__ void __launch_bounds__(256) k_dact(FfnGradArgs s) {
  __shared__ __align__(16) float Xs[kDBK][BM + 4];
  __shared__ __align__(16) float Ys[kDBK][BM + 4];
  __shared__ __align__(16) float W1s[kDBK][BN + 4];
  __shared__ __align__(16) float W3s[GLU ? kDBK : 1][BN + 4];
  __shared__ __align__(16) float W2s[kDBK][BN + 4];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int g = group_of_tile(s.mprefix, s.G, blockIdx.y);
  if (g < 0) return;
  const int row0 = s.offsets[g] + ((int)blockIdx.y - s.mprefix[g]) * BM;
  const int nrows = min(BM, s.offsets[g + 1] - row0);
  const int n0 = blockIdx.x * BN, F = s.F, d = s.d;
  const int tx = tid % (BN / TN), ty = tid / (BN / TN);
  const T *x = static_cast<const T *>(s.x) + (size_t)row0 * d;
  const T *dy = static_cast<const T *>(s.dy) + (size_t)row0 * d;
  const T *w1 = static_cast<const T *>(s.w1) + ((size_t)g * F + n0) * d;
  const T *w3 = GLU ? static_cast<const T *>(s.w3) + ((size_t)g * F + n0) * d : nullptr;
  const T *w2 = static_cast<const T *>(s.w2) + (size_t)g * d * F + n0;
  float a1[TM][TN], a3[GLU ? TM : 1][TN], a2[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      a1[i][j] = a2[i][j] = 0.f;
      if (GLU) a3[i][j] = 0.f;
    }
  float rx[kDA], ry[kDA], r1[kDB], r3[GLU ? kDB : 1], r2[kDB];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kDA; ++j) {
      const int i = tid + 256 * j, m = i / kDBK, kk = i % kDBK;
      const bool ok = m < nrows && k0 + kk < d;
      rx[j] = ok ? Elem<T>::to_f(x[(size_t)m * d + k0 + kk]) : 0.f;
      ry[j] = ok ? Elem<T>::to_f(dy[(size_t)m * d + k0 + kk]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kDB; ++j) {
      const int i = tid + 256 * j, n = i / kDBK, kk = i % kDBK;
      const bool ok = n0 + n < F && k0 + kk < d;
      r1[j] = ok ? Elem<T>::to_f(w1[(size_t)n * d + k0 + kk]) : 0.f;
      if (GLU) r3[j] = ok ? Elem<T>::to_f(w3[(size_t)n * d + k0 + kk]) : 0.f;
      const int n2 = i % BN, k2 = i / BN;
      r2[j] = (n0 + n2 < F && k0 + k2 < d) ? Elem<T>::to_f(w2[(size_t)(k0 + k2) * F + n2]) : 0.f;
    }
  };
  fetch(0);
  for (int k0 = 0; k0 < d; k0 += kDBK) {
#pragma unroll
    for (int j = 0; j < kDA; ++j) {
      const int i = tid + 256 * j;
      Xs[i % kDBK][i / kDBK] = rx[j];
      Ys[i % kDBK][i / kDBK] = ry[j];
    }
#pragma unroll
    for (int j = 0; j < kDB; ++j) {
      const int i = tid + 256 * j;
      W1s[i % kDBK][i / kDBK] = r1[j];
      if (GLU) W3s[i % kDBK][i / kDBK] = r3[j];
      W2s[i / BN][i % BN] = r2[j];
    }
    __syncthreads();
    if (k0 + kDBK < d) fetch(k0 + kDBK);
#pragma unroll
    for (int kk = 0; kk < kDBK; ++kk) {
      float xv[TM], yv[TM];
#pragma unroll
      for (int i = 0; i < TM; i += 4) {
        const float4 p = *reinterpret_cast<const float4 *>(&Xs[kk][ty * TM + i]);
        xv[i] = p.x; xv[i + 1] = p.y; xv[i + 2] = p.z; xv[i + 3] = p.w;
        const float4 q = *reinterpret_cast<const float4 *>(&Ys[kk][ty * TM + i]);
        yv[i] = q.x; yv[i + 1] = q.y; yv[i + 2] = q.z; yv[i + 3] = q.w;
      }
      const float4 b1 = *reinterpret_cast<const float4 *>(&W1s[kk][tx * TN]);
      const float4 b2 = *reinterpret_cast<const float4 *>(&W2s[kk][tx * TN]);
      const float v1[TN] = {b1.x, b1.y, b1.z, b1.w}, v2[TN] = {b2.x, b2.y, b2.z, b2.w};
      float v3[TN] = {0.f, 0.f, 0.f, 0.f};
      if (GLU) {
        const float4 b3 = *reinterpret_cast<const float4 *>(&W3s[kk][tx * TN]);
        v3[0] = b3.x; v3[1] = b3.y; v3[2] = b3.z; v3[3] = b3.w;
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          a1[i][j] = fmaf(xv[i], v1[j], a1[i][j]);
          a2[i][j] = fmaf(yv[i], v2[j], a2[i][j]);
          if (GLU) a3[i][j] = fmaf(xv[i], v3[j], a3[i][j]);
        }
    }
    __syncthreads();
  }
  float col[TN], dot[TM];
#pragma unroll
  for (int j = 0; j < TN; ++j) col[j] = 0.f;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = ty * TM + i;
    dot[i] = 0.f;
    if (m >= nrows) continue;
    const size_t r = (size_t)(row0 + m);
    const float w = s.row_w ? s.row_w[r] : 1.f;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + tx * TN + j;
      if (n >= F) continue;
      const float q = a2[i][j];
      float h, da, du = 0.f;
      if (GLU) {
        const float v = a1[i][j], u = a3[i][j];
        const float sg = 1.f / (1.f + expf(-v));
        h = v * sg * u;
        du = q * v * sg;
        da = q * u * sg * (1.f + v * (1.f - sg));
      } else {
        float sl;
        act_and_slope(s.act, a1[i][j] + (s.b1 ? s.b1[(size_t)g * F + n] : 0.f), h, sl);
        da = q * sl;
      }
      dot[i] = fmaf(q, h, dot[i]);
      col[j] += w * da;
      static_cast<T *>(s.h)[r * F + n] = Elem<T>::from_f(w * h);
      static_cast<T *>(s.dg)[r * F + n] = Elem<T>::from_f(w * da);
      if (GLU) static_cast<T *>(s.du)[r * F + n] = Elem<T>::from_f(w * du);
    }
  }
  if (s.row_dot) {  // the tile's 16 column threads of a row
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int o = BN / TN / 2; o > 0; o >>= 1) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
      const int m = ty * TM + i;
      if (tx == 0 && m < nrows) s.dot_part[(size_t)blockIdx.x * s.rows + row0 + m] = dot[i];
    }
  }
  if (s.db1) {  // the tile's 16 row threads of a column, through shared memory
    float(*red)[BN] = reinterpret_cast<float(*)[BN]>(&Xs[0][0]);
#pragma unroll
    for (int j = 0; j < TN; ++j) red[ty][tx * TN + j] = col[j];
    __syncthreads();
    if (tid < BN && n0 + tid < F) {
      float v = 0.f;
      for (int i = 0; i < BM / TM; ++i) v += red[i][tid];
      s.col_part[(size_t)blockIdx.y * F + n0 + tid] = v;
    }
  }
}

// w_r-weighted column sums of dy over a 128-row tile -> part [tiles, d]
template <typename T>
__global__ void __launch_bounds__(256) k_col_sums(FfnGradArgs s) {
  __shared__ float red[4][64];
  pdl_wait();
  pdl_trigger();
  const int g = group_of_tile(s.mprefix, s.G, blockIdx.y), d = s.d;
  if (g < 0) return;
  const int in = ((int)blockIdx.y - s.mprefix[g]) * BM;
  const int row0 = s.poff[g] + in;
  const int nrows = min(BM, s.offsets[g + 1] - s.offsets[g] - in);
  const int n = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
  const T *dy = static_cast<const T *>(s.dy);
  float v = 0.f;
  if (n < d) {
#pragma unroll 8
    for (int m = q; m < nrows; m += 4) {
      const size_t r = (size_t)(row0 + m);
      const float f = Elem<T>::to_f(dy[r * d + n]);
      v += s.row_w ? s.row_w[r] * f : f;
    }
  }
  red[q][threadIdx.x & 63] = v;
  __syncthreads();
  if (q == 0 && n < d) {
    const int c = threadIdx.x;
    s.col_part[(size_t)blockIdx.y * d + n] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
  }
}

// out [G, N]: the expert's partials in order (0 for an expert without rows); expert g's
// are first[g] / unit up to first[g + 1] / unit
__global__ void __launch_bounds__(256) k_col_reduce(const float *part, const int32_t *first,
                                                    int unit, int N, float *out) {
  pdl_wait();
  pdl_trigger();
  const int n = blockIdx.x * 256 + threadIdx.x, g = blockIdx.y;
  if (n >= N) return;
  float v = 0.f;
#pragma unroll 4
  for (int t = first[g] / unit; t < first[g + 1] / unit; ++t) v += part[(size_t)t * N + n];
  out[(size_t)g * N + n] = v;
}

// row_dot[r] = sum of the row's column-tile partials (+ <dy_r, b2 of its expert>), a
// warp per row (padding rows are left out)
template <typename T>
__global__ void __launch_bounds__(256) k_row_dot(FfnGradArgs s, int nt) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= s.poff[s.G]) return;
  int lo = 0, hi = s.G - 1;  // last g with poff[g] <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.poff[mid] <= r) lo = mid; else hi = mid - 1;
  }
  if (r - s.poff[lo] >= s.offsets[lo + 1] - s.offsets[lo]) return;
  float v = 0.f;
  for (int i = lane; i < nt; i += 32) v += s.dot_part[(size_t)i * s.rows + r];
  if (s.b2) {
    const T *dy = static_cast<const T *>(s.dy) + (size_t)r * s.d;
    const float *b = s.b2 + (size_t)lo * s.d;
    for (int i = lane; i < s.d; i += 32) v = fmaf(Elem<T>::to_f(dy[i]), b[i], v);
  }
  v = warp_sum(v);
  if (lane == 0) s.row_dot[r] = v;
}

// One warp: offsets -> checked copy (all zero when they are no partition of at most
// max_rows rows), the 128-row tile prefix, and the prefix of the row counts rounded up to
// multiples of `pad`.
__global__ void k_grad_tables(const int32_t *offsets, int G, int max_rows, int pad,
                              int32_t *checked, int32_t *mprefix, int32_t *poff, int32_t *err) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x;
  int bad = G;
  for (int g = lane; g < G; g += 32) {
    const int a0 = offsets[g], a1 = offsets[g + 1];
    if (a0 < 0 || (g == 0 && a0 != 0) || a1 < a0 || a1 > max_rows) bad = min(bad, g);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bad = min(bad, __shfl_xor_sync(0xffffffffu, bad, o));
  const bool ok = bad == G;
  int sm = 0, sp = 0, mt[8], pr[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // G <= 256: eight groups per lane
    const int g = lane * 8 + j;
    const int n = (ok && g < G) ? offsets[g + 1] - offsets[g] : 0;
    mt[j] = ceil_div(n, kRowTile);
    pr[j] = ceil_div(n, pad) * pad;
    sm += mt[j];
    sp += pr[j];
  }
  int im = sm, ip = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, im, o), u = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      im += v;
      ip += u;
    }
  }
  int rm = im - sm, rp = ip - sp;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int g = lane * 8 + j;
    if (g < G) {
      mprefix[g] = rm;
      poff[g] = rp;
      checked[g] = ok ? offsets[g] : 0;
    }
    rm += mt[j];
    rp += pr[j];
  }
  if (lane == 31) {
    mprefix[G] = im;
    poff[G] = ip;
    checked[G] = ok ? offsets[G] : 0;
  }
  if (!ok && lane == 0) report_error(err, MOE_DEVERR_OFFSETS, bad);
}

__global__ void k_one_group(int n, int pad, int32_t *offsets, int32_t *mprefix, int32_t *poff) {
  pdl_wait();
  pdl_trigger();
  offsets[0] = mprefix[0] = poff[0] = 0;
  offsets[1] = n;
  mprefix[1] = ceil_div(n, kRowTile);
  poff[1] = ceil_div(n, pad) * pad;
}

// `groups`: the partials of db1 are one per 32 padded rows, those of row_dot one per 32
// columns; else one per 128-row and per 64-column tile
template <typename T>
cudaError_t bias_and_row_grads(const FfnGradArgs &a, bool groups, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.db1) {  // col_part holds step 1's sums
    e = launch_pdl(k_col_reduce, dim3(ceil_div(a.F, 256), a.G), dim3(256), 0, st,
                   (const float *)a.col_part, groups ? a.poff : a.mprefix, groups ? 32 : 1, a.F,
                   a.db1);
    if (e != cudaSuccess) return e;
  }
  if (a.db2) {
    e = launch_pdl(k_col_sums<T>, dim3(ceil_div(a.d, 64), a.m_tiles_ub), dim3(256), 0, st,
                   a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_col_reduce, dim3(ceil_div(a.d, 256), a.G), dim3(256), 0, st,
                   (const float *)a.col_part, a.mprefix, 1, a.d, a.db2);
    if (e != cudaSuccess) return e;
  }
  if (a.row_dot)
    e = launch_pdl(k_row_dot<T>, dim3(ceil_div(a.rows, 8)), dim3(256), 0, st, a,
                   groups ? a.F / 32 : ceil_div(a.F, BN));
  return e;
}

template <typename T>
cudaError_t ffn_bwd_simt(const FfnGradArgs &a, cudaStream_t st) {
  const bool glu = a.act == MOE_ACT_SWIGLU;
  const dim3 b(256);
  const dim3 g1(ceil_div(a.F, BN), a.m_tiles_ub);
  cudaError_t e = glu ? launch_pdl(k_dact<T, true>, g1, b, 0, st, a)
                      : launch_pdl(k_dact<T, false>, g1, b, 0, st, a);
  if (e != cudaSuccess) return e;
  e = bias_and_row_grads<T>(a, false, st);
  if (e != cudaSuccess) return e;
  if (a.dx) {
    const dim3 g2(ceil_div(a.d, BN), a.m_tiles_ub);
    auto run = [&](auto *out) {
      using TO = typename std::remove_pointer<decltype(out)>::type;
      Gemm<T, T, TO> m{};
      m.a[0] = static_cast<const T *>(a.dg);
      m.a[1] = static_cast<const T *>(a.du);
      m.b[0] = static_cast<const T *>(a.w1);
      m.b[1] = static_cast<const T *>(a.w3);
      m.c[0] = out;
      m.N[0] = a.d;
      m.lda[0] = m.lda[1] = a.F;
      m.ldb[0] = m.ldb[1] = a.d;
      m.nseg = glu ? 2 : 1;
      m.K = a.F;
      m.G = a.G;
      m.offsets = a.offsets;
      m.mprefix = a.mprefix;
      return launch_pdl(k_gemm<T, T, TO, false>, g2, b, 0, st, m);
    };
    e = (a.dx_f32 || sizeof(T) == 4) ? run(static_cast<float *>(a.dx)) : run(static_cast<T *>(a.dx));
    if (e != cudaSuccess) return e;
  }
  // the weights' gradients: up to three jobs in one launch
  Gemm<T, T, T> w{};
  int n = 0, mt = 0, nt = 0;
  auto job = [&](const void *p, const void *q, void *c, int M, int N) {
    if (c == nullptr) return;
    w.a[n] = static_cast<const T *>(p);
    w.b[n] = static_cast<const T *>(q);
    w.c[n] = static_cast<T *>(c);
    w.M[n] = w.lda[n] = M;
    w.N[n] = w.ldb[n] = N;
    mt = mt > ceil_div(M, BM) ? mt : ceil_div(M, BM);
    nt = nt > ceil_div(N, BN) ? nt : ceil_div(N, BN);
    ++n;
  };
  job(a.dg, a.x, a.dw1, a.F, a.d);
  if (glu) job(a.du, a.x, a.dw3, a.F, a.d);
  job(a.dy, a.h, a.dw2, a.d, a.F);
  if (n == 0) return cudaSuccess;
  w.nseg = n;
  w.G = a.G;
  w.offsets = a.offsets;
  w.mprefix = a.mprefix;
  return launch_pdl(k_gemm<T, T, T, true>, dim3(nt, mt, n * a.G), b, 0, st, w);
}

// bf16: the three steps on the tensor cores
cudaError_t ffn_bwd_tc(const FfnGradArgs &a, cudaStream_t st) {
  cudaError_t e = launch_act_grad_tc(a, st);
  if (e != cudaSuccess) return e;
  e = bias_and_row_grads<__nv_bfloat16>(a, true, st);
  if (e != cudaSuccess) return e;
  if (a.dx) {
    e = launch_dx_tc(a, st);
    if (e != cudaSuccess) return e;
  }
  return launch_dw_tc(a, st);
}

}  // namespace

cudaError_t launch_grad_tables(const int32_t *offsets, int G, int max_rows, int pad,
                               int32_t *checked, int32_t *mprefix, int32_t *poff, int32_t *err,
                               cudaStream_t st) {
  return launch_pdl(k_grad_tables, dim3(1), dim3(32), 0, st, offsets, G, max_rows, pad, checked,
                    mprefix, poff, err);
}

cudaError_t launch_one_group(int n, int pad, int32_t *offsets, int32_t *mprefix, int32_t *poff,
                             cudaStream_t st) {
  return launch_pdl(k_one_group, dim3(1), dim3(1), 0, st, n, pad, offsets, mprefix, poff);
}

cudaError_t launch_ffn_bwd(const FfnGradArgs &a, int dtype, cudaStream_t st) {
  return dtype == MOE_DTYPE_F32 ? ffn_bwd_simt<float>(a, st) : ffn_bwd_tc(a, st);
}

}  // namespace moe
