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

// w_r-weighted sums of 64 columns of dy over the `unit` rows of row tile y -> part2
// [tiles, d], a block's work
template <typename T>
__device__ __forceinline__ void col_sums(const FfnGradArgs &s, int unit, int x, int y) {
  __shared__ float red[4][64];
  const int g = group_of_tile(s.mprefix, s.G, y), d = s.d;
  if (g < 0) return;
  const int in = (y - s.mprefix[g]) * unit;
  const int row0 = s.poff[g] + in;
  const int nrows = min(unit, s.offsets[g + 1] - s.offsets[g] - in);
  const int n = x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
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
    s.part2[(size_t)y * d + n] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
  }
}
// (one dimension, as for fp32: the row tiles can be more than the 65535 of a grid's y)
template <typename T>
__global__ void __launch_bounds__(kThreads) k_col_sums(FfnGradArgs s, int unit) {
  pdl_wait();
  pdl_trigger();
  const int dn = ceil_div(s.d, 64);
  col_sums<T>(s, unit, blockIdx.x % dn, blockIdx.x / dn);
}

// What follows from the activations' gradients beside the matrix products, as blocks of
// one launch: db1 and db2 from their partials (in order; 0 for an expert without rows),
// and row_dot[r] = the sum of the row's column-tile partials (+ <dy_r, b2 of its expert>).
struct Reduce {
  int db1, db2, rows;      // blocks of each
  const int32_t *first;    // partials of db1: expert g's are first[g] / unit up to
  int unit;                // first[g + 1] / unit
  int dots;                // partials of a row
};
__device__ __forceinline__ void col_reduce(const float *part, const int32_t *first, int unit, int N,
                                           int x, float *out) {
  const int blocks = ceil_div(N, kThreads), g = x / blocks;
  const int n = (x - g * blocks) * kThreads + threadIdx.x;
  if (n >= N) return;
  float v = 0.f;
#pragma unroll 4
  for (int t = first[g] / unit; t < first[g + 1] / unit; ++t) v += part[(size_t)t * N + n];
  out[(size_t)g * N + n] = v;
}
// a warp per row (padding rows are left out)
template <typename T>
__device__ __forceinline__ void row_dot(const FfnGradArgs &s, int nt, int x) {
  const int r = x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= s.poff[s.G]) return;
  int lo = 0, hi = s.G - 1;  // last g with poff[g] <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.poff[mid] <= r) lo = mid; else hi = mid - 1;
  }
  if (r - s.poff[lo] >= s.offsets[lo + 1] - s.offsets[lo]) return;
  float v = 0.f;
#pragma unroll 4
  for (int i = lane; i < nt; i += 32) v += s.dot_part[(size_t)i * s.rows + r];
  if (s.b2) {
    const T *dy = static_cast<const T *>(s.dy) + (size_t)r * s.d;
    const float *b = s.b2 + (size_t)lo * s.d;
    for (int i = lane; i < s.d; i += 32) v = fmaf(Elem<T>::to_f(dy[i]), b[i], v);
  }
  v = warp_sum(v);
  if (lane == 0) s.row_dot[r] = v;
}
template <typename T>
__device__ __forceinline__ void reduce(const FfnGradArgs &s, const Reduce &q, int x) {
  if (x < q.db1) {
    col_reduce(s.col_part, q.first, q.unit, s.F, x, s.db1);
  } else if (x < q.db1 + q.db2) {
    col_reduce(s.part2, s.mprefix, 1, s.d, x - q.db1, s.db2);
  } else {
    row_dot<T>(s, q.dots, x - q.db1 - q.db2);
  }
}
Reduce reduce_blocks(const FfnGradArgs &a) {
  Reduce q{};
  q.db1 = a.db1 ? ceil_div(a.F, kThreads) * a.G : 0;
  q.db2 = a.db2 ? ceil_div(a.d, kThreads) * a.G : 0;
  q.rows = a.row_dot ? ceil_div(a.rows, 8) : 0;
  return q;
}
template <typename T>
__global__ void __launch_bounds__(kThreads) k_reduce(FfnGradArgs s, Reduce q) {
  pdl_wait();
  pdl_trigger();
  reduce<T>(s, q, blockIdx.x);
}

// --------------------------------------------------------------- fp32, CUDA cores
// Step 1: one BM-row x 64-column tile of h, da (and du) from the three products, all with
// reduction length d; blocks behind the tiles add up db2's columns. Two blocks an SM hold
// the MLP's 128-row tiles (16 experts of 416 x 6540 on 1,961 rows: the pass 1.89 -> 1.67 ms);
// SwiGLU's three sums do not fit so (3.08 ms where one block takes 2.71).
template <class T, bool GLU, bool VEC>
__global__ void __launch_bounds__(kThreads, !GLU && T::BM == 128 ? 2 : 0)
    k_dact(FfnGradArgs s, int tiles_n, int tiles) {
  constexpr int BM = T::BM, BK = T::BK, TM = T::TM, TN = T::TN;
  struct Smem {
    alignas(16) float x[BK][T::LDA], y[BK][T::LDA];
    alignas(16) float w1[BK][T::LDB], w3[GLU ? BK : 1][T::LDB], w2[BK][T::LDB];
  };
  __shared__ Smem sm;
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= tiles) {
    const int i = (int)blockIdx.x - tiles, dn = ceil_div(s.d, 64);
    col_sums<float>(s, BM, i % dn, i / dn);
    return;
  }
  const int tile_m = blockIdx.x / tiles_n, tile_n = blockIdx.x % tiles_n;
  const int g = group_of_tile(s.mprefix, s.G, tile_m);
  if (g < 0) return;
  const int row0 = s.offsets[g] + (tile_m - s.mprefix[g]) * BM;
  const int nrows = min(BM, s.offsets[g + 1] - row0);
  const int n0 = tile_n * BN, F = s.F, d = s.d, ncols = min(BN, F - n0);
  const int tx = threadIdx.x % T::TX, ty = threadIdx.x / T::TX;
  const float *x = static_cast<const float *>(s.x) + (size_t)row0 * d;
  const float *dy = static_cast<const float *>(s.dy) + (size_t)row0 * d;
  const float *w1 = static_cast<const float *>(s.w1) + ((size_t)g * F + n0) * d;
  const float *w3 = GLU ? static_cast<const float *>(s.w3) + ((size_t)g * F + n0) * d : nullptr;
  const float *w2 = static_cast<const float *>(s.w2) + (size_t)g * d * F + n0;
  float a1[TM][TN], a3[GLU ? TM : 1][TN], a2[TM][TN];
  clear(a1);
  clear(a2);
  if (GLU) clear(a3);
  // small tiles have the registers to add up their sums in parts of 512 (the error of a
  // running sum grows with the root of its length)
  constexpr bool kParts = BM < 128;
  float t1[kParts ? TM : 1][TN], t3[kParts && GLU ? TM : 1][TN], t2[kParts ? TM : 1][TN];
  clear(t1);
  clear(t2);
  if (GLU) clear(t3);
  Slice<BM, BK, T::LDA, true, true> sx, sy;  // d is a multiple of 4
  Slice<BN, BK, T::LDB, true, true> s1, s3;
  Slice<BN, BK, T::LDB, false, VEC> s2;
  auto fetch = [&](int k0) {
    sx.fetch(x, d, nrows, k0, d);
    sy.fetch(dy, d, nrows, k0, d);
    s1.fetch(w1, d, ncols, k0, d);
    if (GLU) s3.fetch(w3, d, ncols, k0, d);
    s2.fetch(w2, F, ncols, k0, d);
  };
  fetch(0);
  for (int k0 = 0; k0 < d; k0 += BK) {
    __syncthreads();
    sx.put(sm.x);
    sy.put(sm.y);
    s1.put(sm.w1);
    if constexpr (GLU) s3.put(sm.w3);
    s2.put(sm.w2);
    __syncthreads();
    if (k0 + BK < d) fetch(k0 + BK);
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      float xv[TM], yv[TM];
      values(&sm.x[k][ty * TM], xv);
      values(&sm.y[k][ty * TM], yv);
      outer(a1, xv, &sm.w1[k][tx * TN]);
      if constexpr (GLU) outer(a3, xv, &sm.w3[k][tx * TN]);
      outer(a2, yv, &sm.w2[k][tx * TN]);
    }
    if constexpr (kParts) {
      if (k0 + BK >= d || (k0 + BK) % 512 == 0) {
        flush(t1, a1);
        flush(t2, a2);
        if constexpr (GLU) flush(t3, a3);
      }
    }
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
      const float q = kParts ? t2[i][j] : a2[i][j], v = kParts ? t1[i][j] : a1[i][j];
      float h, da, du = 0.f;
      if constexpr (GLU) {
        const float u = kParts ? t3[i][j] : a3[i][j];
        const float sg = 1.f / (1.f + expf(-v));
        h = v * sg * u;
        du = q * v * sg;
        da = q * u * sg * (1.f + v * (1.f - sg));
      } else {
        float sl;
        act_and_slope(s.act, v + (s.b1 ? s.b1[(size_t)g * F + n] : 0.f), h, sl);
        da = q * sl;
      }
      dot[i] = fmaf(q, h, dot[i]);
      col[j] += w * da;
      static_cast<float *>(s.h)[r * F + n] = w * h;
      static_cast<float *>(s.dg)[r * F + n] = w * da;
      if (GLU) static_cast<float *>(s.du)[r * F + n] = w * du;
    }
  }
  if (s.row_dot) {  // the tile's column threads of a row
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int o = T::TX / 2; o > 0; o >>= 1) dot[i] += __shfl_xor_sync(0xffffffffu, dot[i], o);
      const int m = ty * TM + i;
      if (tx == 0 && m < nrows) s.dot_part[(size_t)tile_n * s.rows + row0 + m] = dot[i];
    }
  }
  if (s.db1) {  // the tile's row threads of a column, through shared memory
    float(*red)[BN] = reinterpret_cast<float(*)[BN]>(&sm.w1[0][0]);
    static_assert(sizeof(sm.w1) >= 16 * BN * sizeof(float), "reduction buffer");
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TN; ++j) red[ty][tx * TN + j] = col[j];
    __syncthreads();
    if (threadIdx.x < ncols) {
      float v = 0.f;
      for (int i = 0; i < T::TY; ++i) v += red[i][threadIdx.x];
      s.col_part[(size_t)tile_m * F + n0 + threadIdx.x] = v;
    }
  }
}

// Step 2, one launch: tiles of dx = da W1 (+ du W3), tiles of the weights' gradients
// (reduction over the expert's rows), and the reductions. The long reduction of dx over F is
// split into `splits` pieces, which k_dx_sum adds in order: so that few tiles fill the GPU
// (two rows of a 2100 x 13008 expert took 530 us in 33 blocks, 125 us so), and that no
// running sum grows too long (see dx_splits).
struct Products {
  int dx, dw;              // blocks of each (then come the reductions')
  int dx_n, splits, piece; // column tiles of dx; pieces of F, `piece` long
  int jobs;                // weights: products of M x N
  const float *a[3], *b[3];
  float *c[3];
  int M[3], N[3], tiles[3];
};
template <class TD, class TW, bool VEC>
__global__ void __launch_bounds__(kThreads, TW::BN == 128 ? 2 : 0)
    k_products(FfnGradArgs s, Products p, Reduce q) {
  __shared__ union Smem {
    GemmSmem<TD> d;
    GemmSmem<TW> w;
  } sm;
  pdl_wait();
  pdl_trigger();
  int x = blockIdx.x;
  if (x < p.dx) {
    const int split = x % p.splits, n0 = x / p.splits % p.dx_n * TD::BN;
    const int tile_m = x / (p.splits * p.dx_n);
    const int g = group_of_tile(s.mprefix, s.G, tile_m);
    if (g < 0) return;
    const int row0 = s.offsets[g] + (tile_m - s.mprefix[g]) * TD::BM;
    const int rows = min(TD::BM, s.offsets[g + 1] - row0), cols = min(TD::BN, s.d - n0);
    const int k0 = split * p.piece, K = min(p.piece, s.F - k0);
    const size_t ao = (size_t)row0 * s.F + k0, wo = ((size_t)g * s.F + k0) * s.d + n0;
    float acc[TD::TM][TD::TN];
    clear(acc);
    mma_tile<TD, false, VEC>(sm.d, acc, static_cast<const float *>(s.dg) + ao, s.F, rows,
                             static_cast<const float *>(s.w1) + wo, s.d, cols, K);
    if (s.act == MOE_ACT_SWIGLU)
      mma_tile<TD, false, VEC>(sm.d, acc, static_cast<const float *>(s.du) + ao, s.F, rows,
                               static_cast<const float *>(s.w3) + wo, s.d, cols, K);
    float *out = p.splits > 1 ? s.dx_part + (size_t)split * s.rows * s.d
                              : static_cast<float *>(s.dx);
    store_tile<TD, true>(acc, out + (size_t)row0 * s.d + n0, s.d, rows, cols);
    return;
  }
  x -= p.dx;
  if (x < p.dw) {
    // in parts of kSumRows rows (see sum_rows); the tile is worked out anew for each, so that
    // nothing but its number stays in a register beside the sums (the layer of 191 rows of
    // 3152 x 8764 takes 1394 us so, 1435 through sum_rows, 1382 with one sum)
    int k0 = 0, left;
    do {
      int y = x;
      asm volatile("" : "+r"(y));
      int j = 0;
      while (y >= s.G * p.tiles[j]) {
        y -= s.G * p.tiles[j];
        ++j;
      }
      const int g = y / p.tiles[j], t = y % p.tiles[j];
      const int M = p.M[j], N = p.N[j], nt = ceil_div(N, TW::BN);
      const int m0 = t / nt * TW::BM, n0 = t % nt * TW::BN;
      const size_t row0 = (size_t)s.offsets[g] + k0;
      left = s.offsets[g + 1] - (int)row0;
      float acc[TW::TM][TW::TN];
      clear(acc);
      mma_tile<TW, true, VEC>(sm.w, acc, p.a[j] + row0 * M + m0, M, M - m0, p.b[j] + row0 * N + n0,
                              N, N - n0, min(left, kSumRows));
      store_tile<TW, VEC>(acc, p.c[j] + ((size_t)g * M + m0) * N + n0, N, min(TW::BM, M - m0),
                          min(TW::BN, N - n0), k0 > 0);
      k0 += kSumRows;
    } while (left > kSumRows);
    return;
  }
  reduce<float>(s, q, x - p.dw);
}

__global__ void __launch_bounds__(kThreads) k_dx_sum(FfnGradArgs s, int splits) {
  pdl_wait();
  pdl_trigger();
  const size_t n = (size_t)s.offsets[s.G] * s.d, all = (size_t)s.rows * s.d;
  const size_t i = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 4;  // d is a multiple of 4
  if (i >= n) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < splits; ++j) {
    const float4 p = __ldg(reinterpret_cast<const float4 *>(s.dx_part + j * all + i));
    v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
  }
  *reinterpret_cast<float4 *>(static_cast<float *>(s.dx) + i) = v;
}

// One warp: offsets -> checked copy (all zero when they are no partition of at most
// max_rows rows), the prefixes of their tiles, and the prefix of the row counts rounded up to
// multiples of `pad`.
__global__ void k_grad_tables(const int32_t *offsets, int G, int max_rows, int unit,
                              int pad, int32_t *checked, int32_t *mprefix, int32_t *pre256,
                              int32_t *poff, int32_t *err) {
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
  int sm = 0, s2 = 0, sp = 0, mt[8], m2[8], pr[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // G <= 256: eight groups per lane
    const int g = lane * 8 + j;
    const int n = (ok && g < G) ? offsets[g + 1] - offsets[g] : 0;
    mt[j] = ceil_div(n, unit);
    pr[j] = ceil_div(n, pad) * pad;
    m2[j] = ceil_div(n, 2 * kRowTile);
    sm += mt[j];
    s2 += m2[j];
    sp += pr[j];
  }
  int im = sm, i2 = s2, ip = sp;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, im, o), u = __shfl_up_sync(0xffffffffu, ip, o);
    const int w = __shfl_up_sync(0xffffffffu, i2, o);
    if (lane >= o) {
      im += v;
      i2 += w;
      ip += u;
    }
  }
  int rm = im - sm, r2 = i2 - s2, rp = ip - sp;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int g = lane * 8 + j;
    if (g < G) {
      mprefix[g] = rm;
      pre256[g] = r2;
      poff[g] = rp;
      checked[g] = ok ? offsets[g] : 0;
    }
    rm += mt[j];
    r2 += m2[j];
    rp += pr[j];
  }
  if (lane == 31) {
    mprefix[G] = im;
    pre256[G] = i2;
    poff[G] = ip;
    checked[G] = ok ? offsets[G] : 0;
  }
  if (!ok && lane == 0) report_error(err, MOE_DEVERR_OFFSETS, bad);
}

__global__ void k_one_group(int n, int unit, int pad, int32_t *offsets, int32_t *mprefix, int32_t *pre256,
                            int32_t *poff) {
  pdl_wait();
  pdl_trigger();
  offsets[0] = mprefix[0] = pre256[0] = poff[0] = 0;
  offsets[1] = n;
  mprefix[1] = ceil_div(n, unit);
  pre256[1] = ceil_div(n, 2 * kRowTile);
  poff[1] = ceil_div(n, pad) * pad;
}

template <class TD, class TW, bool VEC>
cudaError_t ffn_bwd_f32(const FfnGradArgs &a, cudaStream_t st) {
  const bool glu = a.act == MOE_ACT_SWIGLU;
  const dim3 b(kThreads);
  const int nt = ceil_div(a.F, BN), tiles = nt * a.m_tiles_ub;
  const int sums = a.db2 ? ceil_div(a.d, 64) * a.m_tiles_ub : 0;
  cudaError_t e =
      glu ? launch_pdl(k_dact<Tile<TD::BM>, true, VEC>, dim3(tiles + sums), b, 0, st, a, nt, tiles)
          : launch_pdl(k_dact<Tile<TD::BM>, false, VEC>, dim3(tiles + sums), b, 0, st, a, nt, tiles);
  if (e != cudaSuccess) return e;
  Reduce q = reduce_blocks(a);
  q.first = a.mprefix;
  q.unit = 1;
  q.dots = nt;
  Products p{};
  p.dx_n = ceil_div(a.d, TD::BN);
  p.splits = a.dx ? dx_splits(a.rows, a.m_tiles_ub, a.d, a.F, glu) : 1;
  p.piece = ceil_div(ceil_div(a.F, p.splits), 32) * 32;
  p.splits = ceil_div(a.F, p.piece);
  p.dx = a.dx ? p.dx_n * a.m_tiles_ub * p.splits : 0;
  auto job = [&](const void *x, const void *y, void *c, int M, int N) {
    if (c == nullptr) return;
    const int j = p.jobs++;
    p.a[j] = static_cast<const float *>(x);
    p.b[j] = static_cast<const float *>(y);
    p.c[j] = static_cast<float *>(c);
    p.M[j] = M;
    p.N[j] = N;
    p.tiles[j] = ceil_div(M, TW::BM) * ceil_div(N, TW::BN);
    p.dw += a.G * p.tiles[j];
  };
  job(a.dg, a.x, a.dw1, a.F, a.d);
  if (glu) job(a.du, a.x, a.dw3, a.F, a.d);
  job(a.dy, a.h, a.dw2, a.d, a.F);
  const int blocks = p.dx + p.dw + q.db1 + q.db2 + q.rows;
  if (blocks == 0) return cudaSuccess;
  e = launch_pdl(k_products<TD, TW, VEC>, dim3(blocks), b, 0, st, a, p, q);
  if (e != cudaSuccess || p.dx == 0 || p.splits == 1) return e;
  return launch_pdl(k_dx_sum, dim3((unsigned)(((size_t)a.rows * a.d / 4 + kThreads - 1) / kThreads)),
                    b, 0, st, a, p.splits);
}

// The weights' gradients take 128-row tiles unless those leave SMs without one. With 128
// rows, they and dx take 128 columns where those give every SM its two blocks: 2.86 -> 2.69
// ms with 448 tiles of dW1, but 313 -> 331 us with 180.
template <class TD, bool VEC>
cudaError_t ffn_bwd_f32(const FfnGradArgs &a, cudaStream_t st) {
  const long long m = (long long)a.G * ceil_div(a.F, 128);
  if constexpr (TD::BM == 128) {
    if (m * ceil_div(a.d, 128) >= 2 * 148)
      return ffn_bwd_f32<Tile<128, 128>, Tile<128, 128>, VEC>(a, st);
  }
  return m * ceil_div(a.d, BN) >= 148 ? ffn_bwd_f32<TD, Tile<128>, VEC>(a, st)
                                      : ffn_bwd_f32<TD, Tile<32>, VEC>(a, st);
}
template <class TD>
cudaError_t ffn_bwd_f32(const FfnGradArgs &a, cudaStream_t st) {
  return a.F % 4 == 0 ? ffn_bwd_f32<TD, true>(a, st) : ffn_bwd_f32<TD, false>(a, st);  // d always is
}

// dx of the padded rows from its parts, in order: a warp per row
template <typename TO>
__global__ void __launch_bounds__(kThreads) k_dx_join(FfnGradArgs s, int splits) {
  pdl_wait();
  pdl_trigger();
  const int p = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (p >= s.poff[s.G]) return;
  int lo = 0, hi = s.G - 1;  // last g with poff[g] <= p
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.poff[mid] <= p) lo = mid; else hi = mid - 1;
  }
  const int local = p - s.poff[lo];
  if (local >= s.offsets[lo + 1] - s.offsets[lo]) return;
  const float *from = s.dx_part + (size_t)p * s.d;
  TO *to = static_cast<TO *>(s.dx) + (size_t)(s.dx_off[lo] + local) * s.d;
  const size_t all = (size_t)s.rows * s.d;
  for (int i = 4 * lane; i < s.d; i += 128) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = 0; j < splits; ++j) {
      const float4 q = __ldg(reinterpret_cast<const float4 *>(from + j * all + i));
      v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
    }
    if constexpr (sizeof(TO) == 4)
      *reinterpret_cast<float4 *>(to + i) = v;
    else
      *reinterpret_cast<uint2 *>(to + i) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

// bf16: the steps on the tensor cores
cudaError_t ffn_bwd_tc(const FfnGradArgs &a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (a.db2) {
    e = launch_pdl(k_col_sums<__nv_bfloat16>, dim3(ceil_div(a.d, 64) * a.m_tiles_ub), dim3(kThreads),
                   0, st, a, a.tile_rows);
    if (e != cudaSuccess) return e;
  }
  e = launch_act_grad_tc(a, st);
  if (e != cudaSuccess) return e;
  Reduce q = reduce_blocks(a);
  q.first = a.poff;
  q.unit = 32;  // db1's partials are sums over 32 padded rows, row_dot's over 32 columns
  q.dots = a.F / 32;
  if (q.db1 + q.db2 + q.rows > 0) {
    e = launch_pdl(k_reduce<__nv_bfloat16>, dim3(q.db1 + q.db2 + q.rows), dim3(kThreads), 0, st, a,
                   q);
    if (e != cudaSuccess) return e;
  }
  const int splits =
      a.dx ? dx_splits_tc(a.pair_tiles_ub, a.d, a.F, a.act == MOE_ACT_SWIGLU) : 1;
  e = launch_products_tc(a, splits, st);
  if (e != cudaSuccess || splits == 1) return e;
  const dim3 g(ceil_div(a.rows, 8)), b(kThreads);
  return a.dx_f32 ? launch_pdl(k_dx_join<float>, g, b, 0, st, a, splits)
                  : launch_pdl(k_dx_join<__nv_bfloat16>, g, b, 0, st, a, splits);
}

}  // namespace

cudaError_t launch_grad_tables(const int32_t *offsets, int G, int max_rows, int unit, int pad,
                               int32_t *checked, int32_t *mprefix, int32_t *pre256, int32_t *poff,
                               int32_t *err, cudaStream_t st) {
  return launch_pdl(k_grad_tables, dim3(1), dim3(32), 0, st, offsets, G, max_rows, unit, pad, checked,
                    mprefix, pre256, poff, err);
}

cudaError_t launch_one_group(int n, int unit, int pad, int32_t *offsets, int32_t *mprefix,
                             int32_t *pre256, int32_t *poff, cudaStream_t st) {
  return launch_pdl(k_one_group, dim3(1), dim3(1), 0, st, n, unit, pad, offsets, mprefix, pre256,
                    poff);
}

cudaError_t launch_ffn_bwd(const FfnGradArgs &a, int dtype, cudaStream_t st) {
  if (dtype != MOE_DTYPE_F32) return ffn_bwd_tc(a, st);
  if (a.tile_rows == 8) return ffn_bwd_f32<Tile<8>>(a, st);
  return a.tile_rows == 32 ? ffn_bwd_f32<Tile<32>>(a, st) : ffn_bwd_f32<Tile<128>>(a, st);
}

}  // namespace moe
