// Gradients of the token movement: the gate-weighted combine and the
// expert-contiguous permutation, and the padded rows that the experts' gradients start
// with.
//
//   combine  y[t] = sum_s g[t,s] Y[inv[t,s]]   dY[inv[t,s]] = g[t,s] dy[t]
//                                              dg[t,s] = <dy[t], Y[inv[t,s]]>
//   permute  X[inv[t,s]] = x[t]                dx[t] = sum_s dX[inv[t,s]]
//
// Both are gathers over (token, slot), like the forward combine: every output is
// written by one warp (or the warps of one block), so there are no atomics and the
// result does not depend on the schedule. A dropped slot (inv < 0) reads and writes
// no row and has a zero gate gradient.
#include "grad.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// the row of pair p, or -1: dropped, or outside [0, R) (recorded)
__device__ __forceinline__ int checked_row(const int32_t *inv, size_t p, int R, int32_t *err,
                                           bool report) {
  int r = inv[p];
  if (r < -1 || r >= R) {
    if (report) report_error(err, MOE_DEVERR_ROW_INDEX, (int32_t)p);
    r = -1;
  }
  return r;
}

// `wpt` warps of a block share a token: warp `sub` of them takes the vectors
// 32 (sub + wpt i) + lane. NB vectors of dy and of each kept slot's row are requested
// before any is used. DRAM bounds it: 437 MB (8192 tokens, six rows of 4 KB each) take 80
// us, 85 % of a copy's rate; a call of 32 tokens is its launch.
template <typename T, int KMAX, int NB>
__global__ void __launch_bounds__(kThreads) k_combine_bwd(CombineBwdArgs a, int wpt) {
  constexpr int VE = Elem<T>::kPerVec;
  __shared__ float red[kWarps][KMAX];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % wpt;
  const int t = blockIdx.x * (kWarps / wpt) + warp / wpt;
  pdl_wait();
  pdl_trigger();
  const int k = a.k;
  const bool live = t < a.T;
  int row[KMAX];
  float g[KMAX], dot[KMAX];
#pragma unroll
  for (int s = 0; s < KMAX; ++s) {
    row[s] = -1;
    g[s] = dot[s] = 0.f;
    if (live && s < k) {
      row[s] = checked_row(a.inv, (size_t)t * k + s, a.R, a.err, lane == 0 && sub == 0);
      if (a.dy_perm) g[s] = a.gate[(size_t)t * k + s];
    }
  }
  const int nvec = a.d / VE;
  const uint4 *dy = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.dy) + (size_t)t * a.d);
  const T *yp = static_cast<const T *>(a.y_perm);
  T *out = static_cast<T *>(a.dy_perm);
  bool any = false;
#pragma unroll
  for (int s = 0; s < KMAX; ++s) any |= row[s] >= 0;
  for (int v0 = sub * 32 + lane; any && v0 < nvec; v0 += 32 * wpt * NB) {
    uint4 q[NB], u[KMAX][NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int v = v0 + 32 * wpt * b;
      q[b] = v < nvec ? __ldg(dy + v) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (a.dgate) {
#pragma unroll
      for (int s = 0; s < KMAX; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int v = v0 + 32 * wpt * b;
          u[s][b] = (row[s] >= 0 && v < nvec)
                        ? __ldg(reinterpret_cast<const uint4 *>(yp + (size_t)row[s] * a.d) + v)
                        : make_uint4(0u, 0u, 0u, 0u);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int v = v0 + 32 * wpt * b;
      if (v >= nvec) break;
      float f[VE];
      unpack16(q[b], f);
#pragma unroll
      for (int s = 0; s < KMAX; ++s) {
        if (row[s] < 0) continue;
        if (a.dgate) {
          float y[VE];
          unpack16(u[s][b], y);
#pragma unroll
          for (int i = 0; i < VE; ++i) dot[s] = fmaf(f[i], y[i], dot[s]);
        }
        if (out) {
          float o[VE];
#pragma unroll
          for (int i = 0; i < VE; ++i) o[i] = g[s] * f[i];
          reinterpret_cast<uint4 *>(out + (size_t)row[s] * a.d)[v] = pack16(o);
        }
      }
    }
  }
  if (a.dgate == nullptr) return;
#pragma unroll
  for (int s = 0; s < KMAX; ++s) dot[s] = warp_sum(dot[s]);
  if (wpt > 1) {
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < KMAX; ++s) red[warp][s] = dot[s];
    }
    __syncthreads();
    if (sub == 0) {
#pragma unroll
      for (int s = 0; s < KMAX; ++s)
        for (int w = 1; w < wpt; ++w) dot[s] += red[warp + w][s];
    }
  }
  if (live && sub == 0 && lane == 0) {
#pragma unroll
    for (int s = 0; s < KMAX; ++s)
      if (s < k) a.dgate[(size_t)t * k + s] = dot[s];
  }
}

// VE values as they lie in memory: 16 bytes of bf16, 16 or 32 of fp32
template <typename TI, int VE>
struct RawVec {
  static constexpr int N = VE * (int)sizeof(TI) / 16;
  uint4 u[N];
  __device__ __forceinline__ void load(const TI *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void add_to(float (&o)[VE]) const {
    constexpr int per = VE / N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[per];
      unpack16(u[i], f);
#pragma unroll
      for (int j = 0; j < per; ++j) o[i * per + j] += f[j];
    }
  }
};

// dx[t] = the kept slots' rows in slot order, then the addends; summed in fp32 and
// rounded once. TI: the rows' type. NB vectors of each row and addend are requested before
// any is used; one slot alone leaves room for four of them (32 -> 24 us on the top-1
// layer, whose rows are four vectors to a lane).
template <typename T, typename TI, int KMAX, int NB, int ADDS>
__global__ void __launch_bounds__(kThreads) k_permute_bwd(PermuteBwdArgs a, int wpt) {
  constexpr int VE = Elem<T>::kPerVec;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % wpt;
  const int t = blockIdx.x * (kWarps / wpt) + warp / wpt;
  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;
  const float *add[2] = {a.add0 ? a.add0 + (size_t)t * a.d : nullptr,
                         a.add1 ? a.add1 + (size_t)t * a.d : nullptr};
  const int nvec = a.d / VE;
  RawVec<float, VE> av[ADDS][NB];
  auto request = [&](int v0) {  // the addends do not wait for the slots' rows to be known
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int v = v0 + 32 * wpt * b;
#pragma unroll
      for (int i = 0; i < ADDS; ++i)
        if (add[i] && v < nvec) av[i][b].load(add[i] + (size_t)v * VE);
    }
  };
  request(sub * 32 + lane);
  int row[KMAX];
#pragma unroll
  for (int s = 0; s < KMAX; ++s)
    row[s] = s < a.k ? checked_row(a.inv, (size_t)t * a.k + s, a.R, a.err, lane == 0 && sub == 0)
                     : -1;
  const TI *xp = static_cast<const TI *>(a.dx_perm);
  T *dx = static_cast<T *>(a.dx) + (size_t)t * a.d;
  for (int v0 = sub * 32 + lane; v0 < nvec; v0 += 32 * wpt * NB) {
    RawVec<TI, VE> f[KMAX][NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int v = v0 + 32 * wpt * b;
#pragma unroll
      for (int s = 0; s < KMAX; ++s)
        if (row[s] >= 0 && v < nvec) f[s][b].load(xp + (size_t)row[s] * a.d + (size_t)v * VE);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int v = v0 + 32 * wpt * b;
      if (v >= nvec) break;
      float o[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) o[i] = 0.f;
#pragma unroll
      for (int s = 0; s < KMAX; ++s)
        if (row[s] >= 0) f[s][b].add_to(o);
#pragma unroll
      for (int i = 0; i < ADDS; ++i)
        if (add[i]) av[i][b].add_to(o);
      reinterpret_cast<uint4 *>(dx)[v] = pack16(o);
    }
    request(v0 + 32 * wpt * NB);
  }
}

// NB vectors of two rows, requested before any is used, to up to kMaxTopK places
template <int N>
__device__ __forceinline__ void copy_rows(const PadRowsArgs &a, int from, const int (&to)[N],
                                          int v0, int step) {
  constexpr int NB = 4;
  const int nvec = a.row_bytes / 16;
  const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) +
                                                   (size_t)from * a.row_bytes);
  const uint4 *dy = reinterpret_cast<const uint4 *>(static_cast<const char *>(a.dy) +
                                                    (size_t)from * a.row_bytes);
  for (; v0 < nvec; v0 += step * NB) {
    uint4 p[NB], q[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int v = v0 + step * b;
      if (v < nvec) {
        p[b] = __ldg(x + v);
        q[b] = __ldg(dy + v);
      }
    }
#pragma unroll
    for (int s = 0; s < N; ++s) {
      if (to[s] < 0) continue;
      uint4 *xo = reinterpret_cast<uint4 *>(static_cast<char *>(a.x_pad) +
                                            (size_t)to[s] * a.row_bytes);
      uint4 *yo = reinterpret_cast<uint4 *>(static_cast<char *>(a.dy_pad) +
                                            (size_t)to[s] * a.row_bytes);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int v = v0 + step * b;
        if (v < nvec) {
          xo[v] = p[b];
          yo[v] = q[b];
        }
      }
    }
  }
}
__device__ __forceinline__ void zero_rows(const PadRowsArgs &a, int to, int v0, int step) {
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  uint4 *xo = reinterpret_cast<uint4 *>(static_cast<char *>(a.x_pad) + (size_t)to * a.row_bytes);
  uint4 *yo = reinterpret_cast<uint4 *>(static_cast<char *>(a.dy_pad) + (size_t)to * a.row_bytes);
  for (int v = v0; v < a.row_bytes / 16; v += step) xo[v] = yo[v] = z;
}
// last g < G with first[g] <= r (r below first[G])
__device__ __forceinline__ int group_of(const int32_t *first, int G, int r) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Expert-contiguous rows to padded rows: a warp per padded row. It costs a copy of x and dy
// (22 us of 1350 on 16384 rows of 1024, 48 of 7200 on 8192 rows of 4096), against masks in
// every K slice of the weights' gradients.
__global__ void __launch_bounds__(kThreads) k_pad_rows(PadRowsArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int p = blockIdx.x * kWarps + warp;
  if (p >= a.poff[a.G]) return;
  const int g = group_of(a.poff, a.G, p), local = p - a.poff[g];
  if (local < a.offsets[g + 1] - a.offsets[g]) {
    const int to[1] = {p};
    copy_rows<1>(a, a.offsets[g] + local, to, lane, 32);
  } else {
    zero_rows(a, p, lane, 32);
  }
}

// Tokens to their slots' padded rows: `wpt` warps per token in the first blocks; the
// blocks behind them zero each expert's padding rows.
__global__ void __launch_bounds__(kThreads) k_gather_rows(PadRowsArgs a, int wpt, int token_blocks) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x >= token_blocks) {
    const int g = blockIdx.x - token_blocks;
    for (int p = a.poff[g] + a.offsets[g + 1] - a.offsets[g] + warp; p < a.poff[g + 1];
         p += kWarps) {
      zero_rows(a, p, lane, 32);
      if (lane == 0) a.row_w[p] = 0.f;
    }
    return;
  }
  const int sub = warp % wpt;
  const int t = blockIdx.x * (kWarps / wpt) + warp / wpt;
  if (t >= a.T) return;
  const int live = a.offsets[a.G];  // rows past it belong to nobody
  int row[kMaxTopK];
  bool any = false;
#pragma unroll
  for (int s = 0; s < kMaxTopK; ++s) {
    row[s] = -1;
    if (s < a.k) {
      const size_t p = (size_t)t * a.k + s;
      const bool first = lane == 0 && sub == 0;
      const int r = checked_row(a.inv, p, live, a.err, first);
      if (r >= 0) {
        const int g = group_of(a.offsets, a.G, r);
        row[s] = r + a.poff[g] - a.offsets[g];
      }
      if (first) {
        a.inv_pad[p] = row[s];
        if (row[s] >= 0) a.row_w[row[s]] = a.gate[p];
      }
    }
    any |= row[s] >= 0;
  }
  if (any) copy_rows<kMaxTopK>(a, t, row, sub * 32 + lane, 32 * wpt);
}

// Warps per token: one while the tokens alone give the GPU its warps, more (up to
// the block's eight, and no more than the row has 32-vector pieces) when there are
// few tokens and the rows are long.
int warps_per_token(int T, int nvec) {
  int wpt = 1;
  while (wpt < kWarps && (long long)T * wpt < 148 * 16 && 32 * wpt < nvec) wpt *= 2;
  return wpt;
}

template <typename T>
cudaError_t combine_bwd(const CombineBwdArgs &a, cudaStream_t st) {
  const int wpt = warps_per_token(a.T, a.d / Elem<T>::kPerVec);
  const dim3 g(ceil_div(a.T, kWarps / wpt)), b(kThreads);
  if (a.k <= 2) return launch_pdl(k_combine_bwd<T, 2, 4>, g, b, 0, st, a, wpt);
  return launch_pdl(k_combine_bwd<T, kMaxTopK, 1>, g, b, 0, st, a, wpt);
}

template <typename T, typename TI>
cudaError_t permute_bwd(const PermuteBwdArgs &a, cudaStream_t st) {
  const int wpt = warps_per_token(a.T, a.d / Elem<T>::kPerVec);
  const dim3 g(ceil_div(a.T, kWarps / wpt)), b(kThreads);
  auto run = [&](auto kernel) { return launch_pdl(kernel, g, b, 0, st, a, wpt); };
  if constexpr (sizeof(TI) == 4) {  // the second addend comes with fp32 rows only
    if (a.add1) {
      if (a.k == 1) return run(k_permute_bwd<T, TI, 1, 2, 2>);
      if (a.k == 2) return run(k_permute_bwd<T, TI, 2, 2, 2>);
      return run(k_permute_bwd<T, TI, kMaxTopK, 1, 2>);
    }
  }
  if (a.k == 1) return run(k_permute_bwd<T, TI, 1, 4, 1>);
  if (a.k == 2) return run(k_permute_bwd<T, TI, 2, 2, 1>);
  return run(k_permute_bwd<T, TI, kMaxTopK, 1, 1>);
}

}  // namespace

cudaError_t launch_combine_bwd(const CombineBwdArgs &a, int dtype, cudaStream_t st) {
  if (a.T == 0 || (a.dy_perm == nullptr && a.dgate == nullptr)) return cudaSuccess;
  return dtype == MOE_DTYPE_F32 ? combine_bwd<float>(a, st) : combine_bwd<__nv_bfloat16>(a, st);
}

cudaError_t launch_permute_bwd(const PermuteBwdArgs &a, int dtype, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  if (dtype == MOE_DTYPE_F32) return permute_bwd<float, float>(a, st);
  return a.dx_perm_f32 ? permute_bwd<__nv_bfloat16, float>(a, st)
                       : permute_bwd<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_pad_rows(const PadRowsArgs &a, cudaStream_t st) {
  if (a.inv == nullptr)
    return launch_pdl(k_pad_rows, dim3(ceil_div(a.rows, kWarps)), dim3(kThreads), 0, st, a);
  const int wpt = warps_per_token(a.T, a.row_bytes / 16);
  const int tb = ceil_div(a.T, kWarps / wpt);
  return launch_pdl(k_gather_rows, dim3(tb + a.G), dim3(kThreads), 0, st, a, wpt, tb);
}

}  // namespace moe
