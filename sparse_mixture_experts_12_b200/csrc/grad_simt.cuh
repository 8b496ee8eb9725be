// fp32 matrix products of the gradients on CUDA cores (FFMA): 128 x 64 tiles of
// C = A B with B row-major [K, N], A row-major [M, K] or (AT) [K, M].
//
// Two groupings:
//  * rows:  the rows of A and C are expert-contiguous (or one plain matrix); B is
//           the expert's own. Up to two (A, B) pairs add into the same C.
//  * k:     the reduction runs over an expert's rows (or over one of `chunk`-row
//           pieces of a plain matrix), and C is the expert's (the piece's) own. Up
//           to three independent (A, B, C) jobs share a launch.
#pragma once

#include "kernels.cuh"

namespace moe {
namespace simt {

constexpr int BM = kRowTile, BN = 64, BK = 32;
constexpr int TM = 8, TN = 4;  // per-thread micro tile; (BM/TM)*(BN/TN) = 256 threads
constexpr int kAPer = BM * BK / 256, kBPer = BN * BK / 256;

// the expert of 128-row tile mt (mprefix [G+1]), or -1 past the last tile
__device__ __forceinline__ int group_of_tile(const int32_t *mprefix, int G, int mt) {
  if (mt >= mprefix[G]) return -1;
  int lo = 0, hi = G - 1;  // last g with mprefix[g] <= mt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mprefix[mid] <= mt) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <typename TA, typename TB, typename TO>
struct Gemm {
  const TA *a[3];
  const TB *b[3];
  TO *c[3];
  int M[3], N[3];       // k grouping: per job; rows: M[0] = rows, N[0]
  int lda[3], ldb[3];
  int nseg;             // rows: (A, B) pairs added; k: jobs
  int K;                // rows: reduction length; k: rows of the plain matrix
  int chunk;            // k, plain matrix: rows per piece
  int G;                // experts (k, plain matrix: pieces)
  const int32_t *offsets, *mprefix;  // nullptr: a plain matrix
};

template <typename TA, typename TB, typename TO, bool KGROUP>
__global__ void __launch_bounds__(256) k_gemm(Gemm<TA, TB, TO> s) {
  __shared__ __align__(16) float As[BK][BM + 4];
  __shared__ __align__(16) float Bs[BK][BN + 4];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  int job = 0, g = 0, row0, nrows, K;  // row0: first row of A and C (rows) or of the reduction (k)
  const int n0 = blockIdx.x * BN;
  int m0;
  if (KGROUP) {
    job = blockIdx.z / s.G;
    g = blockIdx.z % s.G;
    m0 = blockIdx.y * BM;
    if (m0 >= s.M[job] || n0 >= s.N[job]) return;
    nrows = min(BM, s.M[job] - m0);
    const int e0 = s.offsets ? s.offsets[g] : g * s.chunk;
    const int e1 = s.offsets ? s.offsets[g + 1] : min(s.K, e0 + s.chunk);
    row0 = e0;
    K = max(0, e1 - e0);
  } else {
    m0 = blockIdx.y * BM;
    if (s.offsets) {
      g = group_of_tile(s.mprefix, s.G, blockIdx.y);
      if (g < 0) return;
      m0 = s.offsets[g] + ((int)blockIdx.y - s.mprefix[g]) * BM;
      nrows = min(BM, s.offsets[g + 1] - m0);
    } else {
      nrows = min(BM, s.M[0] - m0);
    }
    row0 = m0;
    K = s.K;
  }
  const int N = s.N[job];
  const int tx = tid % (BN / TN), ty = tid / (BN / TN);
  float acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
  const int nseg = KGROUP ? 1 : s.nseg;
  for (int seg = 0; seg < nseg; ++seg) {
    const int q = KGROUP ? job : seg;
    const int lda = s.lda[q], ldb = s.ldb[q];
    const TA *ap = s.a[q] + (size_t)row0 * lda + (KGROUP ? m0 : 0);
    const TB *bp = s.b[q] + (KGROUP ? (size_t)row0 : (size_t)g * s.K) * ldb + n0;
    float ra[kAPer], rb[kBPer];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int j = 0; j < kAPer; ++j) {
        const int i = tid + 256 * j;
        const int m = KGROUP ? i % BM : i / BK, kk = KGROUP ? i / BM : i % BK;
        const bool ok = m < nrows && k0 + kk < K;
        ra[j] = ok ? Elem<TA>::to_f(ap[KGROUP ? (size_t)(k0 + kk) * lda + m
                                              : (size_t)m * lda + k0 + kk])
                   : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kBPer; ++j) {
        const int i = tid + 256 * j, n = i % BN, kk = i / BN;
        const bool ok = n0 + n < N && k0 + kk < K;
        rb[j] = ok ? Elem<TB>::to_f(bp[(size_t)(k0 + kk) * ldb + n]) : 0.f;
      }
    };
    fetch(0);
    for (int k0 = 0; k0 < K; k0 += BK) {
#pragma unroll
      for (int j = 0; j < kAPer; ++j) {
        const int i = tid + 256 * j;
        if (KGROUP) As[i / BM][i % BM] = ra[j];
        else As[i % BK][i / BK] = ra[j];
      }
#pragma unroll
      for (int j = 0; j < kBPer; ++j) {
        const int i = tid + 256 * j;
        Bs[i / BN][i % BN] = rb[j];
      }
      __syncthreads();
      if (k0 + BK < K) fetch(k0 + BK);
#pragma unroll
      for (int kk = 0; kk < BK; ++kk) {
        float av[TM], bv[TN];
#pragma unroll
        for (int i = 0; i < TM; i += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(&As[kk][ty * TM + i]);
          av[i] = v.x; av[i + 1] = v.y; av[i + 2] = v.z; av[i + 3] = v.w;
        }
        const float4 v = *reinterpret_cast<const float4 *>(&Bs[kk][tx * TN]);
        bv[0] = v.x; bv[1] = v.y; bv[2] = v.z; bv[3] = v.w;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
      }
      __syncthreads();
    }
  }
  TO *c = s.c[job] + (KGROUP ? (size_t)g * s.M[job] * N : 0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = ty * TM + i;
    if (m >= nrows) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = n0 + tx * TN + j;
      if (n < N) c[(size_t)(m0 + m) * N + n] = Elem<TO>::from_f(acc[i][j]);
    }
  }
}

}  // namespace simt
}  // namespace moe
