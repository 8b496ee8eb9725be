// fp32 tiles on CUDA cores (FFMA) shared by the gradients: 256 threads compute a
// BM x 64 tile of C = A B with B row-major [K, N], A row-major [M, K] or (AT) [K, M], from
// K slices in shared memory while the next slice is fetched into registers.
//
// BM 128 (8 x 4 values a thread, 16-wide slices) is for experts with many rows, BM 32 (2 x
// 4, 32-wide) and BM 8 (1 x 2) for few: on 16 rows a 128-row tile took 22 us where the
// 32-row one takes 8, and on a handful the 32-row one computes more than it loads.
#pragma once

#include "kernels.cuh"

namespace moe {
namespace simt {

constexpr int BN = 64, kThreads = 256;
template <int BM_>
struct Tile {
  static constexpr int BM = BM_, BK = BM == 128 ? 16 : 32;
  static constexpr int TN = BM == 8 ? 2 : 4, TX = BN / TN;  // columns a thread, threads across
  static constexpr int TY = kThreads / TX, TM = BM / TY;    // threads down, rows a thread
  static constexpr int LDA = BM + (BM == 32 ? 2 : 4), LDB = BN + 4;
};

// the expert of row tile mt (mprefix [G+1]), or -1 past the last tile
__device__ __forceinline__ int group_of_tile(const int32_t *mprefix, int G, int mt) {
  if (mt >= mprefix[G]) return -1;
  int lo = 0, hi = G - 1;  // last g with mprefix[g] <= mt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mprefix[mid] <= mt) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// up to four consecutive values, n of them inside (n <= 0: none). VEC: 16-byte aligned,
// and all dimensions are multiples of 4.
template <bool VEC>
__device__ __forceinline__ float4 ld4(const float *p, int n) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (VEC) {
    if (n > 0) v = __ldg(reinterpret_cast<const float4 *>(p));
  } else {
    if (n > 0) v.x = __ldg(p);
    if (n > 1) v.y = __ldg(p + 1);
    if (n > 2) v.z = __ldg(p + 2);
    if (n > 3) v.w = __ldg(p + 3);
  }
  return v;
}

// A slice of an operand with ROWS rows (of M or N), BK wide, in registers and then in
// shared memory as [BK][LD]. KMAJOR: the reduction's index is the contiguous one.
template <int ROWS, int BK, int LD, bool KMAJOR, bool VEC>
struct Slice {
  static constexpr int kAll = ROWS * BK / 4, N4 = (kAll + kThreads - 1) / kThreads;
  float4 r[N4];
  __device__ __forceinline__ void fetch(const float *p, size_t ld, int rows, int k0, int K) {
#pragma unroll
    for (int j = 0; j < N4; ++j) {
      const int i = threadIdx.x + kThreads * j;
      if (kAll % kThreads && i >= kAll) break;
      if (KMAJOR) {
        const int m = i / (BK / 4), k = k0 + (i % (BK / 4)) * 4;
        r[j] = ld4<VEC>(p + (size_t)m * ld + k, m < rows ? K - k : 0);
      } else {
        const int k = k0 + i / (ROWS / 4), m = (i % (ROWS / 4)) * 4;
        r[j] = ld4<VEC>(p + (size_t)k * ld + m, k < K ? rows - m : 0);
      }
    }
  }
  __device__ __forceinline__ void put(float (*s)[LD]) const {
#pragma unroll
    for (int j = 0; j < N4; ++j) {
      const int i = threadIdx.x + kThreads * j;
      if (kAll % kThreads && i >= kAll) break;
      if (KMAJOR) {
        const int m = i / (BK / 4), k = (i % (BK / 4)) * 4;
        s[k][m] = r[j].x;
        s[k + 1][m] = r[j].y;
        s[k + 2][m] = r[j].z;
        s[k + 3][m] = r[j].w;
      } else {
        const int k = i / (ROWS / 4), m = (i % (ROWS / 4)) * 4;
        if (LD % 4 == 0) {
          *reinterpret_cast<float4 *>(&s[k][m]) = r[j];
        } else {
          *reinterpret_cast<float2 *>(&s[k][m]) = make_float2(r[j].x, r[j].y);
          *reinterpret_cast<float2 *>(&s[k][m + 2]) = make_float2(r[j].z, r[j].w);
        }
      }
    }
  }
};

// N consecutive values of shared memory
template <int N>
__device__ __forceinline__ void values(const float *p, float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + i);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else if constexpr (N == 2) {
    const float2 q = *reinterpret_cast<const float2 *>(p);
    v[0] = q.x; v[1] = q.y;
  } else {
    v[0] = *p;
  }
}
template <int TM, int TN>
__device__ __forceinline__ void outer(float (&acc)[TM][TN], const float (&a)[TM], const float *b) {
  float q[TN];
  values(b, q);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i], q[j], acc[i][j]);
}
template <int TM, int TN>
__device__ __forceinline__ void clear(float (&acc)[TM][TN]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
}

// total += acc, acc = 0
template <int TM, int TN>
__device__ __forceinline__ void flush(float (&total)[TM][TN], float (&acc)[TM][TN]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      total[i][j] += acc[i][j];
      acc[i][j] = 0.f;
    }
}

template <class T>
struct GemmSmem {
  alignas(16) float a[T::BK][T::LDA];
  alignas(16) float b[T::BK][T::LDB];
};

// acc += A B over K for the tile whose operands begin at a and b: `rows` rows of A, `cols`
// columns of B inside
template <class T, bool AT, bool VEC>
__device__ __forceinline__ void mma_tile(GemmSmem<T> &s, float (&acc)[T::TM][T::TN],
                                         const float *a, size_t lda, int rows, const float *b, size_t ldb, int cols,
                                         int K) {
  const int tx = threadIdx.x % T::TX, ty = threadIdx.x / T::TX;
  Slice<T::BM, T::BK, T::LDA, !AT, VEC> sa;
  Slice<BN, T::BK, T::LDB, false, VEC> sb;
  sa.fetch(a, lda, rows, 0, K);
  sb.fetch(b, ldb, cols, 0, K);
  for (int k0 = 0; k0 < K; k0 += T::BK) {
    __syncthreads();
    sa.put(s.a);
    sb.put(s.b);
    __syncthreads();
    if (k0 + T::BK < K) {
      sa.fetch(a, lda, rows, k0 + T::BK, K);
      sb.fetch(b, ldb, cols, k0 + T::BK, K);
    }
#pragma unroll
    for (int k = 0; k < T::BK; ++k) {
      float av[T::TM];
      values(&s.a[k][ty * T::TM], av);
      outer(acc, av, &s.b[k][tx * T::TN]);
    }
  }
}

// c: the tile's first element
template <class T, bool VEC>
__device__ __forceinline__ void store_tile(const float (&acc)[T::TM][T::TN], float *c, size_t ldc,
                                           int rows, int cols) {
  constexpr int TN = T::TN;
  const int tx = threadIdx.x % T::TX, ty = threadIdx.x / T::TX;
#pragma unroll
  for (int i = 0; i < T::TM; ++i) {
    const int m = ty * T::TM + i;
    if (m >= rows) continue;
    float *p = c + (size_t)m * ldc + tx * TN;
    const int n = cols - tx * TN;
    if constexpr (VEC) {
      if (n <= 0) continue;
      if constexpr (TN == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      else
        *reinterpret_cast<float2 *>(p) = make_float2(acc[i][0], acc[i][1]);
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (j < n) p[j] = acc[i][j];
    }
  }
}

}  // namespace simt
}  // namespace moe
