// fp32 tiles on CUDA cores (FFMA) shared by the gradients: 256 threads compute a BM x BN
// tile of C = A B with B row-major [K, N], A row-major [M, K] or (AT) [K, M], from K slices
// in shared memory while the next slice is fetched into registers.
//
// BM 128 (8 x 4 values a thread, 16-wide slices; 8 x 8 where BN is 128, two thirds of the
// reads of shared memory per product) is for experts with many rows, BM 32 (2 x 4, 32-wide)
// and BM 8 (1 x 2) for few: on 16 rows a 128-row tile took 22 us where the 32-row one takes
// 8, and on a handful the 32-row one computes more than it loads. Products are issued in
// pairs, which leaves issue slots for the reads: 7 to 13 % of the expert gradients' time.
#pragma once

#include "kernels.cuh"

namespace moe {
namespace simt {

constexpr int BN = 64, kThreads = 256;  // BN: columns of a tile but the widest
template <int BM_, int BN_ = 64>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, BK = BM == 128 ? 16 : 32;
  static constexpr int TN = BN == 128 ? 8 : (BM == 8 ? 2 : 4);  // columns a thread
  static constexpr int TX = BN / TN, TY = kThreads / TX, TM = BM / TY;
  static constexpr int LDA = BM + (BM == 32 ? 2 : 4), LDB = BN + 4;
  // thread tx has columns TC tx .. TC tx + TC - 1, and with TN = 8 those 64 further on
  static constexpr int TC = TN == 8 ? 4 : TN;
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
// c += a b for two values at once: one instruction, each rounded as an fmaf
__device__ __forceinline__ void fma2(float &c0, float &c1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "+f"(c0), "+f"(c1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
template <int TM, int TN>
__device__ __forceinline__ void outer(float (&acc)[TM][TN], const float (&a)[TM], const float *b) {
  float q[TN];
  if constexpr (TN == 8) {
    float lo[4], hi[4];
    values(b, lo);
    values(b + 64, hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[j] = lo[j];
      q[4 + j] = hi[j];
    }
  } else {
    values(b, q);
  }
  if constexpr (TM >= 4) {
#pragma unroll
    for (int i = 0; i < TM; i += 2)
#pragma unroll
      for (int j = 0; j < TN; ++j) fma2(acc[i][j], acc[i + 1][j], a[i], a[i + 1], q[j], q[j]);
  } else {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; j += 2) fma2(acc[i][j], acc[i][j + 1], a[i], a[i], q[j], q[j + 1]);
  }
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
                                         const float *a, size_t lda, int rows, const float *b,
                                         size_t ldb, int cols, int K) {
  const int tx = threadIdx.x % T::TX, ty = threadIdx.x / T::TX;
  Slice<T::BM, T::BK, T::LDA, !AT, VEC> sa;
  Slice<T::BN, T::BK, T::LDB, false, VEC> sb;
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
      outer(acc, av, &s.b[k][tx * T::TC]);
    }
  }
}

// c: the tile's first element; `add`: to what the same thread stored there before
template <class T, bool VEC>
__device__ __forceinline__ void store_tile(const float (&acc)[T::TM][T::TN], float *c, size_t ldc,
                                           int rows, int cols, bool add = false) {
  constexpr int TC = T::TC;
  const int tx = threadIdx.x % T::TX, ty = threadIdx.x / T::TX;
#pragma unroll
  for (int i = 0; i < T::TM; ++i) {
    const int m = ty * T::TM + i;
    if (m >= rows) continue;
#pragma unroll
    for (int g = 0; g < T::TN / TC; ++g) {
      const int n0 = 64 * g + tx * TC, n = cols - n0;
      float *p = c + (size_t)m * ldc + n0;
      const float *v = &acc[i][g * TC];
      if constexpr (VEC) {
        if (n <= 0) continue;
        if constexpr (TC == 4) {
          float4 o = make_float4(v[0], v[1], v[2], v[3]);
          if (add) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            o = make_float4(q.x + o.x, q.y + o.y, q.z + o.z, q.w + o.w);
          }
          *reinterpret_cast<float4 *>(p) = o;
        } else {
          float2 o = make_float2(v[0], v[1]);
          if (add) {
            const float2 q = *reinterpret_cast<const float2 *>(p);
            o = make_float2(q.x + o.x, q.y + o.y);
          }
          *reinterpret_cast<float2 *>(p) = o;
        }
      } else {
#pragma unroll
        for (int j = 0; j < TC; ++j)
          if (j < n) p[j] = add ? p[j] + v[j] : v[j];
      }
    }
  }
}

// Rows in one running sum of a weight's gradient: the fp32 error of a sum grows with the root
// of its length, and a tile's read and write for each part are few beside its products' reads.
// (65536 rows: 4.6e-6 of the result in one sum, 6.7e-7 in parts.)
constexpr int kSumRows = 1024;
// c = A^T B over K rows, in such parts, which the tile's threads add up in c
template <class T, bool VEC, bool VECC>
__device__ __forceinline__ void sum_rows(GemmSmem<T> &s, const float *a, size_t lda, int rows,
                                         const float *b, size_t ldb, int cols, int K, float *c,
                                         size_t ldc) {
  int k0 = 0;
  do {
    float acc[T::TM][T::TN];
    clear(acc);
    mma_tile<T, true, VEC>(s, acc, a + (size_t)k0 * lda, lda, rows, b + (size_t)k0 * ldb, ldb, cols,
                           min(kSumRows, K - k0));
    store_tile<T, VECC>(acc, c, ldc, min(T::BM, rows), min(T::BN, cols), k0 > 0);
    k0 += kSumRows;
  } while (k0 < K);
}

}  // namespace simt
}  // namespace moe
