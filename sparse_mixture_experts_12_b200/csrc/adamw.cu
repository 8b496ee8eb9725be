// AdamW over many tensors in one launch, and its C ABI entry point.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// computed in fp32 per element. The update reads and writes every element once and
// does some twenty operations on it: memory bandwidth bounds it.
//
// States of 8 bits: m and r = sqrt(v) are kept as e4m3 with one fp32 scale for each
// 256 consecutive elements, the block's largest magnitude standing at 448. The root
// halves the range of exponents that v needs. An element's step uses the new m and v
// before they are rounded. A nonzero r keeps at least the smallest code, so that an
// element with a small second moment beside large ones is not divided by eps alone.
#include <cuda_fp8.h>
#include <math.h>

#include <type_traits>

#include "api.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                            // elements per lane and step
constexpr int kQBlock = MOE_ADAMW_BLOCK;           // elements of one 8-bit scale: a warp's step
constexpr int kChunk = kThreads * kVec;            // elements per CTA
constexpr long long kMaxCtas = 0x7fffffff;         // of a grid
static_assert(kQBlock == 32 * kVec, "a warp's step is one scale block");
constexpr float kE4M3Max = 448.f;
constexpr float kE4M3Tiny = 0.001953125f;          // 2^-9, the smallest positive code
constexpr float kFloor = 7.8886090522101181e-31f;  // 2^-100: keeps 448 / top finite

struct Step {
  float b1, b2, e1, e2, keep, size, root2, eps, gs;
  // e1 = 1 - b1, e2 = 1 - b2; keep = 1 - lr wd; size = lr / c1; root2 = 1 / sqrt(c2);
  // c1 = 1 - b1^t, c2 = 1 - b2^t
};
__host__ __device__ inline void set_rates(Step &s, double lr, double decay, double c1, double c2) {
  s.keep = (float)(1.0 - lr * decay);
  s.size = (float)(lr / c1);
  s.root2 = (float)(1.0 / sqrt(c2));
}

template <int N>
struct Batch {
  moe_adamw_tensor_t t[N];
  unsigned first[N + 1];  // first CTA of each tensor
  int n;
  Step s;                 // without the device scalars
  // with step_dev or lr_dev the rates are worked out on the device
  double beta1, beta2, c1, c2;
  float lr, decay;
  const int64_t *step_dev;
  const float *lr_dev, *grad_scale, *found_inf;
};

// Eight elements as they lie in memory: raw(p) of any of the types, values by get()
template <typename T>
struct Raw8 {
  static constexpr int kWords = 8 * (int)sizeof(T) / 4;
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const T *p, int n) {
    if (n >= 8) {
      if constexpr (kWords == 2) {
        const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(p));
        u[0] = q.x; u[1] = q.y;
      } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p) + i / 4);
          u[i] = q.x; u[i + 1] = q.y; u[i + 2] = q.z; u[i + 3] = q.w;
        }
      }
      return;
    }
    // a tensor's end
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t w = 0;
      constexpr int per = 4 / (int)sizeof(T);
#pragma unroll
      for (int j = 0; j < per; ++j) {
        const int e = i * per + j;
        if (e < n) w |= bits(p[e]) << (8 * (int)sizeof(T) * j);
      }
      u[i] = w;
    }
  }
  static __device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
  static __device__ __forceinline__ uint32_t bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
  static __device__ __forceinline__ uint32_t bits(uint8_t v) { return v; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(u[i]);
        f[i + 1] = __uint_as_float(u[i + 1]);
      } else if constexpr (sizeof(T) == 2) {
        f[i] = __uint_as_float(u[i / 2] << 16);
        f[i + 1] = __uint_as_float(u[i / 2] & 0xffff0000u);
      } else {  // e4m3: exact in half precision
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(u[i / 4] >> (8 * (i & 2))), __NV_E4M3);
        const float2 q = __half22float2(__half2(h));
        f[i] = q.x;
        f[i + 1] = q.y;
      }
    }
  }
};
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(p) = pack16(f);
}
template <typename T>
__device__ __forceinline__ void store_any(T *p, int n, const float (&f)[8]) {
  if (n >= 8) {
    store8(p, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = Elem<T>::from_f(f[i]);
}
// A block's (a warp's 256 elements) codes and scale
template <bool ROOT>
__device__ __forceinline__ void quantise(uint8_t *codes, float *scale, int n, float (&f)[8]) {
  float top = kFloor;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
  top = warp_max(top);
  const float up = __fmul_rn(__frcp_rn(top), kE4M3Max);
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float2 y = make_float2(__fmul_rn(f[i], up), __fmul_rn(f[i + 1], up));
    if (ROOT) {
      y.x = f[i] > 0.f ? fmaxf(y.x, kE4M3Tiny) : y.x;
      y.y = f[i + 1] > 0.f ? fmaxf(y.y, kE4M3Tiny) : y.y;
    }
    // nearest even, saturating
    c[i / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (8 * (i & 2));
  }
  if (n >= 8) {
    *reinterpret_cast<uint2 *>(codes) = make_uint2(c[0], c[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) codes[i] = (uint8_t)(c[i / 4] >> (8 * (i & 3)));
  }
  if ((threadIdx.x & 31) == 0 && n > 0) *scale = __fmul_rn(top, 1.f / kE4M3Max);
}

// What a lane reads for 8 elements at element i of the tensor (n <= 8 of them exist; none
// or less: nothing)
template <typename P, typename G, bool Q>
struct Lane {
  using S = typename std::conditional<Q, uint8_t, float>::type;
  Raw8<P> p;
  Raw8<float> w;
  Raw8<G> g;
  Raw8<S> m, v;
  float ms, vs;
  __device__ __forceinline__ void load(const moe_adamw_tensor_t &t, size_t i, int n) {
    g.load(static_cast<const G *>(t.grad) + i, n);
    if (sizeof(P) == 2 && t.master) w.load(t.master + i, n);
    else p.load(static_cast<const P *>(t.param) + i, n);
    m.load(static_cast<const S *>(t.exp_avg) + i, n);
    v.load(static_cast<const S *>(t.exp_avg_sq) + i, n);
    if (Q) {
      ms = n > 0 ? t.exp_avg_scale[i / kQBlock] : 0.f;
      vs = n > 0 ? t.exp_avg_sq_scale[i / kQBlock] : 0.f;
    }
  }
  // The moments' sums are rounded product by product, as the plain formula's in fp32: a
  // contraction left to the compiler could differ from one build or element to the next and
  // move 8-bit codes that lie at a border. (Explicit fused operations would not, and are fewer.)
  __device__ __forceinline__ void update(const moe_adamw_tensor_t &t, size_t i, int n,
                                         const Step &s) {
    const bool copy = sizeof(P) == 2 && t.master;
    float pf[8], gf[8], mf[8], vf[8], r[8];
    g.get(gf);
    m.get(mf);
    v.get(vf);
    if (copy) w.get(pf);
    else p.get(pf);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (Q) {
        mf[j] = __fmul_rn(mf[j], ms);
        vf[j] = __fmul_rn(vf[j], vs);
        vf[j] = __fmul_rn(vf[j], vf[j]);
      }
      const float gr = __fmul_rn(gf[j], s.gs);
      mf[j] = __fadd_rn(__fmul_rn(s.b1, mf[j]), __fmul_rn(s.e1, gr));
      vf[j] = __fadd_rn(__fmul_rn(s.b2, vf[j]), __fmul_rn(__fmul_rn(s.e2, gr), gr));
      r[j] = __fsqrt_rn(vf[j]);
      // a quotient good to two units: far below what a step moves a weight
      pf[j] = fmaf(pf[j], s.keep, -s.size * __fdividef(mf[j], fmaf(r[j], s.root2, s.eps)));
    }
    if (copy) store_any(t.master + i, n, pf);
    store_any(static_cast<P *>(t.param) + i, n, pf);
    if constexpr (Q) {
      quantise<false>(static_cast<uint8_t *>(t.exp_avg) + i, t.exp_avg_scale + i / kQBlock, n, mf);
      quantise<true>(static_cast<uint8_t *>(t.exp_avg_sq) + i, t.exp_avg_sq_scale + i / kQBlock, n,
                     r);
    } else {
      store_any(static_cast<float *>(t.exp_avg) + i, n, mf);
      store_any(static_cast<float *>(t.exp_avg_sq) + i, n, vf);
    }
  }
};

// A CTA's elements: requested, then the step's scalars, then the update. With 8-bit states
// a warp stays together (its 256 elements share a scale); a warp past the end leaves.
// Eight elements a thread and five CTAs an SM hide the loads better than longer walks with
// the next elements prefetched (8-bit states, 805 M elements: 2.00 ms; the walks took 4 to
// 40 % longer).
template <typename P, typename G, bool Q, typename F>
__device__ __forceinline__ void chunk(const moe_adamw_tensor_t &t, size_t base, const F &ready) {
  const size_t at = base + (size_t)threadIdx.x * kVec;
  const long long left = (long long)t.n - (long long)at;
  const int n = left >= 8 ? 8 : (int)(left > 0 ? left : 0);
  Lane<P, G, Q> lane;
  lane.load(t, at, n);
  const Step s = ready();
  if (Q ? (long long)t.n <= (long long)(at - (threadIdx.x & 31) * kVec) : n == 0) return;
  lane.update(t, at, n, s);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 5) k_adamw(const __grid_constant__ Batch<N> b) {
  // waits for the kernels that wrote the gradients, and never lets the next kernel begin
  // early: the layer's GEMMs read weights before their own wait
  __shared__ Step sh;
  int lo = 0, hi = b.n - 1;  // last tensor whose first CTA <= this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= blockIdx.x) lo = mid; else hi = mid - 1;
  }
  pdl_wait();
  if (b.found_inf && *b.found_inf != 0.f) return;  // the step is skipped
  auto ready = [&]() {
    Step s = b.s;
    if (b.step_dev || b.lr_dev) {
      if (threadIdx.x == 0) {
        double c1 = b.c1, c2 = b.c2;
        if (b.step_dev) {
          const double step = (double)*b.step_dev;
          c1 = 1.0 - pow(b.beta1, step);
          c2 = 1.0 - pow(b.beta2, step);
        }
        set_rates(s, b.lr_dev ? (double)*b.lr_dev : (double)b.lr, (double)b.decay, c1, c2);
        sh = s;
      }
      __syncthreads();
      s = sh;
    }
    if (b.grad_scale) s.gs = *b.grad_scale;
    return s;
  };
  const moe_adamw_tensor_t &t = b.t[lo];
  const size_t base = (size_t)(blockIdx.x - b.first[lo]) * kChunk;
  const bool pf = t.param_dtype == MOE_DTYPE_F32, gf = t.grad_dtype == MOE_DTYPE_F32;
  const bool q = t.state_bits == 8;
  if (pf) {
    if (gf) q ? chunk<float, float, true>(t, base, ready) : chunk<float, float, false>(t, base, ready);
    else q ? chunk<float, __nv_bfloat16, true>(t, base, ready)
           : chunk<float, __nv_bfloat16, false>(t, base, ready);
  } else {
    if (gf) q ? chunk<__nv_bfloat16, float, true>(t, base, ready)
              : chunk<__nv_bfloat16, float, false>(t, base, ready);
    else q ? chunk<__nv_bfloat16, __nv_bfloat16, true>(t, base, ready)
           : chunk<__nv_bfloat16, __nv_bfloat16, false>(t, base, ready);
  }
}

// Tensors per launch: kernel parameters of 3, 10 and 22 KB, which the launch copies (96
// tensors: a call of 13 us with the largest, 6 us with the middle one).
constexpr int kFew = 32, kSome = 128, kMany = 288;
static_assert(sizeof(Batch<kMany>) <= 32764, "kernel parameters");

template <int N>
moe_status_t launch(const moe_adamw_tensor_t *ts, int n, const moe_adamw_t &o, cudaStream_t st) {
  Batch<N> b{};
  b.s.b1 = (float)o.beta1;
  b.s.b2 = (float)o.beta2;
  b.s.e1 = (float)(1.0 - o.beta1);
  b.s.e2 = (float)(1.0 - o.beta2);
  b.s.eps = o.eps;
  b.s.gs = 1.f;
  b.beta1 = o.beta1;
  b.beta2 = o.beta2;
  b.lr = o.lr;
  b.decay = o.weight_decay;
  b.step_dev = o.step_dev;
  b.lr_dev = o.lr_dev;
  b.grad_scale = o.grad_scale;
  b.found_inf = o.found_inf;
  if (!o.step_dev) {
    b.c1 = 1.0 - pow(o.beta1, (double)o.step);
    b.c2 = 1.0 - pow(o.beta2, (double)o.step);
    set_rates(b.s, o.lr, o.weight_decay, b.c1, b.c2);
  }
  unsigned ctas = 0;
  for (int i = 0; i < n; ++i) {
    if (ts[i].n == 0) continue;
    b.t[b.n] = ts[i];
    b.first[b.n++] = ctas;
    ctas += (unsigned)((ts[i].n + kChunk - 1) / kChunk);
  }
  b.first[b.n] = ctas;
  if (ctas == 0) return MOE_OK;
  return cuda_status(launch_pdl(k_adamw<N>, dim3(ctas), dim3(kThreads), 0, st, b));
}

moe_status_t check_tensor(const moe_adamw_tensor_t &t) {
  if (t.n < 0) return MOE_ERR_INVALID_ARG;
  if ((t.param_dtype != MOE_DTYPE_F32 && t.param_dtype != MOE_DTYPE_BF16) ||
      (t.grad_dtype != MOE_DTYPE_F32 && t.grad_dtype != MOE_DTYPE_BF16) ||
      (t.state_bits != 8 && t.state_bits != 32))
    return MOE_ERR_INVALID_ARG;
  if (t.master && t.param_dtype == MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (t.n > kMaxCtas * kChunk) return MOE_ERR_UNSUPPORTED;
  if (t.n == 0) return MOE_OK;
  const bool q = t.state_bits == 8;
  if (!q && (t.exp_avg_scale || t.exp_avg_sq_scale)) return MOE_ERR_INVALID_ARG;
  return check_ptrs({{t.param, true}, {t.grad, true}, {t.exp_avg, true}, {t.exp_avg_sq, true},
                     {t.master, false}, {t.exp_avg_scale, q}, {t.exp_avg_sq_scale, q}});
}

}  // namespace
}  // namespace moe

using namespace moe;

MOE_API moe_status_t moe_adamw_step(const moe_adamw_tensor_t *tensors, int32_t n_tensors,
                                    const moe_adamw_t *opt, moe_stream_t stream) {
  if (opt == nullptr || n_tensors < 0 || (n_tensors > 0 && tensors == nullptr))
    return MOE_ERR_INVALID_ARG;
  const moe_adamw_t &o = *opt;
  if (!(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0) ||
      !(o.eps >= 0.f) || !isfinite(o.eps) || !isfinite(o.weight_decay) ||
      (!o.lr_dev && !isfinite(o.lr)) || (!o.step_dev && o.step < 1))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(o.step_dev, 8) || !aligned(o.lr_dev, 4) || !aligned(o.grad_scale, 4) ||
      !aligned(o.found_inf, 4))
    return MOE_ERR_MISALIGNED;
  for (int i = 0; i < n_tensors; ++i) MOE_TRY(check_tensor(tensors[i]));
  for (int i = 0; i < n_tensors;) {
    // as many tensors as one launch's parameters and grid hold
    long long ctas = 0;
    int m = 0;
    while (i + m < n_tensors && m < kMany) {
      const long long c = (tensors[i + m].n + kChunk - 1) / kChunk;
      if (ctas + c > kMaxCtas) break;  // (never at m = 0: check_tensor)
      ctas += c;
      ++m;
    }
    MOE_TRY(m <= kFew    ? launch<kFew>(tensors + i, m, o, stream)
            : m <= kSome ? launch<kSome>(tensors + i, m, o, stream)
                         : launch<kMany>(tensors + i, m, o, stream));
    i += m;
  }
  return MOE_OK;
}
