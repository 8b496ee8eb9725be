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

#include "api.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                            // elements per lane and step
constexpr int kQBlock = MOE_ADAMW_BLOCK;           // elements of one 8-bit scale: a warp's step
constexpr int kSteps = 2;                          // steps per thread
constexpr int kChunk = kThreads * kVec * kSteps;   // elements per CTA
static_assert(kQBlock == 32 * kVec, "a warp's step is one scale block");
constexpr float kE4M3Max = 448.f;
constexpr float kE4M3Tiny = 0.001953125f;          // 2^-9, the smallest positive code
constexpr float kFloor = 7.8886090522101181e-31f;  // 2^-100: keeps 448 / top finite

template <int N>
struct Batch {
  moe_adamw_tensor_t t[N];
  unsigned first[N + 1];  // first CTA of each tensor
  int n;
  float beta1, beta2, lr, eps, decay;
  double c1, c2;               // 1 - b1^t, 1 - b2^t (without step_dev)
  double beta1_d, beta2_d;
  const int64_t *step_dev;
  const float *lr_dev, *grad_scale, *found_inf;
};

__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
  unpack16(*reinterpret_cast<const uint4 *>(p), f);
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(p) = pack16(f);
}
// n < 8 elements of a tensor's end
template <typename T>
__device__ __forceinline__ void load_n(const T *p, int n, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = i < n ? Elem<T>::to_f(p[i]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_n(T *p, int n, const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = Elem<T>::from_f(f[i]);
}
template <typename T>
__device__ __forceinline__ void load_any(const T *p, int n, float (&f)[8]) {
  if (n >= 8) load8(p, f);
  else load_n(p, n, f);
}
template <typename T>
__device__ __forceinline__ void store_any(T *p, int n, const float (&f)[8]) {
  if (n >= 8) store8(p, f);
  else store_n(p, n, f);
}
__device__ __forceinline__ void load_codes(const uint8_t *p, int n, float scale, float (&f)[8]) {
  uint8_t c[8];
  if (n >= 8) {
    *reinterpret_cast<uint2 *>(c) = *reinterpret_cast<const uint2 *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = i < n ? p[i] : 0;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __nv_fp8_e4m3 q;
    q.__x = c[i];
    f[i] = (float)q * scale;
  }
}
__device__ __forceinline__ void store_codes(uint8_t *p, int n, const float (&f)[8]) {
  uint8_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __nv_fp8_e4m3(f[i]).__x;  // nearest even, saturating
  if (n >= 8) {
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = c[i];
  }
}
// A block's (a warp's 256 elements) codes and scale
template <bool ROOT>
__device__ __forceinline__ void quantise(uint8_t *codes, float *scale, int n, float (&f)[8]) {
  float top = kFloor;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
  top = warp_max(top);
  const float up = kE4M3Max / top;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = f[i] * up;
    f[i] = (ROOT && f[i] > 0.f) ? fmaxf(y, kE4M3Tiny) : y;
  }
  store_codes(codes, n, f);
  if ((threadIdx.x & 31) == 0 && n > 0) *scale = top / kE4M3Max;
}

struct Step {
  float b1, b2, e1, e2, keep, size, root2, eps, gs;
  // e1 = 1 - b1, e2 = 1 - b2; keep = 1 - lr wd; size = lr / c1; root2 = sqrt(c2)
};

// n <= 8 elements at element i of the tensor; with 8-bit states the whole warp calls
// it together (lanes past the end with n <= 0)
template <typename P, typename G, bool Q>
__device__ __forceinline__ void update(const moe_adamw_tensor_t &t, size_t i, int n,
                                       const Step &s) {
  float p[8], g[8], m[8], v[8];
  float *w32 = t.master ? t.master + i : nullptr;
  P *pw = static_cast<P *>(t.param) + i;
  if (!Q && n <= 0) return;
  load_any(static_cast<const G *>(t.grad) + i, n, g);
  if (w32) load_any(w32, n, p);
  else load_any(pw, n, p);
  const size_t blk = i / kQBlock;
  if (Q) {
    load_codes(static_cast<const uint8_t *>(t.exp_avg) + i, n, n > 0 ? t.exp_avg_scale[blk] : 0.f, m);
    load_codes(static_cast<const uint8_t *>(t.exp_avg_sq) + i, n,
               n > 0 ? t.exp_avg_sq_scale[blk] : 0.f, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= v[j];
  } else {
    load_any(static_cast<const float *>(t.exp_avg) + i, n, m);
    load_any(static_cast<const float *>(t.exp_avg_sq) + i, n, v);
  }
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gr = g[j] * s.gs;
    m[j] = fmaf(s.b1, m[j], s.e1 * gr);
    v[j] = fmaf(s.b2, v[j], s.e2 * gr * gr);
    r[j] = sqrtf(v[j]);
    p[j] = fmaf(p[j], s.keep, -s.size * (m[j] / (r[j] / s.root2 + s.eps)));
  }
  if (w32) store_any(w32, n, p);
  store_any(pw, n, p);
  if (Q) {
    quantise<false>(static_cast<uint8_t *>(t.exp_avg) + i, t.exp_avg_scale + blk, n, m);
    quantise<true>(static_cast<uint8_t *>(t.exp_avg_sq) + i, t.exp_avg_sq_scale + blk, n, r);
  } else {
    store_any(static_cast<float *>(t.exp_avg) + i, n, m);
    store_any(static_cast<float *>(t.exp_avg_sq) + i, n, v);
  }
}

template <typename P, typename G, bool Q>
__device__ __forceinline__ void chunk(const moe_adamw_tensor_t &t, size_t base, const Step &s) {
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const size_t i = base + (size_t)j * kThreads * kVec + (size_t)threadIdx.x * kVec;
    const long long left = (long long)t.n - (long long)i;
    const int n = left >= 8 ? 8 : (int)(left > 0 ? left : 0);
    // a whole warp past the end has nothing to do
    if ((long long)t.n <= (long long)(i - (threadIdx.x & 31) * kVec)) return;
    update<P, G, Q>(t, i, n, s);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Batch<N> b) {
  // waits for the kernels that wrote the gradients, and never lets the next kernel begin
  // early: the layer's GEMMs read weights before their own wait
  pdl_wait();
  __shared__ Step sh;
  if (b.found_inf && *b.found_inf != 0.f) return;  // the step is skipped
  if (threadIdx.x == 0) {
    double c1 = b.c1, c2 = b.c2;
    if (b.step_dev) {
      const double step = (double)*b.step_dev;
      c1 = 1.0 - pow(b.beta1_d, step);
      c2 = 1.0 - pow(b.beta2_d, step);
    }
    const double lr = b.lr_dev ? (double)*b.lr_dev : (double)b.lr;
    sh.b1 = b.beta1;
    sh.b2 = b.beta2;
    sh.e1 = (float)(1.0 - b.beta1_d);
    sh.e2 = (float)(1.0 - b.beta2_d);
    sh.keep = (float)(1.0 - lr * (double)b.decay);
    sh.size = (float)(lr / c1);
    sh.root2 = (float)sqrt(c2);
    sh.eps = b.eps;
    sh.gs = b.grad_scale ? *b.grad_scale : 1.f;
  }
  __syncthreads();
  const Step s = sh;
  int lo = 0, hi = b.n - 1;  // last tensor whose first CTA <= this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const moe_adamw_tensor_t &t = b.t[lo];
  const size_t base = (size_t)(blockIdx.x - b.first[lo]) * kChunk;
  const bool pf = t.param_dtype == MOE_DTYPE_F32, gf = t.grad_dtype == MOE_DTYPE_F32;
  const bool q = t.state_bits == 8;
  if (pf) {
    if (gf) q ? chunk<float, float, true>(t, base, s) : chunk<float, float, false>(t, base, s);
    else q ? chunk<float, __nv_bfloat16, true>(t, base, s)
           : chunk<float, __nv_bfloat16, false>(t, base, s);
  } else {
    if (gf) q ? chunk<__nv_bfloat16, float, true>(t, base, s)
              : chunk<__nv_bfloat16, float, false>(t, base, s);
    else q ? chunk<__nv_bfloat16, __nv_bfloat16, true>(t, base, s)
           : chunk<__nv_bfloat16, __nv_bfloat16, false>(t, base, s);
  }
}

constexpr int kFew = 32, kMany = 288;  // tensors per launch (kernel parameters of 4 KB, 32 KB)
static_assert(sizeof(Batch<kFew>) <= 4096 && sizeof(Batch<kMany>) <= 32764, "kernel parameters");

template <int N>
moe_status_t launch(const moe_adamw_tensor_t *ts, int n, const moe_adamw_t &o, cudaStream_t st) {
  Batch<N> b{};
  b.beta1 = (float)o.beta1;
  b.beta2 = (float)o.beta2;
  b.beta1_d = o.beta1;
  b.beta2_d = o.beta2;
  b.lr = o.lr;
  b.eps = o.eps;
  b.decay = o.weight_decay;
  b.step_dev = o.step_dev;
  b.lr_dev = o.lr_dev;
  b.grad_scale = o.grad_scale;
  b.found_inf = o.found_inf;
  if (!o.step_dev) {
    b.c1 = 1.0 - pow(o.beta1, (double)o.step);
    b.c2 = 1.0 - pow(o.beta2, (double)o.step);
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
  if (t.n > (1ll << 42)) return MOE_ERR_UNSUPPORTED;  // the grid holds 2^31 - 1 chunks
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
      if (ctas + c > 0x7fffffffll) break;
      ctas += c;
      ++m;
    }
    MOE_TRY(m <= kFew ? launch<kFew>(tensors + i, m, o, stream)
                      : launch<kMany>(tensors + i, m, o, stream));
    i += m;
  }
  return MOE_OK;
}
