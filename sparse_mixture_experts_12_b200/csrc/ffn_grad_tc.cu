// Gradient of the grouped expert FFN on the 5th-generation tensor cores (bf16 layers):
// the formulas of ffn_grad.cu as two persistent grids of CTA pairs.
//
//   k_act_grad    a = x W1^T (and u = x W3^T) and q = dy W2, reduction length d, into
//                 tensor memory together; the epilogue turns them into h, da, du
//   k_pair_gemm   dx = da W1 (+ du W3), reduction length F (2 F), and
//                 dW1 = da^T x, dW3 = du^T x, dW2 = dy^T h, reduction over an expert's rows
//
// Every product is a 256-row tcgen05.mma.cta_group::2 over K slices of 64; operands whose
// contiguous index is not the reduction's (W2 in q, W1 / W3 in dx, both in the weights'
// gradients) are loaded as they lie and marked MN-major, so nothing is transposed in
// memory. x, dy and the scratch rows lie padded: each expert begins at a multiple of 64
// rows and the rows up to the next are zero. A slice of an expert's rows is then a whole
// K slice, with no masking in the weights' gradients (zero rows add exact zeros).
//
// A CTA pair's roles, barriers and bounded waits are those of the forward's GEMM
// (ffn_tc.cu): warp 0 of each CTA loads its operand halves, warp 1 of the leader issues
// the MMAs (k_act_grad: warps 0 and 3, 1 and 2), warps 4.. drain tensor memory; a wait that runs out records
// MOE_DEVERR_WAIT_TIMEOUT and ends both CTAs.
#include <algorithm>
#include <mutex>

#include "grad.cuh"
#include "grad_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr int kPairM = 2 * kRowTile;
constexpr int kOperand = kRowTile * kBlockK * 2;  // 16 KB: a CTA's half of a 256-wide operand
constexpr int kMnBlock = kBlockK * kBlockK * 2;   // 8 KB: 64 K rows x 64 contiguous elements
constexpr int kTmemCols = 512;
constexpr int kMaxStages = 8;
constexpr int kStageOutBytes = kStoreBox * kStoreBox * 2;  // 2 KB: a 32 x 32 output chunk
constexpr uint64_t kDrainNs = 50000000ull;

struct Ctl {
  uint64_t full[kMaxStages];   // leader: both CTAs' copies of the stage landed
  uint64_t empty[kMaxStages];  // each CTA: the pair's MMAs are done with the stage
  uint64_t tfull[2];           // each CTA: the tile's accumulators are complete
  uint64_t tempty[2];          // leader: both epilogues have drained them
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int pre[kMaxExperts + 1];  // prefix of the experts' 256-row tiles, or their first rows
};

// what both kernels do before their roles split up
struct Setup {
  uint8_t *smem;
  Ctl *ctl;
  uint32_t tmem, peer_abort;
  uint32_t full0;  // the leader's full[0] (pairs)
  int rank, c0, cstep;
};

// `bytes` of operand stages and output staging come before the control block; `issuers`
// threads complete a tile's accumulators, `drainers` warps of both CTAs drain them (one
// arrival each).
// `unit`: rows of a tile whose prefix over the experts goes to pre[] (0: their first rows).
template <bool PAIR>
__device__ __forceinline__ Setup set_up(uint8_t *raw, size_t bytes, int issuers, int drainers,
                                        const int32_t *poff, int G, int unit) {
  Setup s;
  s.smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                       ~static_cast<uintptr_t>(1023));
  s.ctl = reinterpret_cast<Ctl *>(s.smem + bytes);
  Ctl *ctl = s.ctl;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  s.rank = PAIR ? (int)cluster_ctarank() : 0;
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], issuers);
      mbar_init(&ctl->tempty[i], drainers);
      mbar_init(&ctl->drain[i], 1);
    }
    ctl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&ctl->tmem_base, kTmemCols);
      tmem_relinquish();
    }
  }
  pdl_wait();
  if (unit == 0) {
    for (int i = tid; i <= G; i += blockDim.x) ctl->pre[i] = poff[i];
  } else if (warp == 1) {
    const int per = ceil_div(G, 32);
    const int j0 = min(G, lane * per), j1 = min(G, j0 + per);
    int sum = 0;
    for (int j = j0; j < j1; ++j) sum += ceil_div(poff[j + 1] - poff[j], unit);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - sum;
    for (int j = j0; j < j1; ++j) {
      ctl->pre[j] = run;
      run += ceil_div(poff[j + 1] - poff[j], unit);
    }
    if (lane == 31) ctl->pre[G] = incl;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers and tensor memory exist
  pdl_trigger();
  tc_fence_after();
  s.tmem = ctl->tmem_base;
  if constexpr (PAIR) {
    s.peer_abort = mapa_rank(smem_u32(&ctl->abort_flag), (uint32_t)(s.rank ^ 1));
    s.full0 = mapa_rank(smem_u32(&ctl->full[0]), 0);
    s.c0 = (int)cluster_index();
    s.cstep = (int)cluster_count();
  } else {
    s.peer_abort = s.full0 = 0;
    s.c0 = (int)blockIdx.x;
    s.cstep = (int)gridDim.x;
  }
  return s;
}

__device__ __forceinline__ bool wait_on(const Setup &s, uint64_t *bar, uint32_t parity,
                                        int32_t *err, int site, bool honour_abort = true,
                                        uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_mbar(bar, parity, &s.ctl->abort_flag, s.peer_abort, err, site, honour_abort,
                   limit_ns);
}

// arrive on `bar` (in both CTAs of a pair) once the MMAs issued so far are done
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (PAIR) umma_commit_pair_both(bar);
  else umma_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t acc, uint64_t a, uint64_t b, uint32_t idesc,
                                    bool accumulate) {
  if constexpr (PAIR) umma_bf16_pair(acc, a, b, idesc, accumulate);
  else umma_bf16(acc, a, b, idesc, accumulate);
}
// a draining warp's arrival on the leader's tempty[i] (tempty0: the first's address)
template <bool PAIR>
__device__ __forceinline__ void release_tmem(const Setup &s, uint32_t tempty0, int i) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) != 0) return;
  if constexpr (PAIR) mbar_arrive_remote(tempty0 + (uint32_t)(i * sizeof(uint64_t)));
  else mbar_arrive(&s.ctl->tempty[i]);
}

// A ring of N operand stages of BYTES each, from stage FIRST of the barriers on; producer
// and MMA issuer hold one each and walk through it in step.
template <bool PAIR, int N, int FIRST, int BYTES>
struct Ring {
  uint8_t *base;
  int stage = 0;
  uint32_t phase = 0, issued = 0, last_phase = 0;
  __device__ __forceinline__ explicit Ring(uint8_t *b) : base(b) {}
  // producer: the next stage, free to be filled with `bytes` by each CTA, or nullptr
  __device__ __forceinline__ uint8_t *acquire(const Setup &s, int bytes, int32_t *err, int site) {
    if (!wait_on(s, &s.ctl->empty[FIRST + stage], phase ^ 1u, err, site)) return nullptr;
    if (s.rank == 0) mbar_expect_tx(&s.ctl->full[FIRST + stage], PAIR ? 2 * bytes : bytes);
    issued |= 1u << stage;
    last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
    return base + (size_t)stage * BYTES;
  }
  // ... and a copy into it
  __device__ __forceinline__ void load(const Setup &s, const CUtensorMap *map, uint8_t *dst, int c0,
                                       int c1) const {
    if constexpr (PAIR) tma_load_2d_pair(map, bar(s), dst, c0, c1);
    else tma_load_2d(map, &s.ctl->full[FIRST + stage], dst, c0, c1);
  }
  __device__ __forceinline__ uint32_t bar(const Setup &s) const {  // the leader's (pairs)
    return s.full0 + (uint32_t)((FIRST + stage) * sizeof(uint64_t));
  }
  // issuer: the next stage, filled
  __device__ __forceinline__ bool filled(const Setup &s, int32_t *err, int site) const {
    const bool ok = wait_on(s, &s.ctl->full[FIRST + stage], phase, err, site);
    tc_fence_after();
    return ok;
  }
  __device__ __forceinline__ uint32_t addr() const { return smem_u32(base) + stage * BYTES; }
  // ... handed back once the MMAs issued so far are done
  __device__ __forceinline__ void release(const Setup &s) const {
    commit<PAIR>(&s.ctl->empty[FIRST + stage]);
  }
  __device__ __forceinline__ void next() {
    if (++stage == N) { stage = 0; phase ^= 1u; }
  }
  // producer, at its end: the MMAs have released every stage this CTA filled
  __device__ __forceinline__ void drain(const Setup &s, bool ok) const {
    for (int i = 0; i < N; ++i)
      if (issued & (1u << i))
        wait_on(s, &s.ctl->empty[FIRST + i], (last_phase >> i) & 1u, nullptr, 0, false,
                ok ? kWaitLimitNs : kDrainNs);
  }
};

// issuer, at its end: the MMAs in flight retire before tensor memory is released
template <bool PAIR>
__device__ __forceinline__ void retire(const Setup &s, uint64_t *bar) {
  if constexpr (PAIR) umma_commit_pair_own(bar);
  else umma_commit(bar);
  wait_on(s, bar, 0, nullptr, 0, false, kDrainNs);
}

template <bool PAIR>
__device__ __forceinline__ void tear_down(const Setup &s) {
  if (*(volatile int *)&s.ctl->abort_flag) settle_ns(100000);  // copies in flight land
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // the peer's remote arrivals are done before exit
  if ((threadIdx.x >> 5) == 2) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(s.tmem, kTmemCols);
    else tmem_dealloc(s.tmem, kTmemCols);
  }
}

// First row of this CTA's half of the tile that begins at row m0 of expert g, or `rows` (past the operand's
// bounds: zeros, no traffic) when the expert ends before it. The MMAs of such a half take
// their time all the same, but on zeros, which cost less of the power that limits long
// grids.
__device__ __forceinline__ int first_row(const int32_t *poff, int g, int m0, int rank, int rows) {
  const int r = poff[g] + m0 + rank * kRowTile;
  return r < poff[g + 1] ? r : rows;
}

// One 32-row x 32-column chunk (a lane's row of 64 bytes) through the warp's 2 KB of
// shared memory: 16-byte pieces swizzled, one TMA store. The buffer is written again once
// the store before has read it.
__device__ __forceinline__ void put32(uint8_t *buf, const CUtensorMap *map, const uint32_t *p,
                                      int col0, int row0) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
  uint4 *row = reinterpret_cast<uint4 *>(buf + lane * 64);
  const int sw = (lane >> 1) & 3;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    row[q ^ sw] = make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, buf, col0, row0);
    bulk_commit();
  }
}

// ================================================================= activations
struct ActArgs {
  const int32_t *poff, *offsets;  // padded first rows; the experts' row counts
  int G, F, d, act, n_tiles;
  const float *b1, *row_w;
  float *dot_part;  // [F / 32, rows] or nullptr
  float *col_part;  // [rows / 32, F] or nullptr
  int rows, x_rows;
  int32_t *err;
};
struct ActMaps {
  CUtensorMap x, dy, w1, w3, w2, h, dg, du;
};

// Column sums of 16 values per lane over the warp's 32 lanes: lane l ends with column
// l & 15 (a butterfly that halves the columns a lane holds at each step).
__device__ __forceinline__ float column_sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int w = 8; w > 0; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = up ? v[i] : v[i + w];
      const float keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// gelu and d gelu / dv, with the forward's erf (formula 7.1.26 of Abramowitz & Stegun): its
// exp(-(v / sqrt 2)^2) is the density's exponential as well.
__device__ __forceinline__ void gelu_and_slope(float v, float &h, float &s) {
  const float e = __expf(-0.5f * v * v);
  const float t = rcp_approx(fmaf(0.3275911f * 0.70710678118654752f, fabsf(v), 1.f));
  const float p =
      fmaf(fmaf(fmaf(fmaf(0.5f * 1.061405429f, t, -0.5f * 1.453152027f), t, 0.5f * 1.421413741f),
                t, -0.5f * 0.284496736f), t, 0.5f * 0.254829592f) * t;
  const float c = 0.5f + copysignf(fmaf(-p, e, 0.5f), v);  // (1 + erf(v / sqrt 2)) / 2
  h = v * c;
  s = fmaf(v * 0.39894228040143268f, e, c);
}

// One tile: 256 rows x 128 columns of F. Tensor memory: a | u at columns 0-255 (SwiGLU) or
// a at 0 / 128 (alternating, MLP); q at 256 / 384 (alternating). q and a (| u) have a ring,
// a loading and an issuing thread of their own: one thread for both spent more time on
// issuing (about 400 clocks a slice and thread) than the MMAs took, and q of the next tile
// runs while the epilogue drains the one a | u region of SwiGLU.
// The MMAs keep the tensor pipe busy 78 % of the time (1024 rows per expert of 4096 x 14336,
// SwiGLU); with 100 rows the weights' bytes bound it, read at 83 % of a copy's rate (128
// experts of 1024 x 4096: 451 us).
// Experts of few rows (MLP, at most 128 on average) take single-CTA tiles of 128 rows
// (PAIR false): a pair's MMAs take their time for 256 rows, and shared memory's bandwidth
// bounds them: some 940 clocks a slice for a pair against 1060 for one CTA.
constexpr int kTileN = 128;
template <bool GLU, bool PAIR>
struct ActCfg {
  static_assert(PAIR || !GLU, "SwiGLU: pairs only");
  static constexpr int kTileM = PAIR ? kPairM : kRowTile;
  static constexpr int kEpiWarps = GLU ? 8 : 16;  // MLP tiles are shorter, their epilogue longer
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kWeights = PAIR ? kMnBlock : kOperand;  // a CTA's share of 128 columns
  static constexpr int kBytesQ = kOperand + kWeights;
  static constexpr int kBytesA = GLU ? 2 * kOperand : kOperand + kWeights;
  static constexpr int kStagesQ = GLU || !PAIR ? 3 : 4, kStagesA = PAIR ? 4 : 3;
  // K slices of one accumulation. The tensor cores truncate what they add, a bias of some
  // 2^-26 of the sum for each 16 products (-4.3e-6 at d = 4096). It does not matter beside
  // the rounding of h and da, but db1 keeps it: with biases (MLP) the epilogue adds up
  // parts of 512 products in fp32.
  static constexpr int kPart = GLU ? 1 << 30 : 8;
  static constexpr size_t kRings = (size_t)kStagesQ * kBytesQ + (size_t)kStagesA * kBytesA;
  static constexpr size_t kBytes = kRings + (size_t)kEpiWarps * kStageOutBytes;
  static constexpr size_t kSmem = kBytes + sizeof(Ctl) + 1024;
};

template <bool GLU, bool PAIR>
__global__ void __launch_bounds__(ActCfg<GLU, PAIR>::kThreads, 1)
k_act_grad(const __grid_constant__ ActMaps maps, ActArgs a) {
  using C = ActCfg<GLU, PAIR>;
  using RingQ = Ring<PAIR, C::kStagesQ, 0, C::kBytesQ>;
  using RingA = Ring<PAIR, C::kStagesA, C::kStagesQ, C::kBytesA>;
  extern __shared__ uint8_t smem_raw[];
  const Setup s = set_up<PAIR>(smem_raw, C::kBytes, 2, (PAIR ? 2 : 1) * C::kEpiWarps, a.poff, a.G,
                               C::kTileM);
  Ctl *ctl = s.ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = ctl->pre[a.G] * a.n_tiles;
  const int nkb = ceil_div(a.d, kBlockK);
  uint8_t *const ring_q = s.smem, *const ring_a = s.smem + C::kStagesQ * C::kBytesQ;

  if (warp == 0 && lane == 0) {
    // ----------------------------------------------- TMA producer of dy and W2
    prefetch_map(&maps.dy);
    prefetch_map(&maps.w2);
    RingQ ring(ring_q);
    bool ok = true;
    for (int t = s.c0; ok && t < total; t += s.cstep) {
      int g, n, m;
      decode_tile(t, ctl->pre, a.G, a.n_tiles, g, n, m);
      const int arow = first_row(a.poff, g, m * C::kTileM, s.rank, a.x_rows);
      const int col = n * kTileN + s.rank * kBlockK, brow = g * a.d;
      for (int i = 0; i < nkb; ++i) {
        uint8_t *st = ring.acquire(s, C::kBytesQ, a.err, 21);
        if (!(ok = st != nullptr)) break;
        ring.load(s, &maps.dy, st, i * kBlockK, arow);
        ring.load(s, &maps.w2, st + kOperand, col, brow + i * kBlockK);
        if (!PAIR)  // both blocks of 64 columns
          ring.load(s, &maps.w2, st + kOperand + kMnBlock, col + kBlockK, brow + i * kBlockK);
        ring.next();
      }
    }
    ring.drain(s, ok);
  } else if (warp == 3 && lane == 0) {
    // ----------------------------------------- TMA producer of x and W1 (| W3)
    const CUtensorMap *w = GLU && s.rank ? &maps.w3 : &maps.w1;
    prefetch_map(&maps.x);
    prefetch_map(w);
    RingA ring(ring_a);
    bool ok = true;
    for (int t = s.c0; ok && t < total; t += s.cstep) {
      int g, n, m;
      decode_tile(t, ctl->pre, a.G, a.n_tiles, g, n, m);
      const int arow = first_row(a.poff, g, m * C::kTileM, s.rank, a.x_rows);
      const int brow = g * a.F + n * kTileN + (GLU ? 0 : s.rank * kBlockK);
      for (int i = 0; i < nkb; ++i) {
        uint8_t *st = ring.acquire(s, C::kBytesA, a.err, 21);
        if (!(ok = st != nullptr)) break;
        ring.load(s, &maps.x, st, i * kBlockK, arow);
        ring.load(s, w, st + kOperand, i * kBlockK, brow);
        ring.next();
      }
    }
    ring.drain(s, ok);
  } else if (warp == 1 && lane == 0 && s.rank == 0) {
    // ------------------------------------------------------------ MMAs of q
    constexpr uint32_t idesc = make_idesc(C::kTileM, kTileN) | kIdescMnB;
    RingQ ring(ring_q);
    bool ok = true, any = false;
    int it = 0;
    for (int t = s.c0; ok && t < total; t += s.cstep) {
      for (int i0 = 0; ok && i0 < nkb; i0 += C::kPart, ++it) {
        const int buf = it & 1, i1 = min(nkb, i0 + C::kPart);
        const uint32_t acc = s.tmem + 256u + (uint32_t)(buf * kTileN);
        // part it - 2, which used the same buffer, has been drained
        if (!(ok = wait_on(s, &ctl->tempty[buf], ((it >> 1) & 1) ^ 1u, a.err, 22))) break;
        tc_fence_after();
        for (int i = i0; i < i1; ++i) {
          if (!(ok = ring.filled(s, a.err, 23))) break;
          const uint64_t xa = sw128_desc(ring.addr());
          const uint64_t xb = sw128_desc_mn(ring.addr() + kOperand, kMnBlock);
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            mma<PAIR>(acc, xa + 2 * kk, xb + 128 * kk, idesc, ((i - i0) | kk) != 0);
          any = true;
          ring.release(s);
          ring.next();
        }
        if (ok) commit<PAIR>(&ctl->tfull[buf]);
      }
    }
    if (!ok && any) retire<PAIR>(s, &ctl->drain[0]);
  } else if (warp == 2 && lane == 0 && s.rank == 0) {
    // ------------------------------------------------------- MMAs of a (| u)
    constexpr uint32_t idesc = make_idesc(C::kTileM, GLU ? 2 * kTileN : kTileN);
    RingA ring(ring_a);
    bool ok = true, any = false;
    int it = 0;
    for (int t = s.c0; ok && t < total; t += s.cstep) {
      for (int i0 = 0; ok && i0 < nkb; i0 += C::kPart, ++it) {
        const int buf = it & 1, i1 = min(nkb, i0 + C::kPart);
        const uint32_t acc = s.tmem + (GLU ? 0u : (uint32_t)(buf * kTileN));
        // SwiGLU has one a | u region: part it - 1 (the tile before) has been drained
        const int old = GLU ? it - 1 : it - 2;
        if (old >= 0 && !(ok = wait_on(s, &ctl->tempty[old & 1], (old >> 1) & 1, a.err, 22)))
          break;
        tc_fence_after();
        for (int i = i0; i < i1; ++i) {
          if (!(ok = ring.filled(s, a.err, 23))) break;
          const uint64_t xa = sw128_desc(ring.addr()), xb = sw128_desc(ring.addr() + kOperand);
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            mma<PAIR>(acc, xa + 2 * kk, xb + 2 * kk, idesc, ((i - i0) | kk) != 0);
          any = true;
          ring.release(s);
          ring.next();
        }
        if (ok) commit<PAIR>(&ctl->tfull[buf]);
      }
    }
    if (!ok && any) retire<PAIR>(s, &ctl->drain[1]);
  } else if (warp >= 4) {
    // ----------------------------------------------------------------- epilogue
    const int ew = warp & 3, part = (warp - 4) >> 2;  // lanes 32 ew.., column chunks part..
    constexpr int kParts = C::kEpiWarps / 4;
    const uint32_t tempty0 = PAIR ? mapa_rank(smem_u32(&ctl->tempty[0]), 0) : 0u;
    uint8_t *stage = s.smem + C::kRings + (warp - 4) * kStageOutBytes;
    int it = 0;
    bool ok = true;
    for (int t = s.c0; ok && t < total; t += s.cstep) {
      int g, n, m;
      decode_tile(t, ctl->pre, a.G, a.n_tiles, g, n, m);
      const int lrow = m * C::kTileM + s.rank * kRowTile + ew * 32;  // the warp's first row
      const int prow = a.poff[g] + lrow;
      // padded groups of 32 rows belong to the expert as a whole or not at all; F is a
      // multiple of 64
      const bool rows_mine = prow < a.poff[g + 1];
      const bool valid = lrow + lane < a.offsets[g + 1] - a.offsets[g];
      const float w = (a.row_w && rows_mine) ? a.row_w[prow + lane] : 1.f;
      auto wait_full = [&]() {
        ok = wait_on(s, &ctl->tfull[it & 1], (it >> 1) & 1, a.err, 24);
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
        if (ok) tc_fence_after();
        return ok;
      };
      auto drained = [&]() { release_tmem<PAIR>(s, tempty0, it & 1); };
      const uint32_t lanes = s.tmem + ((uint32_t)(ew * 32) << 16);
      float as[GLU ? 1 : 32], qs[GLU ? 1 : 32];  // MLP: the warp's one chunk, all parts
      if constexpr (GLU) {
        if (!wait_full()) break;
      } else {
        const int col = n * kTileN + part * 32;
        const bool bias = a.b1 && col < a.F;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {  // a begins with the bias, the same for every lane
          const float4 b = bias ? __ldg(reinterpret_cast<const float4 *>(a.b1 + (size_t)g * a.F +
                                                                         col + j))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
          as[j] = b.x; as[j + 1] = b.y; as[j + 2] = b.z; as[j + 3] = b.w;
          qs[j] = qs[j + 1] = qs[j + 2] = qs[j + 3] = 0.f;
        }
        for (int i0 = 0; i0 < nkb; i0 += C::kPart) {
          if (!wait_full()) break;
          const uint32_t at = lanes + (uint32_t)((it & 1) * kTileN + part * 32);
          if (rows_mine) {
#pragma unroll
            for (int j2 = 0; j2 < 2; ++j2) {
              uint32_t av[16], qv[16];
              tmem_ld16(at + j2 * 16, av);
              tmem_ld16(at + 256u + j2 * 16, qv);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                as[j2 * 16 + j] += __uint_as_float(av[j]);
                qs[j2 * 16 + j] += __uint_as_float(qv[j]);
              }
            }
          }
          drained();
          ++it;
        }
        if (!ok) break;
      }
      // (MLP: one chunk, said so that its sums need not outlive it)
#pragma unroll 1
      for (int c = part; c < (GLU ? kTileN / 32 : part + 1); c += kParts) {
        const int col0 = n * kTileN + c * 32;
        const bool mine = rows_mine && col0 < a.F;
        const uint32_t ta = lanes + (uint32_t)(c * 32);               // SwiGLU
        const uint32_t tq = ta + 256u + (uint32_t)((it & 1) * kTileN);
        float dot = 0.f;
        uint32_t hp[16], gp[16], up[GLU ? 16 : 1];  // packed pairs of columns
        if (mine) {
#pragma unroll
          for (int j2 = 0; j2 < 2; ++j2) {
            uint32_t av[GLU ? 16 : 1], uv[GLU ? 16 : 1], qv[GLU ? 16 : 1];
            if constexpr (GLU) {
              tmem_ld16(ta + j2 * 16, av);
              tmem_ld16(ta + kTileN + j2 * 16, uv);
              tmem_ld16(tq + j2 * 16, qv);
              tmem_ld_wait();
            }
            float da[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float h[2], du[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float q, v, x;
                if constexpr (GLU) {
                  q = __uint_as_float(qv[j + i]);
                  v = __uint_as_float(av[j + i]);
                  const float u = __uint_as_float(uv[j + i]);
                  const float sg = __fdividef(1.f, 1.f + __expf(-v));
                  const float si = v * sg;
                  h[i] = si * u;
                  du[i] = q * si;
                  x = q * u * fmaf(si, 1.f - sg, sg);
                } else {
                  q = qs[j2 * 16 + j + i];
                  v = as[j2 * 16 + j + i];
                  float sl;
                  if (a.act == MOE_ACT_RELU) {
                    h[i] = fmaxf(v, 0.f);
                    sl = v > 0.f ? 1.f : 0.f;
                  } else {
                    gelu_and_slope(v, h[i], sl);
                  }
                  x = q * sl;
                }
                dot = fmaf(q, h[i], dot);
                // rows past the expert's: zeros, whatever the weights hold
                h[i] = valid ? w * h[i] : 0.f;
                da[j + i] = valid ? w * x : 0.f;
                if constexpr (GLU) du[i] = valid ? w * du[i] : 0.f;
              }
              hp[j2 * 8 + j / 2] = pack_bf16x2(h[0], h[1]);
              gp[j2 * 8 + j / 2] = pack_bf16x2(da[j], da[j + 1]);
              if constexpr (GLU) up[j2 * 8 + j / 2] = pack_bf16x2(du[0], du[1]);
            }
            if (!GLU && a.col_part) {
              const float v = column_sum16(da, lane);
              if (lane < 16)
                a.col_part[(size_t)(prow >> 5) * a.F + col0 + j2 * 16 + lane] = v;
            }
          }
        }
        // SwiGLU: the warp's last chunk is in registers
        if (GLU && c + kParts >= kTileN / 32) drained();
        if (mine) {
          put32(stage, &maps.h, hp, col0, prow);
          put32(stage, &maps.dg, gp, col0, prow);
          if constexpr (GLU) put32(stage, &maps.du, up, col0, prow);
          if (a.dot_part && valid) a.dot_part[(size_t)(col0 / 32) * a.rows + prow + lane] = dot;
        }
      }
      if (GLU) ++it;
    }
    if (lane == 0) bulk_wait_all();  // this warp's output stores are done
    __syncwarp();
  }
  tear_down<PAIR>(s);
}

// ============================================================ dx and the weights
// Two kinds of products in one grid, so that the last tiles of one overlap the first of the
// other and a small layer pays for one launch: "rows" products C = sum of nseg A B over the
// groups' rows (dx), and "sums" C = A^T B over a group's rows (the weights' gradients).
// 256 x 256 tiles, two accumulators, so that a tile's epilogue runs under the next one's
// MMAs: the tensor pipe is busy 77 % of the time with 1024 rows per expert of 4096 x 14336;
// with 100 rows of 1024 x 4096 the gradients' writes bound it (5.1 TB/s of reads and
// writes).
struct GemmArgs {
  // rows: groups' first (padded) rows, row counts, prefix of their 256-row tiles, first rows
  // in the output; N columns, reduction length K
  const int32_t *poff, *offsets, *pre, *out_off;
  int G, N, K, nseg, a_rows;
  int splits, piece;      // the nseg K / 64 slices in `splits` parts of `piece`, each with an
  int part_rows;          // output of its own, part_rows rows apart
  void *out;
  int out_f32;
  int clipped;            // no other rows lie in a group's last 32 (padding, or the output
                          // ends and its map clips the stores)
  // sums: groups' first rows (multiples of 64); njobs products of M x N each, fp32 or bf16
  const int32_t *first;
  int groups, njobs;
  int M[3], Ns[3];
  float *sum_out;         // fp32
  int32_t *err;
};
struct GemmMaps {
  CUtensorMap a[3], b[3], o;      // rows
  CUtensorMap sa[3], sb[3], so[3];  // sums
};
constexpr int kGemmStages = 5, kGemmStageBytes = 2 * kOperand;
constexpr int kGemmEpiWarps = 16, kGemmThreads = 128 + 32 * kGemmEpiWarps;
constexpr int kStageOut = 4096;  // output staging of an epilogue warp
constexpr size_t kGemmRing = (size_t)kGemmStages * kGemmStageBytes;
constexpr size_t kGemmBytes = kGemmRing + (size_t)kGemmEpiWarps * kStageOut;
constexpr size_t kGemmSmem = kGemmBytes + sizeof(Ctl) + 1024;
using GemmRing = Ring<true, kGemmStages, 0, kGemmStageBytes>;

__global__ void __launch_bounds__(kGemmThreads, 1)
k_pair_gemm(const __grid_constant__ GemmMaps maps, GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // the groups' first rows of the sums stay in shared memory: their tiles can be short
  const Setup s = set_up<true>(smem_raw, kGemmBytes, 1, 2 * kGemmEpiWarps, a.first, a.groups, 0);
  Ctl *ctl = s.ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // sums: a group's tiles are those of job 0, then 1, then 2 (end: their prefix)
  int mt[3] = {1, 1, 1}, end[3] = {0, 0, 0};
  float inv[3] = {1.f, 1.f, 1.f};
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    if (j > 0) end[j] = end[j - 1];
    if (j < a.njobs) {
      mt[j] = ceil_div(a.M[j], kPairM);
      inv[j] = 1.f / (float)mt[j];
      end[j] += mt[j] * ceil_div(a.Ns[j], 256);
    }
  }
  const int per = end[2], n_tiles = ceil_div(a.N, 256);
  const int one_split = n_tiles ? a.pre[a.G] * n_tiles : 0, row_tiles = one_split * a.splits;
  const int total = row_tiles + a.groups * per;
  // a tile: group, job (sums), first row and column, K slices; and the walk over every
  // cstep-th of them
  struct Tile {
    int t, g, job, m0, n0, nkb;
    int row0;   // sums: the reduction's first row; rows: this CTA's first row of A
    int split;  // rows
    bool sums;
  };
  const int nk1 = ceil_div(a.K, kBlockK);
  auto place = [&](Tile &r) {
    if (r.t >= total) return;
    if (r.t >= row_tiles) {
      if (!r.sums) {
        r.sums = true;
        r.g = 0;
      }
      int in = r.t - row_tiles - r.g * per;
      while (in >= per) {
        in -= per;
        ++r.g;
      }
      r.job = (in >= end[0]) + (in >= end[1]);
      const int mts = r.job == 0 ? mt[0] : (r.job == 1 ? mt[1] : mt[2]);
      const float by = r.job == 0 ? inv[0] : (r.job == 1 ? inv[1] : inv[2]);
      in -= r.job == 0 ? 0 : (r.job == 1 ? end[0] : end[1]);
      // n = in / mts (single-thread roles pay for a division in full): exact, since in is
      // below 2^20 and half a tile is more than the product's error
      const int n = __float2int_rd(((float)in + 0.5f) * by);
      r.m0 = (in - n * mts) * kPairM;
      r.n0 = n * 256;
      r.row0 = ctl->pre[r.g];
      r.nkb = (ctl->pre[r.g + 1] - r.row0) / kBlockK;
    } else {
      int n, m, t = r.t;
      r.split = 0;
      while (t >= one_split) {
        t -= one_split;
        ++r.split;
      }
      decode_tile(t, a.pre, a.G, n_tiles, r.g, n, m);
      r.m0 = m * kPairM;
      r.n0 = n * 256;
      r.nkb = min(a.piece, a.nseg * nk1 - r.split * a.piece);
      r.row0 = first_row(a.poff, r.g, r.m0, s.rank, a.a_rows);
    }
  };
  auto first_tile = [&]() {
    Tile r{s.c0, 0, 0, 0, 0, 0, 0, 0, false};
    place(r);
    return r;
  };
  auto next_tile = [&](Tile &r) {
    r.t += s.cstep;
    place(r);
  };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    for (int j = 0; n_tiles && j < a.nseg; ++j) {
      prefetch_map(&maps.a[j]);
      prefetch_map(&maps.b[j]);
    }
    for (int j = 0; j < a.njobs; ++j) {
      prefetch_map(&maps.sa[j]);
      prefetch_map(&maps.sb[j]);
    }
    GemmRing ring(s.smem);
    bool ok = true;
    for (Tile q = first_tile(); ok && q.t < total; next_tile(q)) {
      const int row0 = q.row0, bblk = q.n0 / kBlockK + 2 * s.rank;
      // pair of operands, slice of it
      int seg = 0, k = q.sums ? 0 : q.split * a.piece;
      while (!q.sums && k >= nk1) {
        k -= nk1;
        ++seg;
      }
      for (int kb = 0; kb < q.nkb; ++kb) {
        uint8_t *st = ring.acquire(s, kGemmStageBytes, a.err, 31);
        if (!(ok = st != nullptr)) break;
        const uint32_t bar = ring.bar(s);
        if (q.sums) {
          const int r = row0 + kb * kBlockK;
          tma_load_3d_pair(&maps.sa[q.job], bar, st, 0, r, q.m0 / kBlockK + 2 * s.rank);
          tma_load_3d_pair(&maps.sb[q.job], bar, st + kOperand, 0, r, bblk);
        } else {
          const int k0 = k * kBlockK;
          tma_load_2d_pair(&maps.a[seg], bar, st, k0, row0);
          tma_load_3d_pair(&maps.b[seg], bar, st + kOperand, 0, q.g * a.K + k0, bblk);
          if (++k == nk1) {
            k = 0;
            ++seg;
          }
        }
        ring.next();
      }
    }
    ring.drain(s, ok);
  } else if (warp == 1 && lane == 0 && s.rank == 0) {
    // --------------------------------------------------------------- MMA issuer
    GemmRing ring(s.smem);
    bool ok = true, any = false;
    int it = 0;
    for (Tile q = first_tile(); ok && q.t < total; next_tile(q), ++it) {
      const int buf = it & 1;
      if (!(ok = wait_on(s, &ctl->tempty[buf], ((it >> 1) & 1) ^ 1u, a.err, 32))) break;
      tc_fence_after();
      const uint32_t acc = s.tmem + (uint32_t)(buf * 256);
      const uint32_t idesc = make_idesc(kPairM, 256) | kIdescMnB | (q.sums ? kIdescMnA : 0u);
      const uint64_t step_a = q.sums ? 128 : 2;  // a K = 16 step in the A descriptor
      for (int kb = 0; kb < q.nkb; ++kb) {
        if (!(ok = ring.filled(s, a.err, 33))) break;
        const uint64_t xa =
            q.sums ? sw128_desc_mn(ring.addr(), kMnBlock) : sw128_desc(ring.addr());
        const uint64_t xb = sw128_desc_mn(ring.addr() + kOperand, kMnBlock);
#pragma unroll
        for (int kk = 0; kk < kBlockK / 16; ++kk)
          umma_bf16_pair(acc, xa + step_a * kk, xb + 128 * kk, idesc, (kb | kk) != 0);
        any = true;
        ring.release(s);
        ring.next();
      }
      if (ok) umma_commit_pair_both(&ctl->tfull[buf]);
    }
    if (!ok && any) retire<true>(s, &ctl->drain[0]);
  } else if (warp >= 4) {
    // ----------------------------------------------------------------- epilogue
    const int ew = warp & 3, part = (warp - 4) >> 2;  // lanes 32 ew.., columns 64 part..
    const uint32_t tempty0 = mapa_rank(smem_u32(&ctl->tempty[0]), 0);
    uint8_t *stage = s.smem + kGemmRing + (warp - 4) * kStageOut;
    int it = 0;
    for (Tile q = first_tile(); q.t < total; next_tile(q), ++it) {
      const int buf = it & 1;
      const int lrow = q.m0 + s.rank * kRowTile + ew * 32, col0 = q.n0 + part * 64;
      int rows, N;      // the output's valid rows from q's first, its width
      size_t orow;      // output row of lane 0
      if (q.sums) {
        rows = q.job == 0 ? a.M[0] : (q.job == 1 ? a.M[1] : a.M[2]);
        N = q.job == 0 ? a.Ns[0] : (q.job == 1 ? a.Ns[1] : a.Ns[2]);
        orow = (size_t)q.g * rows + lrow;
      } else {
        rows = a.offsets[q.g + 1] - a.offsets[q.g];
        N = a.N;
        orow = (size_t)q.split * a.part_rows + a.out_off[q.g] + lrow;
      }
      const bool mine = lrow < rows && col0 < N;  // N is a multiple of 64
      const bool valid = lrow + lane < rows;
      // full groups of 32 rows leave through TMA stores, others row by row
      const bool staged = lrow + 32 <= rows || (!q.sums && a.clipped);
      const bool f32 = q.sums ? a.sum_out != nullptr : a.out_f32;
      const CUtensorMap *map = q.sums ? &maps.so[q.job] : &maps.o;
      void *out = q.sums ? a.sum_out : a.out;  // (bf16 sums are always staged: M is a
                                               // multiple of 64)
      bool ok = wait_on(s, &ctl->tfull[buf], (it >> 1) & 1, a.err, 34);
      __syncwarp();
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t ta = s.tmem + ((uint32_t)(ew * 32) << 16) + (uint32_t)(buf * 256 + part * 64);
      if (mine && staged) {
        if (lane == 0) bulk_wait_read_all();  // the previous tile's store has read the buffer
        __syncwarp();
      }
      if (mine) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float f[32];
          if (q.nkb == 0) {  // an expert without rows
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = 0.f;
          } else {
            uint32_t v[32];
            tmem_ld32(ta + c * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
          }
          if (f32 && staged) {  // 32 rows of 128 bytes, 16-byte pieces swizzled
            if (c > 0) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
            float4 *dst = reinterpret_cast<float4 *>(stage + lane * 128);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[j ^ (lane & 7)] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(map, stage, col0 + c * 32, (int)orow);
              bulk_commit();
            }
          } else if (f32) {
            if (valid) {
              float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) +
                                                       (orow + lane) * (size_t)N + col0 + c * 32);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                dst[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
            }
          } else if (valid) {
            // staged: the lane's row of 128 bytes, 16-byte pieces swizzled
            uint4 *dst = staged ? reinterpret_cast<uint4 *>(stage + lane * 128)
                                : reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) +
                                                            (orow + lane) * (size_t)N + col0);
            const int sw = staged ? lane & 7 : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float h[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) h[i] = f[j * 8 + i];
              dst[(c * 4 + j) ^ sw] = pack16(h);
            }
          }
        }
      }
      release_tmem<true>(s, tempty0, buf);
      if (mine && staged && !f32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map, stage, col0, (int)orow);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tear_down<true>(s);
}

// ------------------------------------------------------------------ host side
std::mutex g_mu;

// A persistent grid of CTA pairs (or CTAs), at most `tiles` of them; `slot` names the kernel
// in the per-device table of grid sizes.
template <bool PAIR, typename... KArgs, typename... Args>
cudaError_t launch_grid(void (*kernel)(KArgs...), int slot, int threads, size_t smem,
                         long long tiles, cudaStream_t st, const Args &...args) {
  static int max_groups[64][4] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int &most = max_groups[dev & 63][slot];
  {
    std::lock_guard<std::mutex> lock(g_mu);
    if (most == 0) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)smem);
      if (e != cudaSuccess) return e;
      int n = PAIR ? sm_count() / 2 : sm_count();
      if (PAIR) {
        cfg.gridDim = dim3(2 * n);
        int fit = 0;
        if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) == cudaSuccess && fit > 0) n = fit;
      }
      most = n;
    }
  }
  cfg.gridDim = dim3((unsigned)((PAIR ? 2 : 1) *
                                std::max<long long>(1, std::min<long long>(tiles, most))));
  cfg.numAttrs = take_pdl() ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_act_grad_tc(const FfnGradArgs &f, cudaStream_t st) {
  const bool glu = f.act == MOE_ACT_SWIGLU;
  const bool single = !glu && f.row_bound <= (long long)kRowTile * f.G;
  ActMaps m;
  const uint64_t R = (uint64_t)f.rows, X = (uint64_t)f.x_rows, d = (uint64_t)f.d,
                 F = (uint64_t)f.F, G = (uint64_t)f.G;
  bool ok = make_map(&m.x, f.x, X, d, kRowTile) && make_map(&m.dy, f.dy, X, d, kRowTile) &&
            make_map(&m.w1, f.w1, G * F, d, glu || single ? kRowTile : kBlockK) &&
            make_map(&m.w2, f.w2, G * d, F, kBlockK) && make_store_map(&m.h, f.h, R, F) &&
            make_store_map(&m.dg, f.dg, R, F);
  m.w3 = m.w1;
  m.du = m.dg;
  if (glu)
    ok = ok && make_map(&m.w3, f.w3, G * F, d, kRowTile) && make_store_map(&m.du, f.du, R, F);
  if (!ok) return cudaErrorInvalidValue;
  ActArgs a{};
  a.poff = f.poff;
  a.offsets = f.offsets;
  a.G = f.G;
  a.F = f.F;
  a.d = f.d;
  a.act = f.act;
  a.n_tiles = ceil_div(f.F, kTileN);
  a.b1 = f.b1;
  a.row_w = f.row_w;
  a.dot_part = f.row_dot ? f.dot_part : nullptr;
  a.col_part = f.db1 ? f.col_part : nullptr;
  a.rows = f.rows;
  a.x_rows = f.x_rows;
  a.err = f.err;
  const long long tiles = (long long)f.pair_tiles_ub * a.n_tiles;
  if (glu)
    return launch_grid<true>(k_act_grad<true, true>, 0, ActCfg<true, true>::kThreads,
                             ActCfg<true, true>::kSmem, tiles, st, m, a);
  if (single)
    return launch_grid<false>(k_act_grad<false, false>, 3, ActCfg<false, false>::kThreads,
                              ActCfg<false, false>::kSmem, 2 * tiles, st, m, a);
  return launch_grid<true>(k_act_grad<false, true>, 1, ActCfg<false, true>::kThreads,
                           ActCfg<false, true>::kSmem, tiles, st, m, a);
}

cudaError_t launch_products_tc(const FfnGradArgs &f, int splits, cudaStream_t st) {
  const bool glu = f.act == MOE_ACT_SWIGLU;
  const uint64_t R = (uint64_t)f.rows, X = (uint64_t)f.x_rows, d = (uint64_t)f.d,
                 F = (uint64_t)f.F, G = (uint64_t)f.G;
  GemmMaps m;
  GemmArgs a{};
  bool ok = true;
  long long tiles = 0;
  if (f.dx) {
    ok = make_map(&m.a[0], f.dg, R, F, kRowTile) && make_mn_map(&m.b[0], f.w1, G * F, d);
    if (glu)
      ok = ok && make_map(&m.a[1], f.du, R, F, kRowTile) && make_mn_map(&m.b[1], f.w3, G * F, d);
    ok = ok && (f.dx_f32 ? make_f32_map(&m.o, f.dx, (uint64_t)f.dx_rows, d)
                         : make_map(&m.o, f.dx, (uint64_t)f.dx_rows, d, 32));
    a.poff = f.poff;
    a.offsets = f.offsets;
    a.pre = f.pre256;
    a.out_off = f.dx_off;
    a.G = f.G;
    a.N = f.d;
    a.K = f.F;
    a.nseg = glu ? 2 : 1;
    a.a_rows = f.rows;
    a.out = f.dx;
    a.out_f32 = f.dx_f32;
    a.splits = splits;
    a.piece = ceil_div(a.nseg * ceil_div(f.F, kBlockK), splits);
    if (splits > 1) {
      ok = ok && make_f32_map(&m.o, f.dx_part, (uint64_t)splits * R, d);
      a.out = f.dx_part;
      a.out_f32 = 1;
      a.out_off = f.poff;
      a.part_rows = f.rows;
    }
    a.clipped = a.out_off == f.poff;  // the rows behind an expert's are its own padding
    tiles += (long long)f.pair_tiles_ub * ceil_div(f.d, 256) * splits;
  }
  auto job = [&](const void *p, uint64_t prows, const void *q, uint64_t qrows, void *out, int M,
                 int N) {
    if (out == nullptr) return;
    const int j = a.njobs++;
    ok = ok && make_mn_map(&m.sa[j], p, prows, (uint64_t)M) &&
         make_mn_map(&m.sb[j], q, qrows, (uint64_t)N) &&
         make_map(&m.so[j], out, G * (uint64_t)M, (uint64_t)N, 32);
    a.M[j] = M;
    a.Ns[j] = N;
    tiles += (long long)f.G * ceil_div(M, kPairM) * ceil_div(N, 256);
  };
  job(f.dg, R, f.x, X, f.dw1, f.F, f.d);
  if (glu) job(f.du, R, f.x, X, f.dw3, f.F, f.d);
  job(f.dy, X, f.h, R, f.dw2, f.d, f.F);
  if (tiles == 0) return cudaSuccess;
  if (!ok) return cudaErrorInvalidValue;
  a.first = f.poff;
  a.groups = f.G;
  a.err = f.err;
  return launch_grid<true>(k_pair_gemm, 2, kGemmThreads, kGemmSmem, tiles, st, m, a);
}

cudaError_t launch_route_tc(const RouteTcArgs &r, cudaStream_t st) {
  GemmMaps m;
  GemmArgs a{};
  bool ok = true;
  long long tiles = 0;
  const uint64_t T = (uint64_t)r.T, ld = (uint64_t)kSplit * r.Ep, d = (uint64_t)r.d;
  if (r.dx) {
    for (int j = 0; j < kSplit; ++j)
      ok = ok &&
           make_map_ld(&m.a[j], r.terms + (size_t)j * r.Ep, T, (uint64_t)r.Ep, kRowTile, ld) &&
           make_mn_map(&m.b[j], r.w, (uint64_t)r.E, d);
    ok = ok && make_f32_map(&m.o, r.dx, T, d);
    a.poff = r.all;
    a.offsets = a.out_off = r.all_rows;
    a.pre = r.all_tiles;
    a.G = 1;
    a.N = r.d;
    a.K = r.Ep;
    a.nseg = kSplit;
    a.splits = 1;
    a.piece = kSplit * ceil_div(r.Ep, kBlockK);
    a.a_rows = r.T;
    a.out = r.dx;
    a.out_f32 = 1;
    a.clipped = 1;
    tiles += (long long)ceil_div(r.T, kPairM) * ceil_div(r.d, 256);
  }
  if (r.dw_part) {
    // the terms side by side are the rows of one product: x is read once for both
    const int M = kSplitDw * r.Ep;
    ok = ok && make_mn_map(&m.sa[0], r.terms, T, (uint64_t)M, ld) &&
         make_mn_map(&m.sb[0], r.x, T, d) &&
         make_f32_map(&m.so[0], r.dw_part, (uint64_t)r.pieces * M, d);
    a.groups = r.pieces;
    a.njobs = 1;
    a.M[0] = M;
    a.Ns[0] = r.d;
    a.sum_out = r.dw_part;
    tiles += (long long)r.pieces * ceil_div(M, kPairM) * ceil_div(r.d, 256);
  }
  if (!ok) return cudaErrorInvalidValue;
  a.first = r.piece;  // (read up to `groups`, which is 0 without dw)
  a.err = r.err;
  return launch_grid<true>(k_pair_gemm, 2, kGemmThreads, kGemmSmem, tiles, st, m, a);
}

}  // namespace moe
