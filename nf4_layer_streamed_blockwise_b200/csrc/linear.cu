// Dense bf16 linear with bias, activation and residual in its epilogue, and
// its backward (sm_100a: tcgen05 + TMEM + TMA).
//
//   forward   z = x W^T + b,  y = residual + act(z)       x [M, K], W [N, K]
//   backward  dz = dy act'(z),  db = sum_m dz,  dx = dz W,  dW = dz^T x
//
// All three products are one form, out[q][p] = sum_c Q[q, c] P[p, c], with the
// operands read by TMA in the layout they have (K-major: the contraction is
// the contiguous axis; MN-major: the output axis is):
//   forward  p = n, q = m, c = k:  P = W  K-major,   Q = x  K-major
//   dx       p = k, q = m, c = n:  P = W  MN-major,  Q = dz K-major
//   dW       p = k, q = n, c = m:  P = x  MN-major,  Q = dz MN-major
//
// Two forms share them (one row's forward has a third): one tile per cluster with the contraction split (few
// tiles: bound by what L2 feeds an SM, and below that by start and exchange; dx and dW share a launch there)
// and a persistent CTA-pair form (many tiles: bound by the tensor cores, in a
// long run by the power cap); plan_product picks by a measured cost model.
// Measured on B200 (graph replays): 2048 x 14336 x 4096 forward 155-157 us with
// any activation (1.55 PFLOP/s; 138 us and 86% of the tensor pipe in isolation
// at full clock), 171 with bias, residual and z kept, dx 163, dW 168;
// 333 x 1536 x 576 4.7; 1 x 4096 x 4096 7.4 with the weight from HBM.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "common.cuh"
#include "host_common.h"

namespace lsq {
namespace nrm {
lsq_status col_sum(const float* part, int G, int64_t ld, int64_t n0, int64_t ncols, float* out0, float* out1,
                   int accumulate, cudaStream_t stream);
}
namespace lin {

using ops::pack8;
using ops::unpack8;

// One lane of the converged warp, the same each time.  The producer and issuer warps run their loops whole
// and elect a lane at the asynchronous instructions only: under an `if (lane == 0)` around the loop the compiler
// cannot keep addresses and descriptors in uniform registers, and a 64-deep block cost 0.26 us of issue
// whatever the tile's size; so it costs 0.165 (1 x 4096 x 4096 unsplit: 20.8 -> 14.9 us).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// ---------------------------------------------------------------- activations
// act(z) and act'(z) in fp32 on the fp32 pre-activation, two values at a time (f32x2; scalar, the derivative
// of GELU took longer than its bytes), through the special-function unit's exp2 and reciprocal (relative error
// about 2^-22).  Relative to the result they are off by at most 2^-12, a sixteenth of half a bf16 step, for negative
// z too: the rounding of exp2's argument, up to 126 in size, is 2e-5 of it and the fit of the normal tail 1e-4;
// derivatives by 2^-11 from z = -2 down, and near their zero by 1e-6 in absolute terms.  Factors below 2^-126 are
// flushed to 0 (SiLU from z = -87.3 down, the two GELUs from -13.2 and -10).  The logistic under- and overflows to
// the right limits; what would meet 0 * inf is taken out at the end.
__device__ __forceinline__ float ex2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t both(float x) { return f2(x, x); }
__device__ __forceinline__ uint64_t ex2_2(uint64_t x) {
  const float2 f = f2split(x);
  return f2(ex2_f(f.x), ex2_f(f.y));
}
__device__ __forceinline__ uint64_t rcp_2(uint64_t x) {
  const float2 f = f2split(x);
  return f2(rcp_f(f.x), rcp_f(f.y));
}
constexpr float LOG2E = 1.4426950408889634f;
constexpr float GT_C = 1.5957691216057308f;  // 2 sqrt(2 / pi): z (1 + tanh(u)) / 2 = z logistic(2 u)
constexpr float GT_A = 0.044715f;
// logistic(u) with v = -u log2(e)
__device__ __forceinline__ uint64_t logistic2(uint64_t v) { return rcp_2(add2(ex2_2(v), both(1.0f))); }
__device__ __forceinline__ uint64_t gelu_tanh_arg(uint64_t z) {
  return mul2(z, fma2(mul2(z, z), both(-LOG2E * GT_C * GT_A), both(-LOG2E * GT_C)));
}
// Phi(z); e = exp(-z^2 / 2).  The tail Phi(-|z|) = e R(|z|) is computed itself and only subtracted from 1 for z > 0, so
// small results keep their relative accuracy: formed as 1/2 - (1/2 - tail) it is off by 4% at z = -5.  R(a) =
// erfcx(a / sqrt 2) / 2 as t q(t), t = 1 / (1 + 0.29 a), q of degree 5: an own fit, weighted minimax over 0 <= a <= 13.3
// (where e reaches 2^-126), off by at most 4.8e-8 / e in absolute and 1e-4 in relative terms.
__device__ __forceinline__ uint64_t normal_cdf2(uint64_t z, uint64_t& e) {
  const uint64_t az = z & 0x7fffffff7fffffffull;
  const uint64_t t = rcp_2(fma2(az, both(0.29f), both(1.0f)));
  uint64_t q = fma2(both(-0.08963339f), t, both(0.28783932f));
  q = fma2(q, t, both(-0.09734405f));
  q = fma2(q, t, both(0.18232992f));
  q = fma2(q, t, both(0.09983516f));
  q = fma2(q, t, both(0.11697299f));
  e = ex2_2(mul2(mul2(z, z), both(-0.5f * LOG2E)));
  const uint64_t tail = mul2(mul2(q, t), e);
  const int lo = (int)(uint32_t)z, hi = (int)(uint32_t)(z >> 32);  // by the sign bit, -0 too: 0 + tail or 1 - tail
  return add2(f2(lo < 0 ? 0.0f : 1.0f, hi < 0 ? 0.0f : 1.0f), tail ^ (~z & 0x8000000080000000ull));
}
template <int ACT>
__device__ __forceinline__ uint64_t act2(uint64_t z) {
  if (ACT == LSQ_ACT_NONE) return z;
  const float2 f = f2split(z);
  if (ACT == LSQ_ACT_RELU) return f2(f.x < 0.0f ? 0.0f : f.x, f.y < 0.0f ? 0.0f : f.y);  // a NaN stays one
  uint64_t e, s;
  if (ACT == LSQ_ACT_GELU) s = normal_cdf2(z, e);
  if (ACT == LSQ_ACT_GELU_TANH) s = logistic2(gelu_tanh_arg(z));
  if (ACT == LSQ_ACT_SILU) s = logistic2(mul2(z, both(-LOG2E)));
  const float2 y = f2split(mul2(z, s));
  return f2(f.x == -INFINITY ? 0.0f : y.x, f.y == -INFINITY ? 0.0f : y.y);
}
template <int ACT>
__device__ __forceinline__ uint64_t dact2(uint64_t z) {
  if (ACT == LSQ_ACT_NONE) return both(1.0f);
  const float2 f = f2split(z);
  if (ACT == LSQ_ACT_RELU)
    return f2(f.x > 0.0f ? 1.0f : (f.x == f.x ? 0.0f : f.x), f.y > 0.0f ? 1.0f : (f.y == f.y ? 0.0f : f.y));
  uint64_t e, d;
  if (ACT == LSQ_ACT_GELU) {
    d = normal_cdf2(z, e);
    d = fma2(mul2(z, both(0.3989422804014327f)), e, d);
  }
  if (ACT == LSQ_ACT_GELU_TANH) {  // s + z s (1 - s) u'
    const uint64_t s = logistic2(gelu_tanh_arg(z));
    const uint64_t du = fma2(mul2(z, z), both(3.0f * GT_C * GT_A), both(GT_C));
    d = fma2(mul2(mul2(z, s), du), add2(both(1.0f), s ^ 0x8000000080000000ull), s);
  }
  if (ACT == LSQ_ACT_SILU) {  // s (1 + z (1 - s))
    const uint64_t s = logistic2(mul2(z, both(-LOG2E)));
    d = mul2(s, fma2(z, add2(both(1.0f), s ^ 0x8000000080000000ull), both(1.0f)));
  }
  // beyond |z| = 1e4 every derivative here is 0 or 1 in fp32, and the products above meet inf * 0
  const float2 y = f2split(d);
  return f2(fabsf(f.x) > 1e4f ? (f.x > 0.0f ? 1.0f : 0.0f) : y.x, fabsf(f.y) > 1e4f ? (f.y > 0.0f ? 1.0f : 0.0f) : y.y);
}

template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = f2split(act2<ACT>(f2(v[i], v[i + 1])));
    v[i] = y.x;
    v[i + 1] = y.y;
  }
}
template <int N>
__device__ __forceinline__ void act_of(int act, float (&v)[N]) {
  switch (act) {
    case LSQ_ACT_RELU: act_all<LSQ_ACT_RELU>(v); break;
    case LSQ_ACT_GELU: act_all<LSQ_ACT_GELU>(v); break;
    case LSQ_ACT_GELU_TANH: act_all<LSQ_ACT_GELU_TANH>(v); break;
    case LSQ_ACT_SILU: act_all<LSQ_ACT_SILU>(v); break;
    default: break;
  }
}

struct Epi {
  const __nv_bfloat16* bias;      // [P] or null
  const __nv_bfloat16* residual;  // [Q, P] or null; may alias out
  __nv_bfloat16* z;               // [Q, P] or null
  void* out;                      // [Q, P] bf16, or fp32 (f32)
  int act, f32, accumulate;       // accumulate: fp32 out is added to
};

struct Params {
  int P, Q, nkb;   // output columns and rows, 64-deep contraction blocks
  int tp, splits;  // 128-column tiles; cluster size (contraction split), a power of two
  int lper;        // log2 of the rows each CTA of a cluster finishes
  int bn;          // persistent form: tile columns, a multiple of 32 up to 256
  Epi e;
};
struct Maps {
  CUtensorMap p, q;
};

// What the epilogue of eight neighbouring columns of one output row reads, fetched ahead: the forward's residual, or
// what an accumulating fp32 output holds.
struct Ahead {
  uint4 a, b;
};
template <bool FWD>
__device__ __forceinline__ Ahead epi_fetch(const Epi& e, int64_t off, bool in) {
  Ahead h{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (FWD && in && e.residual) h.a = *reinterpret_cast<const uint4*>(e.residual + off);
  if (!FWD && in && e.accumulate) {
    const uint4* o = reinterpret_cast<const uint4*>(static_cast<const float*>(e.out) + off);
    h.a = o[0];
    h.b = o[1];
  }
  return h;
}
__device__ __forceinline__ uint4 epi_bias(const Epi& e, int col, bool in) {
  return in && e.bias ? *reinterpret_cast<const uint4*>(e.bias + col) : make_uint4(0u, 0u, 0u, 0u);
}
// forward: bias, z, activation, residual, one rounding, one store; a gradient: bf16, or fp32 (added)
template <bool FWD>
__device__ __forceinline__ void finish8(float (&v)[8], const Epi& e, int64_t off, uint4 bias, const Ahead& h) {
  if (!FWD && e.f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(e.out) + off);
    if (e.accumulate) {
      v[0] += __uint_as_float(h.a.x); v[1] += __uint_as_float(h.a.y);
      v[2] += __uint_as_float(h.a.z); v[3] += __uint_as_float(h.a.w);
      v[4] += __uint_as_float(h.b.x); v[5] += __uint_as_float(h.b.y);
      v[6] += __uint_as_float(h.b.z); v[7] += __uint_as_float(h.b.w);
    }
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  if (FWD) {
    float b[8];
    if (e.bias) {
      unpack8(bias, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
    if (e.z) *reinterpret_cast<uint4*>(e.z + off) = pack8(v);
    act_of(e.act, v);
    if (e.residual) {
      unpack8(h.a, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(e.out) + off) = pack8(v);
}

// ---------------------------------------------------------------- one tile per cluster
// 128 output columns (the tensor core's M, so few output rows waste none of it) x BT output rows; the S
// CTAs of a cluster split the contraction, each leaves its fp32 partial tile in the shared memory of the
// CTA that finishes those rows (BT / S of them), and that CTA adds them in rank order: no atomics, no
// second kernel, no workspace.
constexpr int BP = 128, BK = 64, NTHREADS = 256, MAX_S = 8;
constexpr int P_BYTES = BP * BK * 2;

// Descriptor of an operand tile at saddr, and its step per 16 of the contraction (16-byte units).  One thread
// issues every product: with the descriptors rebuilt for each instruction it took about 590 cycles a block,
// more than the tensor core needs for 256 columns, so the loops only add constants to these.
template <int MN>
__device__ __forceinline__ uint64_t op_desc(uint32_t saddr) {
  return MN ? smem_desc(saddr, 8192, 1024, 2) : smem_desc(saddr, 16, 1024, 2);
}
template <int MN>
constexpr uint64_t DSTEP = MN ? 2048 / 16 : 32 / 16;

template <int BT>
struct Cfg {
  static constexpr int Q_BYTES = BT * BK * 2;
  static constexpr int STAGE = P_BYTES + Q_BYTES;
  static constexpr int XCHG = BT * BP * 4;  // [S sources][BT / S rows][128] fp32
  static constexpr int NST = BT <= 16 ? 10 : BT <= 32 ? 8 : BT <= 64 ? 6 : 4;
  static constexpr int OFF_X = NST * STAGE;
  static constexpr int OFF_BAR = OFF_X + XCHG;
  static constexpr int OFF_MISC = OFF_BAR + 8 * (2 * NST + 1);
  static constexpr int BYTES = OFF_MISC + 16 + 1024;
  static constexpr int TCOLS = BT < 32 ? 32 : BT;
  static_assert(BYTES <= 232448, "shared memory");
};

template <int PMN, int QMN, int BT>
__device__ __forceinline__ void split_tile(const Maps& maps, const Params& p, int block, uint8_t* smem_raw) {
  using C = Cfg<BT>;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* afull = empty + C::NST;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits, rank = block % S, tile = block / S;
  const int p0 = (tile % p.tp) * BP, q0 = (tile / p.tp) * BT;
  const int kb0 = (int)((int64_t)p.nkb * rank / S);
  const int kb1 = q0 < p.Q ? (int)((int64_t)p.nkb * (rank + 1) / S) : kb0;  // else a block that fills up a cluster
  const int first = (int)nf4g::cluster_ctarank() - rank;  // the tile's first CTA: a cluster may hold several tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(afull, 1);
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(s_tmem, C::TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  grid_release();
  grid_wait();
  // the cluster's CTAs have started once this phase completes (waited for before the exchange)
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  if (warp == 4) {
    int s = 0;
    uint32_t ph = 1;  // the ring starts empty
    for (int i = kb0; i < kb1; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph, 431))) break;
      if (elect_one()) {
        uint8_t* pd = smem + s * C::STAGE;
        uint8_t* qd = pd + P_BYTES;
        mbar_arrive_expect_tx(&full[s], (uint32_t)C::STAGE);
        if (!PMN) {
          tma_load_2d(pd, &maps.p, &full[s], i * BK, p0);
        } else {
          tma_load_2d(pd, &maps.p, &full[s], p0, i * BK);
          tma_load_2d(pd + 8192, &maps.p, &full[s], p0 + 64, i * BK);
        }
        if (!QMN) {
          tma_load_2d(qd, &maps.q, &full[s], i * BK, q0);
        } else {
#pragma unroll
          for (int c = 0; c < BT / 64; ++c) tma_load_2d(qd + c * 8192, &maps.q, &full[s], q0 + c * 64, i * BK);
        }
      }
      __syncwarp();
      if (++s == C::NST) s = 0, ph ^= 1;
    }
  } else if (warp == 5) {
    const uint32_t id = idesc_bf16(BP, BT, PMN, QMN);
    const uint64_t pd0 = op_desc<PMN>(smem_u32(smem)), qd0 = op_desc<QMN>(smem_u32(smem) + P_BYTES);
    int s = 0;
    uint32_t ph = 0;
    for (int i = kb0; i < kb1; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, 531))) {
        mbar_drain(full, C::NST, s, ph, 532);
        break;
      }
      tc_fence_after();
      const uint64_t at = (uint64_t)(s * (C::STAGE >> 4));
      if (elect_one()) {
        tc_mma(tmem, pd0 + at, qd0 + at, id, i != kb0);
#pragma unroll
        for (int kk = 1; kk < BK / 16; ++kk)
          tc_mma(tmem, pd0 + at + kk * DSTEP<PMN>, qd0 + at + kk * DSTEP<QMN>, id, 1);
        tc_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == C::NST) s = 0, ph ^= 1;
    }
    if (elect_one()) tc_commit(afull);  // also when a wait gave up: the epilogue is not left waiting
    __syncwarp();
  }
  const int lper = p.lper, per = 1 << lper;  // output rows this CTA finishes
  // a thread finishes eight columns (always the same) of the rows fr, fr + 16, ...; what it reads for them is under
  // way before the sums are there (16 x 4096 x 4096 with bias and residual 9.1 us, now 7.9; an accumulating fp32 dW of
  // 333 x 1536 x 576 with its dx 9.0, 7.4)
  const int fr = (int)threadIdx.x / (BP / 8), fc = (int)threadIdx.x % (BP / 8) * 8;
  const bool in = p0 + fc < p.P;
  const int64_t off0 = (int64_t)(q0 + rank * per) * p.P + p0 + fc;
  auto fetch = [&](int r) {
    return epi_fetch<!PMN>(p.e, off0 + (int64_t)r * p.P, in && r < per && q0 + rank * per + r < p.Q);
  };
  const uint4 bias = epi_bias(p.e, p0 + fc, in && !PMN);
  Ahead ahead = fetch(fr);
  if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp < 4) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(afull, 0, 731));
    tc_fence_after();
    if (ok && kb1 > kb0) {
      const uint32_t lb = tmem + ((uint32_t)(warp * 32) << 16);
      // row r of the tile is finished by rank r >> lper, as its row r & (per - 1).  Rolled: the code runs once
      // per block, so what counts is the instructions fetched (unrolled eightfold 333 x 1536 x 576 took 19.1
      // us, not 7.8, with 128 rows in two)
      const uint32_t mine = smem_u32(smem + C::OFF_X) + (uint32_t)(((rank << lper) * BP + warp * 32 + lane) * 4);
#pragma unroll 1
      for (int c = 0; c < BT; c += 16) {
        float v[16];
        tmem_ld16(lb + (uint32_t)c, v);
        tc_wait_ld();
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const uint32_t dst = mine + (uint32_t)(((c + t) & (per - 1)) * (BP * 4));
          uint32_t a;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(dst), "r"(first + ((c + t) >> lper)));
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v[t]) : "memory");
        }
      }
    }
    tc_fence_before();
  }
  if (S > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
  const float* xs = reinterpret_cast<const float*>(smem + C::OFF_X);
  if (!in) return;
#pragma unroll 2  // 512 x 2048 x 2048: 10.2 us rolled, 9.9 by two, 9.9 by four
  for (int r = fr; r < per && q0 + rank * per + r < p.Q; r += NTHREADS / (BP / 8)) {
    const Ahead h = ahead;
    ahead = fetch(r + NTHREADS / (BP / 8));
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll 1
    for (int k = 0; k < S; ++k) {  // rank order
      const float4* a = reinterpret_cast<const float4*>(xs + ((k << lper) + r) * BP + fc);
      const float4 lo = a[0], hi = a[1];
      v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
      v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
    }
    finish8<!PMN>(v, p.e, off0 + (int64_t)r * p.P, bias, h);
  }
}

template <int PMN, int QMN, int BT>
__global__ void __launch_bounds__(NTHREADS, 1) linear_split_kernel(const __grid_constant__ Maps maps,
                                                                   const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  split_tile<PMN, QMN, BT>(maps, p, (int)blockIdx.x, smem_raw);
}

// dx and dW of a small linear in one launch: the first blocks are dx's, the rest dW's, side by side in one round
struct Both {
  Maps mx, mw;
  Params x, w;
  int nx;  // blocks of dx
};
template <int BX, int BW>
__global__ void __launch_bounds__(NTHREADS, 1) linear_both_kernel(const __grid_constant__ Both b) {
  extern __shared__ uint8_t smem_raw[];
  if ((int)blockIdx.x < b.nx) split_tile<1, 0, BX>(b.mx, b.x, (int)blockIdx.x, smem_raw);
  else split_tile<1, 1, BW>(b.mw, b.w, (int)blockIdx.x - b.nx, smem_raw);
}

// ---------------------------------------------------------------- persistent form
// For outputs of many tiles.  A cluster of two CTAs on two SMs computes 256 rows x bn columns (cta_group::2:
// each CTA stages its 128 rows and half of the columns, 32 KB per 64-deep block where a lone CTA's 128 x 256
// tile takes 48: the single-CTA form ran at the rate L2 fed it, 1370 TFLOP/s for 2048 x 14336 x 4096).
// Clusters walk tiles c, c + C, ... (row tile fastest, so those that share a slice of P run together); two
// TMEM accumulators alternate, so the epilogue of a tile runs under the products of the next.  Warps 0-7:
// epilogue (warp w: the 32 rows of TMEM lanes 32 (w % 4), every other 32-column piece from piece w / 4 on:
// two warps per scheduler, since the activations cost about as much as the products of a short
// contraction); warp 8: TMA producer; warp 9: MMA issuer (leader).  Each 32 x 32 piece is staged in shared
// memory (swizzled, no bank conflicts) and leaves by TMA, which clips the edges; an accumulated fp32
// output leaves as a TMA reduction (one addend per element and call: the order of adds is that of the calls).
constexpr int TM = 256, GST = 6, GTHREADS = 320, EPI_WARPS = 8;
constexpr int GA_BYTES = 128 * BK * 2, GSTAGE = 2 * GA_BYTES;
constexpr int G_OFF_STG = GST * GSTAGE;
constexpr int STG_BYTES = 2048;  // one bf16 piece; an fp32 piece takes both of a warp's buffers
constexpr int G_OFF_BAR = G_OFF_STG + EPI_WARPS * 2 * STG_BYTES;
constexpr int G_OFF_MISC = G_OFF_BAR + 8 * (2 * GST + 5);
constexpr int G_BYTES = G_OFF_MISC + 16 + 1024;
static_assert(G_BYTES <= 232448, "shared memory");

struct GMaps {
  CUtensorMap a, b, out, z;  // a: Q side (rows of the output), b: P side (columns)
};

// TMA add of a staged box into fp32 global memory, in the thread's current bulk group
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* m, const void* src, int x, int y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}

template <int AMN, int BMN, int F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GTHREADS, 1)
    linear_pair_kernel(const __grid_constant__ GMaps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G_OFF_BAR);  // the leader's: both CTAs' loads
  uint64_t* empty = full + GST;
  uint64_t* tfull = empty + GST;
  uint64_t* tempty = tfull + 2;  // the leader's: both CTAs' epilogue warps
  uint64_t* drain = tempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + G_OFF_MISC);
  const uint32_t rank = nf4g::cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntm = (p.Q + TM - 1) / TM, tiles = ntm * ((p.P + p.bn - 1) / p.bn);
  const int cid = (int)(blockIdx.x >> 1), ncl = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < GST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 9) {
    nf4g::tmem_alloc_pair(s_tmem, 512);
    nf4g::tmem_relinquish_pair();
  }
  tc_fence_before();
  nf4g::cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  grid_release();
  grid_wait();

  if (warp == 8) {
    const int hb = p.bn / 2, nbox = (hb + 63) / 64;  // this CTA's columns; 64-wide boxes of an MN-major P
    const uint32_t bytes = 2u * (uint32_t)(GA_BYTES + (BMN ? nbox * 8192 : hb * 128));
    const uint32_t full0 = nf4g::cluster_addr(full, 0);
    int s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int t = cid; ok && t < tiles; t += ncl) {
      const int m0 = (t % ntm) * TM + (int)rank * 128, n0 = (t / ntm) * p.bn + (int)rank * hb;
      for (int i = 0; i < p.nkb; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ph, 441));
        if (!ok) break;
        if (elect_one()) {
          uint8_t* ad = smem + s * GSTAGE;
          uint8_t* bd = ad + GA_BYTES;
          const uint32_t fl = full0 + (uint32_t)s * 8;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          if (!AMN) {
            nf4g::tma_load_2d_pair(ad, &maps.a, fl, i * BK, m0);
          } else {
            nf4g::tma_load_2d_pair(ad, &maps.a, fl, m0, i * BK);
            nf4g::tma_load_2d_pair(ad + 8192, &maps.a, fl, m0 + 64, i * BK);
          }
          if (!BMN) {
            nf4g::tma_load_2d_pair(bd, &maps.b, fl, i * BK, n0);
          } else {
            nf4g::tma_load_2d_pair(bd, &maps.b, fl, n0, i * BK);
            if (nbox > 1) nf4g::tma_load_2d_pair(bd + 8192, &maps.b, fl, n0 + 64, i * BK);
          }
        }
        __syncwarp();
        if (++s == GST) s = 0, ph ^= 1;
      }
    }
  } else if (warp == 9) {
    if (rank == 0) {
      const uint32_t id = idesc_bf16(TM, p.bn, AMN, BMN);
      const uint64_t ad0 = op_desc<AMN>(smem_u32(smem)), bd0 = op_desc<BMN>(smem_u32(smem) + GA_BYTES);
      int s = 0, j = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = cid; ok && t < tiles; t += ncl, ++j) {
        const int buf = j & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(&tempty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, 541));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * 256);
        for (int i = 0; i < p.nkb; ++i) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph, 542));
          if (!ok) break;
          tc_fence_after();
          const uint64_t at = (uint64_t)(s * (GSTAGE >> 4));
          if (elect_one()) {
            nf4g::tc_mma_pair(d, ad0 + at, bd0 + at, id, i != 0);
#pragma unroll
            for (int kk = 1; kk < BK / 16; ++kk)
              nf4g::tc_mma_pair(d, ad0 + at + kk * DSTEP<AMN>, bd0 + at + kk * DSTEP<BMN>, id, 1);
            nf4g::tc_commit_pair_mc(&empty[s], 0x3);
          }
          __syncwarp();
          if (++s == GST) s = 0, ph ^= 1;
        }
        if (ok && elect_one()) nf4g::tc_commit_pair_mc(&tfull[buf], 0x3);
        __syncwarp();
      }
      if (!ok) {
        if (elect_one()) nf4g::tc_commit_pair(drain);
        __syncwarp();
        mbar_wait(drain, 0, 543);
        mbar_drain(full, GST, s, ph, 544);
      }
    }
  } else {
    const Epi& e = p.e;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int wg = warp >> 2;
    uint8_t* stg = smem + G_OFF_STG + warp * 2 * STG_BYTES;
    int j = 0, k = 0;
    for (int t = cid; t < tiles; t += ncl, ++j) {
      const int row0 = (t % ntm) * TM + (int)rank * 128 + (warp & 3) * 32, n0 = (t / ntm) * p.bn;
      const int buf = j & 1, row = row0 + lane;
      const int nc = row0 < p.Q ? (min(p.bn, p.P - n0) + 31) / 32 : 0;  // 32-column pieces inside the output
      // under way before the products are done: the bias of the warp's four pieces, sixteen bytes a lane, and each
      // piece's residual while the piece before it is finished (read where they are used they cost each piece
      // their latency: 8192 x 2048 x 128 with bias 19.3 us, not 13.5, 2048 x 4096 x 1024 24.2, not 19.7)
      uint4 bw = make_uint4(0u, 0u, 0u, 0u), rv[4];
      const int bcol = n0 + (wg + (lane >> 2) * 2) * 32 + (lane & 3) * 8;
      if (!F32 && e.bias && lane < 16 && bcol < p.P) bw = *reinterpret_cast<const uint4*>(e.bias + bcol);
      auto fetch_residual = [&](int c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = n0 + c * 32 + q * 8;
          rv[q] = (c < nc && row < p.Q && col < p.P)
                      ? *reinterpret_cast<const uint4*>(e.residual + (int64_t)row * p.P + col)
                      : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      if (!F32 && e.residual) fetch_residual(wg);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], (uint32_t)(j >> 1) & 1u, 741))) break;
      tc_fence_after();
      for (int c = wg; c < nc; c += 2) {
        const int col = n0 + c * 32;
        float v[32];
        tmem_ld32(tmem + lane_base + (uint32_t)(buf * 256 + c * 32), v);
        tc_wait_ld_regs(v);
        if (c + 2 >= nc) {  // this warp's part of the accumulator is in registers: hand it back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) nf4g::mbar_arrive_cluster(nf4g::cluster_addr(&tempty[buf], 0));
        }
        if (F32) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          dense::stage_row<1>(v, smem_u32(stg) + (uint32_t)lane * 128, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (e.accumulate) tma_add_2d(&maps.out, stg, col, row0);
            else tma_store_2d(&maps.out, stg, col, row0);
            bulk_commit();
          }
          continue;
        }
        if (e.bias) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int from = (c >> 1) * 4 + q;
            float b[8];
            unpack8(make_uint4(__shfl_sync(0xffffffffu, bw.x, from), __shfl_sync(0xffffffffu, bw.y, from),
                               __shfl_sync(0xffffffffu, bw.z, from), __shfl_sync(0xffffffffu, bw.w, from)), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q * 8 + i] += b[i];
          }
        }
        if (e.z) {
          if (lane == 0) bulk_wait_read<1>();  // the piece before last has left this buffer
          __syncwarp();
          dense::stage_row<0>(v, smem_u32(stg + k * STG_BYTES) + (uint32_t)lane * 64, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&maps.z, stg + k * STG_BYTES, col, row0);
            bulk_commit();
          }
          k ^= 1;
        }
        act_of(e.act, v);
        if (e.residual) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float r[8];
            unpack8(rv[q], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q * 8 + i] += r[i];
          }
          fetch_residual(c + 2);
        }
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        dense::stage_row<0>(v, smem_u32(stg + k * STG_BYTES) + (uint32_t)lane * 64, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&maps.out, stg + k * STG_BYTES, col, row0);
          bulk_commit();
        }
        k ^= 1;
      }
      if (wg >= nc) {  // no piece of this tile is this warp's
        tc_fence_before();
        __syncwarp();
        if (lane == 0) nf4g::mbar_arrive_cluster(nf4g::cluster_addr(&tempty[buf], 0));
      }
    }
    if (lane == 0) bulk_wait_all();  // the staged stores are written before the CTA exits
  }

  tc_fence_before();
  __syncwarp();
  nf4g::cluster_sync_all();
  if (warp == 9) {
    tc_fence_after();
    nf4g::tmem_dealloc_pair(tmem, 512);
  }
}

template <int AMN, int BMN, int F32>
static lsq_status launch_pair(const GMaps& maps, const Params& p, int64_t tiles, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  LSQ_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 0 && dev < 64 && !configured[dev]) {
    LSQ_CUDA_TRY(
        cudaFuncSetAttribute(linear_pair_kernel<AMN, BMN, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, G_BYTES));
    configured[dev] = 1;
  }
  const unsigned ncl = (unsigned)std::min<int64_t>(tiles, num_sms() / 2);
  return launch_chained("linear_pair_kernel", linear_pair_kernel<AMN, BMN, F32>, dim3(2 * ncl), GTHREADS, G_BYTES, 1,
                        stream, maps, p);
}

// ---------------------------------------------------------------- forward of one row
// A generated token: the weight is read once and HBM decides, so no tensor core and no tile: a block takes
// eight output columns, its warps share the contraction (warp w the 256-wide steps w, w + 8, ...), a lane
// multiplies 16-byte words of the eight weight rows with the row's words of x in f32x2, and the warps' sums
// join in shared memory in warp order.  Eight 16-byte loads a lane and step are in flight, and four blocks run on
// an SM (4096 x 4096 7.4 us with three, 6.4 with four, over three weights that L2 holds in part).  Weights from HBM,
// graph replays, against the tiles above: 4096 x 4096 7.4 us (8.9), 14336 x 4096 21.5 (22.6), 576 x 1536 2.4
// (3.8); the same kernel with two rows loses from 1 M weights on (13.5 us for 9.0: its products take over).
struct OneRow {
  const uint4 *x, *w;
  int N, k8;  // output columns, words of a row
  Epi e;
};
__global__ void __launch_bounds__(256, 4) linear_row_kernel(const __grid_constant__ OneRow p) {
  __shared__ float part[8][8];
  grid_release();
  grid_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 8;
  const uint4* w = p.w + (int64_t)col * p.k8;
  uint64_t acc[8];
#pragma unroll
  for (int f = 0; f < 8; ++f) acc[f] = 0ull;
  for (int c = warp * 32 + lane; c < p.k8; c += 256) {
    uint4 wv[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) wv[f] = w[(int64_t)f * p.k8 + c];
    uint64_t xv[4];
    nrm::unpack_pairs(p.x[c], xv);
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      uint64_t u[4];
      nrm::unpack_pairs(wv[f], u);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[f] = fma2(xv[j], u[j], acc[f]);
    }
  }
  const uint4 bias = epi_bias(p.e, col, threadIdx.x == 0);
  const Ahead ahead = epi_fetch<true>(p.e, col, threadIdx.x == 0);
#pragma unroll
  for (int f = 0; f < 8; ++f) {
    const float v = nrm::warp_sum(nrm::pair_sum(acc[f]));
    if (lane == 0) part[warp][f] = v;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  float v[8];
#pragma unroll
  for (int f = 0; f < 8; ++f) {
    v[f] = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[f] += part[k][f];
  }
  finish8<true>(v, p.e, col, bias, ahead);
}

// K-major operand [rows, C] with box {64, brows}; MN-major operand [C, rows] with box {64, 64}
static lsq_status map_operand(CUtensorMap* m, const void* base, int mn, int64_t rows, int64_t contraction, int brows) {
  return mn ? encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rows, contraction, rows * 2, 64, BK,
                             CU_TENSOR_MAP_SWIZZLE_128B)
            : encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, contraction, rows, contraction * 2, BK, brows,
                             CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int PMN, int QMN, int BT>
static lsq_status launch_split(const Maps& maps, const Params& p, int64_t clusters, cudaStream_t stream) {
  static int configured[64] = {0};
  int dev = 0;
  LSQ_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 0 && dev < 64 && !configured[dev]) {
    LSQ_CUDA_TRY(cudaFuncSetAttribute(linear_split_kernel<PMN, QMN, BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      Cfg<BT>::BYTES));
    configured[dev] = 1;
  }
  return launch_chained("linear_split_kernel", linear_split_kernel<PMN, QMN, BT>, dim3((unsigned)(clusters * p.splits)),
                        NTHREADS, Cfg<BT>::BYTES, (unsigned)p.splits, stream, maps, p);
}

// Which form a product takes, and its tile: the smallest estimate in us, from measurements of both forms on
// B200 (graph replays, 19 shapes from 1 x 4568 x 104 to 8192 x 5120 x 2048, every tile of each form):
//  * one tile per cluster, per round of the CTAs that fit: 0.16 + 0.0006 bt a 64-deep block (what L2 feeds one
//    SM) and 3.9 + 0.02 bt of start, exchange and stores.  1 x 4096 x 4096: 15.8 unsplit, 10.1 in two, 7.2 in
//    four (persistent: 19.2); 130 x 4096 x 4096: 14.2 with 128 rows in two (17.6).
//  * persistent: 4.5, and per round of the pairs the longer of products and epilogue plus a fifth of the
//    shorter.  A block costs 0.345 at 256 columns (the tensor cores, at the clock that the power cap leaves
//    them), in proportion to the columns down to 0.235 (what L2 feeds them); an MN-major P whose half tile is
//    no multiple of the 64-wide boxes loads columns that it does not use, 0.05 more.  Narrower tiles pay where
//    they fill the last round: 2048 x 14336 x 4096 takes 159.6 with 224 columns (6.9 rounds of 74 pairs), 166.2
//    with 256 (6.05); 512 x 4096 x 4096 18.6 with 128, 24.8 with 256 (one cluster a tile: 22.2).
// 64-deep blocks of a contraction; the tail reads as zeros (TMA out-of-bounds fill)
static int kblocks(int64_t C) { return (int)((C + BK - 1) / BK); }
struct Plan {
  int pair, bt, splits, bn;
  double us;
};
static double split_us(int bt, int nkb, int S) {
  return (0.16 + 0.0006 * bt) * ((nkb + S - 1) / S) + 3.9 + 0.02 * bt;
}
// CTAs in clusters of S that run at once: clusters do not straddle GPCs
static double split_fit(int S, int sms) { return S <= 2 ? sms : S == 4 ? sms - sms / 9 : sms - sms / 7; }
static Plan plan_product(int64_t P, int64_t Q, int nkb, int pmn, int qmn) {
  const int sms = num_sms();
  Plan best{};
  double tb = 1e30;
  const int64_t tp = (P + BP - 1) / BP;
  for (int bt = qmn ? 64 : 16; bt <= 128; bt *= 2) {
    const double tiles = (double)(tp * ((Q + bt - 1) / bt));
    for (int S = 1; S <= MAX_S && S <= nkb; S *= 2) {
      const double t = std::ceil(tiles * S / split_fit(S, sms)) * split_us(bt, nkb, S);
      if (t < tb) tb = t, best = Plan{0, bt, S, 0, t};
    }
  }
  for (int bn = 256; bn >= 128; bn -= 32) {
    const double rounds = std::ceil((double)(((Q + TM - 1) / TM) * ((P + bn - 1) / bn)) / (sms / 2.0));
    const double prod = nkb * (std::max(0.235, 0.345 * bn / 256) + (pmn && bn / 2 % 64 ? 0.05 : 0.0));
    const double epi = 0.3 + 1.55 * bn / 256;
    const double t = 4.5 + rounds * (std::max(prod, epi) + 0.2 * std::min(prod, epi));
    if (t < tb) tb = t, best = Plan{1, 0, 0, bn, t};
  }
  return best;
}

// Maps and parameters of the split form's tiles, for a plan
static lsq_status split_args(Maps* maps, Params* p, const void* pop, int pmn, const void* qop, int qmn, int64_t P,
                             int64_t Q, int64_t C, int bt, int splits, const Epi& e) {
  memset(maps, 0, sizeof(*maps));
  *p = Params{};
  p->P = (int)P;
  p->Q = (int)Q;
  p->nkb = kblocks(C);
  p->tp = (int)((P + BP - 1) / BP);
  p->e = e;
  p->splits = splits;
  p->lper = (bt == 16 ? 4 : bt == 32 ? 5 : bt == 64 ? 6 : 7) - (splits == 1 ? 0 : splits == 2 ? 1 : splits == 4 ? 2 : 3);
  lsq_status st = map_operand(&maps->p, pop, pmn, P, C, BP);
  if (st == LSQ_OK) st = map_operand(&maps->q, qop, qmn, Q, C, bt);
  return st;
}

// out[Q, P] = sum over C of the operands (see the top), with the epilogue e
template <int PMN, int QMN>
static lsq_status product(const Plan& plan, const void* pop, const void* qop, int64_t P, int64_t Q, int64_t C,
                          const Epi& e, cudaStream_t stream) {
  Params p{};
  lsq_status st;
  if (plan.pair) {
    p.P = (int)P;
    p.Q = (int)Q;
    p.nkb = kblocks(C);
    p.e = e;
    p.bn = plan.bn;
    GMaps gm;
    memset(&gm, 0, sizeof(gm));
    st = map_operand(&gm.a, qop, QMN, Q, C, TM / 2);
    if (st == LSQ_OK) st = map_operand(&gm.b, pop, PMN, P, C, p.bn / 2);
    if (st == LSQ_OK)
      st = e.f32 ? encode_tmap_2d(&gm.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, e.out, P, Q, P * 4, 32, 32,
                                  CU_TENSOR_MAP_SWIZZLE_128B)
                 : encode_tmap_2d(&gm.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, e.out, P, Q, P * 2, 32, 32,
                                  CU_TENSOR_MAP_SWIZZLE_64B);
    if (st == LSQ_OK && e.z)
      st = encode_tmap_2d(&gm.z, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, e.z, P, Q, P * 2, 32, 32,
                          CU_TENSOR_MAP_SWIZZLE_64B);
    if (st != LSQ_OK) return st;
    const int64_t tiles = ((Q + TM - 1) / TM) * ((P + p.bn - 1) / p.bn);
    if constexpr (QMN)
      if (e.f32) return launch_pair<QMN, PMN, 1>(gm, p, tiles, stream);
    return launch_pair<QMN, PMN, 0>(gm, p, tiles, stream);
  }
  const int bt = plan.bt;
  Maps maps;
  if ((st = split_args(&maps, &p, pop, PMN, qop, QMN, P, Q, C, bt, plan.splits, e)) != LSQ_OK) return st;
  const int64_t tiles = (int64_t)p.tp * ((Q + bt - 1) / bt);
  if constexpr (!QMN) {
    if (bt == 16) return launch_split<PMN, QMN, 16>(maps, p, tiles, stream);
    if (bt == 32) return launch_split<PMN, QMN, 32>(maps, p, tiles, stream);
  }
  if (bt == 64) return launch_split<PMN, QMN, 64>(maps, p, tiles, stream);
  return launch_split<PMN, QMN, 128>(maps, p, tiles, stream);
}

// dx [M, K] and dW [N, K] in one launch where both fit one round of the split form side by side and that is
// estimated shorter than one after the other (the two products together and apart, graph replays: 130 x 576 x 1536
// 6.7 us for 8.5, 256 x 1024 x 1024 7.1 for 9.6, 1000 x 1000 x 1000 13.5 for 19.1; a launch less on the host, 2.7).
// Each keeps the contraction splits that its own launch would have, so the bits do not depend on what else is
// asked for, and a cluster of the larger split may hold several tiles of the other product.
struct BothPlan {
  int bx, bw, cluster;  // bx 0: separate launches
  int nx, nw;           // blocks of each, whole clusters
};
static BothPlan plan_both(int64_t M, int64_t N, int64_t K, const Plan& px, const Plan& pw) {
  const int sx = px.pair ? 1 : px.splits, sw = pw.pair ? 1 : pw.splits, c = std::max(sx, sw), sms = num_sms();
  const int64_t tp = (K + BP - 1) / BP;
  BothPlan best{};
  double tb = px.us + pw.us;
  for (int bx = 16; bx <= 128; bx *= 2)
    for (int bw = 64; bw <= 128; bw *= 2) {
      const int64_t nx = (tp * ((M + bx - 1) / bx) * sx + c - 1) / c * c;
      const int64_t nw = (tp * ((N + bw - 1) / bw) * sw + c - 1) / c * c;
      if ((double)(nx + nw) > split_fit(c, sms)) continue;
      const double t = std::max(split_us(bx, kblocks(N), sx), split_us(bw, kblocks(M), sw));
      if (t < tb) tb = t, best = BothPlan{bx, bw, c, (int)nx, (int)nw};
    }
  return best;
}
template <int BX, int BW>
static lsq_status launch_both(const Both& b, const BothPlan& plan, cudaStream_t stream) {
  static int configured[64] = {0};
  constexpr int bytes = Cfg<BX>::BYTES > Cfg<BW>::BYTES ? Cfg<BX>::BYTES : Cfg<BW>::BYTES;
  int dev = 0;
  LSQ_CUDA_TRY(cudaGetDevice(&dev));
  if (dev >= 0 && dev < 64 && !configured[dev]) {
    LSQ_CUDA_TRY(cudaFuncSetAttribute(linear_both_kernel<BX, BW>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    configured[dev] = 1;
  }
  return launch_chained("linear_both_kernel", linear_both_kernel<BX, BW>, dim3((unsigned)(plan.nx + plan.nw)), NTHREADS,
                        bytes, (unsigned)plan.cluster, stream, b);
}
static lsq_status both(const BothPlan& plan, const Plan& px, const Plan& pw, const void* dz, const void* x,
                       const void* w, int64_t M, int64_t N, int64_t K, const Epi& ex, const Epi& ew,
                       cudaStream_t stream) {
  Both b;
  b.nx = plan.nx;
  lsq_status st = split_args(&b.mx, &b.x, w, 1, dz, 0, K, M, N, plan.bx, px.pair ? 1 : px.splits, ex);
  if (st == LSQ_OK) st = split_args(&b.mw, &b.w, x, 1, dz, 1, K, N, M, plan.bw, pw.pair ? 1 : pw.splits, ew);
  if (st != LSQ_OK) return st;
  if (plan.bw == 64) {
    if (plan.bx == 16) return launch_both<16, 64>(b, plan, stream);
    if (plan.bx == 32) return launch_both<32, 64>(b, plan, stream);
    if (plan.bx == 64) return launch_both<64, 64>(b, plan, stream);
    return launch_both<128, 64>(b, plan, stream);
  }
  if (plan.bx == 16) return launch_both<16, 128>(b, plan, stream);
  if (plan.bx == 32) return launch_both<32, 128>(b, plan, stream);
  if (plan.bx == 64) return launch_both<64, 128>(b, plan, stream);
  return launch_both<128, 128>(b, plan, stream);
}

// ---------------------------------------------------------------- dz and db
// dz = dy act'(z) (bf16: the products' operand type) and, from the fp32 dz, the sums over a strip of rows;
// a warp covers 256 columns of a row (16 bytes a lane), a block's eight warps take rows in turn.  Where at most
// eight strips fill the GPU or the rows are few, a cluster holds a column block's strips (cs) and its first block
// adds them in order into dbias; else each strip leaves a row of part for col_sum_kernel.
template <int ACT>
__global__ void __launch_bounds__(256, 4) dz_kernel(const uint4* dy, const uint4* z, uint4* dz, float* part,
                                                    int64_t rows, int n8, int64_t strip, int strips, int cs,
                                                    float* dbias, int accumulate) {
  __shared__ float comb[8][32][9];
  __shared__ float4 own[64];
  grid_release();
  grid_wait();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int at = (int)blockIdx.x % strips, c = ((int)blockIdx.x / strips) * 32 + l;
  const int64_t r0 = at * strip, r1 = r0 + strip < rows ? r0 + strip : rows;
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
  if (c < n8) {
    // rows in flight, loaded before any of them is stored (the compiler may not move a load over a store that could
    // be to the same place): with 2 / 4 rows 8192 x 5120 takes 47.6 / 45.9 us with GELU, 43.5 / 45.6 with ReLU, and
    // 2048 x 14336 35.0 / 34.3 and 29.9 / 30.2; without an activation, where nothing is stored, 25.3 / 17.6
    constexpr int U = ACT == LSQ_ACT_RELU ? 2 : 4;
    for (int64_t r = r0 + w; r < r1; r += 8 * U) {
      uint4 dv[U], zw[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (r + 8 * i >= r1) break;
        dv[i] = dy[(r + 8 * i) * n8 + c];
        if (ACT != LSQ_ACT_NONE) zw[i] = z[(r + 8 * i) * n8 + c];
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (r + 8 * i >= r1) break;
        uint64_t d[4];
        nrm::unpack_pairs(dv[i], d);
        if (ACT != LSQ_ACT_NONE) {
          uint64_t zv[4];
          nrm::unpack_pairs(zw[i], zv);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = mul2(d[j], dact2<ACT>(zv[j]));
          dz[(r + 8 * i) * n8 + c] = nrm::pack_pairs(d);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = add2(acc[j], d[j]);
      }
    }
  }
  float s[8];
  nrm::split8(acc, s);
  if (!dbias) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) comb[w][l][j] = s[j];
  __syncthreads();
  if (w == 0) {
#pragma unroll
    for (int k = 1; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += comb[k][l][j];
    float4* o = cs ? own + l * 2 : reinterpret_cast<float4*>(part + ((int64_t)at * n8 + c) * 8);
    if (cs || c < n8) {
      o[0] = make_float4(s[0], s[1], s[2], s[3]);
      o[1] = make_float4(s[4], s[5], s[6], s[7]);
    }
  }
  if (!cs) return;
  if (cs > 1) nf4g::cluster_sync_all();
  else __syncthreads();
  const int word = (int)threadIdx.x >> 1;  // 64 threads of the cluster's first block, four columns each
  if (at == 0 && threadIdx.x < 64 && ((int)blockIdx.x / strips) * 32 + word < n8) {
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = 0; k < cs; ++k) {
      const float4 v = nf4g::ldn::ld_dsmem_f4(nf4g::cluster_addr(own + threadIdx.x, (uint32_t)k));
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    float4* o = reinterpret_cast<float4*>(dbias) + ((int64_t)((int)blockIdx.x / strips) * 64 + threadIdx.x);
    if (accumulate) {
      const float4 v = *o;
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    *o = t;
  }
  if (cs > 1) nf4g::cluster_sync_all();  // the sums stay until the first block has read them
}

// row strips of dz_kernel: one round of its blocks (four per SM), at least 8 rows each; at most eight, joined in a
// cluster, where they fill that round or a warp's rows take no longer than the second kernel: 4 with an activation
// (256 x 576, GELU: 4.1 us joined, 4.1 in two kernels; 333 x 1536 5.0 and 4.8; 512 x 1024 5.7 and 4.4; 2048 x 14336,
// 448 of 592 blocks, 38.7 and 34.3), 16 without (512 x 1024 3.2 and 3.8, 1024 x 4096 4.5 and 4.5, 2048 x 4096 6.3 and
// 5.4); the host saves 2.3 us
struct Strips {
  int64_t rows;
  int n, joined;
  int64_t most;  // the rows of partial sums that the workspace has: no fewer for more rows, as n may be
};
static Strips strips_of(int64_t M, int64_t N, int act) {
  const int64_t cb = (N + 255) / 256, slots = 4 * num_sms();
  const bool join = 8 * cb >= slots || M <= (act == LSQ_ACT_NONE ? 1024 : 256);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(slots / cb, join ? 8 : slots));
  Strips s;
  s.rows = std::max<int64_t>(8, (M + want - 1) / want);
  s.n = (int)((M + s.rows - 1) / s.rows);
  s.joined = s.n <= 8;
  s.most = std::min<int64_t>((M + 7) / 8, want);
  return s;
}
static size_t round256(size_t b) { return (b + 255) / 256 * 256; }

static lsq_status check_shape(const char* who, int64_t M, int64_t N, int64_t K, int32_t act) {
  if (M < 1 || M > (1 << 30)) return fail(LSQ_EINVAL, "%s: M out of range (%lld)", who, (long long)M);
  if (N < 8 || N % 8 != 0 || N > (1 << 30) || K < 8 || K % 8 != 0 || K > (1 << 30))
    return fail(LSQ_EINVAL, "%s: N and K must be positive multiples of 8 (got %lld, %lld)", who, (long long)N,
                (long long)K);
  if (((M + 15) / 16) * ((N + 127) / 128) > (1ll << 27) || ((N + 63) / 64) * ((K + 127) / 128) > (1ll << 27) ||
      ((M + 15) / 16) * ((K + 127) / 128) > (1ll << 27))
    return fail(LSQ_EINVAL, "%s: too many output tiles", who);
  if (act < LSQ_ACT_NONE || act > LSQ_ACT_SILU) return fail(LSQ_EINVAL, "%s: unknown activation %d", who, (int)act);
  return LSQ_OK;
}

}  // namespace lin
}  // namespace lsq

using namespace lsq;

extern "C" lsq_status lsq_linear_fwd(const void* x, const void* w, const void* bias, int32_t act, const void* residual,
                                     void* z, void* y, int64_t M, int64_t N, int64_t K, lsq_cuda_stream stream) {
  const char* who = "lsq_linear_fwd";
  if (!x || !w || !y) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = lin::check_shape(who, M, N, K, act);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, w, bias, residual, z, y)) return fail(LSQ_EINVAL, "%s: alignment", who);
  const size_t mn = (size_t)M * N * 2, mk = (size_t)M * K * 2, nk = (size_t)N * K * 2, n1 = (size_t)N * 2;
  for (const void* o : {(const void*)y, (const void*)z})
    if (overlap(o, mn, x, mk) || overlap(o, mn, w, nk) || overlap(o, mn, bias, n1))
      return fail(LSQ_EINVAL, "%s: an output overlaps x, w or bias", who);
  if (overlap(z, mn, y, mn) || overlap(z, mn, residual, mn) || nrm::shifted(residual, y, mn))
    return fail(LSQ_EINVAL, "%s: z, y and residual overlap (residual may be y itself)", who);
  if ((st = check_device()) != LSQ_OK) return st;
  lin::Epi e{};
  e.bias = static_cast<const __nv_bfloat16*>(bias);
  e.residual = static_cast<const __nv_bfloat16*>(residual);
  e.z = static_cast<__nv_bfloat16*>(z);
  e.out = y;
  e.act = act;
  if (M == 1) {
    const lin::OneRow p{(const uint4*)x, (const uint4*)w, (int)N, (int)(K / 8), e};
    return launch_chained("linear_row_kernel", lin::linear_row_kernel, dim3((unsigned)(N / 8)), 256, 0, 1,
                          (cudaStream_t)stream, p);
  }
  return lin::product<0, 0>(lin::plan_product(N, M, lin::kblocks(K), 0, 0), w, x, N, M, K, e, (cudaStream_t)stream);
}

extern "C" size_t lsq_linear_bwd_workspace_size(int64_t M, int64_t N, int64_t K, int32_t act) {
  if (M < 1 || N < 8 || K < 8) return 256;
  return (act == LSQ_ACT_NONE ? 0 : lin::round256((size_t)M * (size_t)N * 2)) +
         lin::round256((size_t)lin::strips_of(M, N, act).most * (size_t)N * sizeof(float));
}

extern "C" lsq_status lsq_linear_bwd(const void* dy, const void* x, const void* w, const void* z, int32_t act, void* dx,
                                     void* dw, int32_t dw_f32, float* dbias, int32_t accumulate, int64_t M, int64_t N,
                                     int64_t K, void* workspace, size_t workspace_bytes, lsq_cuda_stream stream) {
  const char* who = "lsq_linear_bwd";
  if (!dy || (dx && !w) || (dw && !x) || (act != LSQ_ACT_NONE && !z))
    return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = lin::check_shape(who, M, N, K, act);
  if (st != LSQ_OK) return st;
  if (!dx && !dw && !dbias) return fail(LSQ_EINVAL, "%s: no gradient asked for", who);
  if (accumulate && dw && !dw_f32)
    return fail(LSQ_EINVAL, "%s: a gradient that accumulates is fp32 (dw_f32 = 1)", who);
  if (!nrm::aligned16(dy, x, w, z, dx, dw, dbias)) return fail(LSQ_EINVAL, "%s: alignment", who);
  const bool pass = act != LSQ_ACT_NONE || dbias;
  if (pass && (!workspace || !aligned(workspace, 256) ||
               workspace_bytes < lsq_linear_bwd_workspace_size(M, N, K, act)))
    return fail(LSQ_EINVAL, "%s: workspace missing, misaligned or too small", who);
  const size_t mn = (size_t)M * N * 2, mk = (size_t)M * K * 2, nk = (size_t)N * K * 2;
  const nrm::Range in[] = {
      {dy, mn}, {dw ? x : nullptr, mk}, {dx ? w : nullptr, nk}, {act != LSQ_ACT_NONE ? z : nullptr, mn}};
  const nrm::Range out[] = {{dx, mk}, {dw, dw_f32 ? 2 * nk : nk}, {dbias, (size_t)N * 4},
                            {pass ? workspace : nullptr, lsq_linear_bwd_workspace_size(M, N, K, act)}};
  if (nrm::clash(out, in)) return fail(LSQ_EINVAL, "%s: overlapping arguments", who);
  if ((st = check_device()) != LSQ_OK) return st;
  if (pass && workspace_bytes < lsq_linear_bwd_workspace_size(M, N, K, act))  // now that the device's SMs are known
    return fail(LSQ_EINVAL, "%s: workspace too small for this device", who);
  cudaStream_t s = (cudaStream_t)stream;
  const void* dz = dy;
  if (pass) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (act != LSQ_ACT_NONE) {
      dz = ws;
      ws += lin::round256((size_t)M * (size_t)N * 2);
    }
    float* part = reinterpret_cast<float*>(ws);
    const lin::Strips sp = lin::strips_of(M, N, act);
    const int64_t blocks = (N + 255) / 256 * sp.n;
    const int n8 = (int)(N / 8), cs = sp.joined ? sp.n : 0;
    auto k = act == LSQ_ACT_RELU        ? lin::dz_kernel<LSQ_ACT_RELU>
             : act == LSQ_ACT_GELU      ? lin::dz_kernel<LSQ_ACT_GELU>
             : act == LSQ_ACT_GELU_TANH ? lin::dz_kernel<LSQ_ACT_GELU_TANH>
             : act == LSQ_ACT_SILU      ? lin::dz_kernel<LSQ_ACT_SILU>
                                        : lin::dz_kernel<LSQ_ACT_NONE>;
    st = launch_chained("dz_kernel", k, dim3((unsigned)blocks), 256, 0, cs > 1 ? (unsigned)cs : 1u, s, (const uint4*)dy,
                        (const uint4*)z, act == LSQ_ACT_NONE ? (uint4*)nullptr : (uint4*)const_cast<void*>(dz), part, M,
                        n8, sp.rows, sp.n, cs, dbias, accumulate ? 1 : 0);
    if (st != LSQ_OK) return st;
    if (dbias && !cs && (st = nrm::col_sum(part, sp.n, N, N, N, dbias, nullptr, accumulate ? 1 : 0, s)) != LSQ_OK)
      return st;
  }
  lin::Epi ex{}, ew{};
  ex.out = dx;
  ew.out = dw;
  ew.f32 = dw_f32 ? 1 : 0;
  ew.accumulate = accumulate ? 1 : 0;
  const lin::Plan px = dx ? lin::plan_product(K, M, lin::kblocks(N), 1, 0) : lin::Plan{};
  const lin::Plan pw = dw ? lin::plan_product(K, N, lin::kblocks(M), 1, 1) : lin::Plan{};
  if (dx && dw) {
    const lin::BothPlan plan = lin::plan_both(M, N, K, px, pw);
    if (plan.bx) return lin::both(plan, px, pw, dz, x, w, M, N, K, ex, ew, s);
  }
  if (dx && (st = lin::product<1, 0>(px, w, dz, K, M, N, ex, s)) != LSQ_OK) return st;
  return dw ? lin::product<1, 1>(pw, x, dz, K, N, M, ew, s) : LSQ_OK;
}
