// LayerNorm (forward, backward, gradients of gain and bias) and the 8-bit
// activation checkpoint with the RMSNorm passes that write and read it.
//
// All are HBM-bound row passes over bf16 [rows, d].  A row belongs to one warp
// (WARP, d <= 1024; d <= 768 in the LayerNorm backward's rings) or to one
// block; each thread holds V 16-byte words of it from the one load to the last
// use, so every input is read once from HBM (the LayerNorm backward of few
// rows reads x and dy a second time, from L2, for its column sums; the rings
// a second time from shared memory).  Word c of a row belongs to thread c % T
// (T threads per row, a multiple of 32), so eight neighbouring lanes hold one
// 64-column block of the checkpoint.
//
// Measured on B200 in graph replays over three sets of buffers, 8192 x 5120
// (a copy of the same tensor runs at 6.1 TB/s): LayerNorm forward 31.9 us
// (5.3 TB/s: its two dependent reductions a row), backward with frozen gain
// 53.1 (6.3 TB/s), with dg and db 61.4 (the 12 MB of partial sums and their
// second kernel), checkpoint alone 21.2 (6.0), restored alone 20.5 (6.2), norm
// and checkpoint 35.4 (6.0), restore and norm 34.7 (6.1), backward from the
// checkpoint 51.4 (5.7).  2048 x 4096: 8.2, 15.9, 21.6, 4.8, 4.0, 9.4, 8.4,
// 11.8 us.  One row of 4096: 1.6 us, launch and latency.
#include <algorithm>

#include "common.cuh"
#include "host_common.h"

namespace lsq {
namespace nrm {

using ops::pack8;
using ops::unpack8;

constexpr int64_t MAX_D = 16384;  // 2048 words: 512 threads x 4, or 1024 x 2
enum { NONE = 0, RMS = 1, LAYER = 2 };
enum { BF16 = 0, CKPT8 = 1 };

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// sum over the threads of a row, fixed tree, in every thread; a block row needs red[32] and one barrier
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (WARP) return v;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (l == 0) red[w] = v;
  __syncthreads();
  return warp_sum(l < (int)(blockDim.x >> 5) ? red[l] : 0.0f);
}

// eight values as four f32x2 pairs
__device__ __forceinline__ void unpack_pairs(uint4 v, uint64_t (&f)[4]) {
  f[0] = f2(bf16lo(v.x), bf16hi(v.x));
  f[1] = f2(bf16lo(v.y), bf16hi(v.y));
  f[2] = f2(bf16lo(v.z), bf16hi(v.z));
  f[3] = f2(bf16lo(v.w), bf16hi(v.w));
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0]), pack_bf16x2(f[1]), pack_bf16x2(f[2]), pack_bf16x2(f[3]));
}
__device__ __forceinline__ float pair_sum(uint64_t v) {
  const float2 f = f2split(v);
  return f.x + f.y;
}

// ---------------------------------------------------------------- 8-bit checkpoint
// A block of 64 columns keeps amax = max |x| (a bf16, exact) and q = round(127 x / amax), halves away
// from zero; it stands for bf16(q amax / 127).  Both are exact in fp32 arithmetic:
//  * code: 127 |x| / amax is either a half-integer or at least 1.5e-5 (relative) away from one (x and
//    amax have 8-bit significands), so the product with 127 (1 + 2^-17) / amax, off by the factor
//    1 + 7.6e-6 and one fp32 rounding of that reciprocal (1.2e-7), lies on the side of the half that
//    its tie goes to, and the fused multiply-add with 1.5 * 2^23 rounds it to the integer, whose two's
//    complement is the low byte of the sum.
//  * value: q amax / 127 is a bf16 or a distance of 1e-5 from any midpoint of two, so the two fp32
//    roundings of q * (amax * (1/127)) (1.8e-7) do not change its rounding to bf16.
constexpr float CODE_GAIN = 127.0f * (1.0f + 1.0f / 131072.0f);
constexpr float INV_127 = 1.0f / 127.0f;
constexpr float CODE_MAGIC = 12582912.0f;  // 1.5 * 2^23

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// the block's amax bits from this lane's word: max over the word, then over the eight lanes of the block
// (bf16 magnitudes order as integers, infinity and NaN above every finite value)
__device__ __forceinline__ uint32_t block_amax(uint4 w) {
  const uint32_t k = 0x7fff7fffu;
  uint32_t m = max_u16x2(max_u16x2(w.x & k, w.y & k), max_u16x2(w.z & k, w.w & k));
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m >= 0x7f80u) return 0x7fc0u;   // a block with an infinity or a NaN is restored as NaN
  return m < 0x0480u ? 0u : m;        // below 2^-118: zeros (127 / amax would overflow)
}
__device__ __forceinline__ uint2 encode8(uint4 w, uint32_t amax) {
  if (amax == 0u || amax == 0x7fc0u) return make_uint2(0u, 0u);
  const float inv = CODE_GAIN / __uint_as_float(amax << 16);
  uint64_t f[4];
  unpack_pairs(w, f);
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = fma2(f[i], f2(inv, inv), f2(CODE_MAGIC, CODE_MAGIC));
    u[2 * i] = (uint32_t)v;
    u[2 * i + 1] = (uint32_t)(v >> 32);
  }
  return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
}
__device__ __forceinline__ uint4 decode8(uint2 codes, uint32_t amax) {
  const float s = __uint_as_float(amax << 16) * INV_127;
  uint64_t f[4];
  const uint32_t a = codes.x ^ 0x80808080u, b = codes.y ^ 0x80808080u;  // q + 128, unsigned
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 2^23 + q + 128 as a float, two a step
    const uint32_t c = i < 2 ? a : b, at = 0x7440 + 2 * (i & 1);
    const uint64_t v = (uint64_t)__byte_perm(c, 0x4b000000u, at) | (uint64_t)__byte_perm(c, 0x4b000000u, at + 1) << 32;
    f[i] = mul2(add2(v, f2(-8388736.0f, -8388736.0f)), f2(s, s));
  }
  return pack_pairs(f);
}

struct Ckpt {
  uint8_t* codes;   // int8 [rows][d]
  uint16_t* amax;   // bf16 [rows][ceil(d / 64)]
};
static size_t ckpt_amax_off(int64_t rows, int64_t d) { return (size_t)(rows * d + 15) / 16 * 16; }
static size_t ckpt_used(int64_t rows, int64_t d) {
  return ckpt_amax_off(rows, d) + (size_t)rows * (size_t)((d + 63) / 64) * 2;
}
static Ckpt ckpt_of(const void* p, int64_t rows, int64_t d) {
  uint8_t* b = static_cast<uint8_t*>(const_cast<void*>(p));
  return Ckpt{b, reinterpret_cast<uint16_t*>(b + ckpt_amax_off(rows, d))};
}

// ---------------------------------------------------------------- row passes, forward
struct Fwd {
  const uint4* x;         // BF16 source
  Ckpt in;                // CKPT8 source
  Ckpt out;               // PACK
  const uint4 *g, *b;     // gain, bias (b may be null)
  uint4 *xo, *y;          // restored x (CKPT8), normalised row (NORM)
  float *mean, *rstd;     // may be null
  int64_t rows;
  int d8, nb;
  float inv_d, eps;
};

// AHEAD: gain and bias are under way with x, not behind the row's sums
template <int V, bool WARP, int SRC, int NORM, bool PACK, bool AHEAD>
__global__ void __launch_bounds__(WARP ? 256 : V == 4 ? 512 : 1024) row_fwd_kernel(const __grid_constant__ Fwd p) {
  __shared__ float red[2][32];
  const int T = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  grid_release();
  grid_wait();
  if (WARP && row >= p.rows) return;  // whole warps; no block barrier follows
  const int d8 = p.d8;
  const int64_t base = row * d8, bbase = row * p.nb;
  uint4 xv[V];
  if (SRC == BF16) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      xv[i] = c < d8 ? p.x[base + c] : make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    uint2 cv[V];
    uint32_t av[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      const bool in = c < d8;
      cv[i] = in ? reinterpret_cast<const uint2*>(p.in.codes)[base + c] : make_uint2(0u, 0u);
      av[i] = in ? p.in.amax[bbase + (c >> 3)] : 0u;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      xv[i] = decode8(cv[i], av[i]);
      if (c < d8) p.xo[base + c] = xv[i];
    }
  }
  uint4 gv[AHEAD ? V : 1], bv[AHEAD && NORM == LAYER ? V : 1];
  auto gain = [&](int c) { return c < d8 ? p.g[c] : make_uint4(0u, 0u, 0u, 0u); };
  auto bias = [&](int c) { return c < d8 && p.b ? p.b[c] : make_uint4(0u, 0u, 0u, 0u); };
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      gv[i] = gain(t + i * T);
      if constexpr (NORM == LAYER) bv[i] = bias(t + i * T);
    }
  }
  if (PACK) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      const uint32_t am = block_amax(xv[i]);
      if (c < d8) {
        reinterpret_cast<uint2*>(p.out.codes)[base + c] = encode8(xv[i], am);
        if ((c & 7) == 0) p.out.amax[bbase + (c >> 3)] = (uint16_t)am;
      }
    }
  }
  if constexpr (NORM == LAYER) {  // the mean first, then the centred squares: no cancellation
    uint64_t f[V][4], acc = 0ull;  // the row in fp32 pairs: scalar, 8192 x 5120 took 34.2 us, not 32.2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      unpack_pairs(xv[i], f[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = add2(acc, f[i][j]);
    }
    const float mu = row_sum<WARP>(pair_sum(acc), red[0]) * p.inv_d;
    const uint64_t nmu = f2(-mu, -mu);
    acc = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (t + i * T >= d8) break;  // the padding is not centred
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[i][j] = add2(f[i][j], nmu);
        acc = fma2(f[i][j], f[i][j], acc);
      }
    }
    const float rs = 1.0f / sqrtf(row_sum<WARP>(pair_sum(acc), red[1]) * p.inv_d + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = rs;
    }
    const uint64_t rs2 = f2(rs, rs);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c >= d8) break;
      uint64_t g[4], b[4];
      unpack_pairs(AHEAD ? gv[AHEAD ? i : 0] : gain(c), g);
      unpack_pairs(AHEAD ? bv[AHEAD ? i : 0] : bias(c), b);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[i][j] = fma2(mul2(f[i][j], rs2), g[j], b[j]);
      p.y[base + c] = pack_pairs(f[i]);
    }
  }
  if constexpr (NORM == RMS) {
    uint64_t acc = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint64_t f[4];
      unpack_pairs(xv[i], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = fma2(f[j], f[j], acc);
    }
    const float rs = 1.0f / sqrtf(row_sum<WARP>(pair_sum(acc), red[0]) * p.inv_d + p.eps);
    if (t == 0 && p.rstd) p.rstd[row] = rs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c >= d8) break;
      uint64_t f[4], g[4];
      unpack_pairs(xv[i], f);
      unpack_pairs(AHEAD ? gv[AHEAD ? i : 0] : gain(c), g);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = mul2(mul2(f[j], f2(rs, rs)), g[j]);
      p.y[base + c] = pack_pairs(f);
    }
  }
}

// ---------------------------------------------------------------- row passes, backward
struct Bwd {
  const uint4 *dy, *x, *g;
  Ckpt in;
  const float *mean, *rstd;
  const uint4* res;   // dres_in or null; may alias out
  uint4* out;
  float* part;        // [gridDim.x][2][d]: the blocks' sums of dy xhat and dy (GRADS)
  float *dg, *db;     // few rows: written in the one kernel
  int64_t rows;
  int d8, nb, accumulate;
  float inv_d;
};

// RMSNorm from a checkpoint: out = res + rs (dy g) - x rs^3 mean(dy g x), one row per warp or block
template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : V == 4 ? 512 : 1024)
    rms_bwd_unpack8_kernel(const __grid_constant__ Bwd p) {
  __shared__ float red[32];
  const int T = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  grid_release();
  grid_wait();
  if (WARP && row >= p.rows) return;
  const int d8 = p.d8;
  const int64_t base = row * d8, bbase = row * p.nb;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  uint2 cv[V];
  uint32_t av[V];
  uint4 dv[V], gv[V], rv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    const bool in = c < d8;
    cv[i] = in ? reinterpret_cast<const uint2*>(p.in.codes)[base + c] : make_uint2(0u, 0u);
    av[i] = in ? p.in.amax[bbase + (c >> 3)] : 0u;
    dv[i] = in ? p.dy[base + c] : z;
    gv[i] = in ? p.g[c] : z;
    rv[i] = (in && p.res) ? p.res[base + c] : z;
  }
  const float rs = p.rstd[row];
  uint64_t f[V][4], a[V][4], acc = 0ull;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    uint64_t g[4];
    unpack_pairs(decode8(cv[i], av[i]), f[i]);
    unpack_pairs(dv[i], a[i]);
    unpack_pairs(gv[i], g);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[i][j] = mul2(a[i][j], g[j]);
      acc = fma2(a[i][j], f[i][j], acc);
    }
  }
  const float k = -rs * rs * rs * row_sum<WARP>(pair_sum(acc), red) * p.inv_d;
  const uint64_t rs2 = f2(rs, rs), k2 = f2(k, k);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (c >= d8) break;
    uint64_t o[4];
    unpack_pairs(rv[i], o);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = fma2(f[i][j], k2, fma2(a[i][j], rs2, o[j]));
    p.out[base + c] = pack_pairs(o);
  }
}

// LayerNorm: out = res + rs (a - mean(a) - xh mean(a xh)), a = dy g, xh = (x - mean) rs.  Warps (d <= 768)
// or blocks walk the rows in strides and a thread's columns stay the same, so the sums over rows of dy xh
// and dy (dg, db) collect in registers and leave once per block; col_sum_kernel adds the blocks in order.  Few
// rows have a kernel of their own.  The arithmetic runs on pairs (f32x2): scalar, its 30 operations an element took
// as long as the loads.

// one word of the first pass: xh and a, their row sums, and the column sums of dy xh and dy
template <bool GRADS>
__device__ __forceinline__ void ln_bwd_word(uint4 x, uint4 dy, uint4 g, uint64_t nmu, uint64_t rs, uint64_t (&xh)[4],
                                            uint64_t (&a)[4], uint64_t& s1, uint64_t& s2, uint64_t* sg, uint64_t* sb) {
  uint64_t d[4];
  unpack_pairs(x, xh);
  unpack_pairs(dy, d);
  unpack_pairs(g, a);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    xh[j] = mul2(add2(xh[j], nmu), rs);
    a[j] = mul2(d[j], a[j]);
    s1 = add2(s1, a[j]);
    s2 = fma2(a[j], xh[j], s2);
    if (GRADS) {
      sg[j] = fma2(d[j], xh[j], sg[j]);
      sb[j] = add2(sb[j], d[j]);
    }
  }
}
// and of the second: res + rs a - rs m1 - xh rs m2
__device__ __forceinline__ uint4 ln_bwd_out(const uint64_t (&xh)[4], const uint64_t (&a)[4], uint4 res, uint64_t rs,
                                            uint64_t nk1, uint64_t nk2) {
  uint64_t o[4];
  unpack_pairs(res, o);
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = fma2(xh[j], nk2, add2(fma2(a[j], rs, o[j]), nk1));
  return pack_pairs(o);
}
// eight column sums of word c, to row r of the partial sums
__device__ __forceinline__ void ln_put_sums(const Bwd& p, int r, int h, int c, const float (&v)[8]) {
  float4* o = reinterpret_cast<float4*>(p.part + ((int64_t)r * 2 + h) * (p.d8 * 8) + c * 8);
  o[0] = make_float4(v[0], v[1], v[2], v[3]);
  o[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void split8(const uint64_t* s, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = f2split(s[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// The rows of x, dy and the residual gradient come through rings of shared-memory stages filled by bulk
// copies, one ring per row walker (a warp or a block), so that the bytes in flight do not depend on the
// registers, which the sums take: with the loads in registers 8192 x 5120 took 103 us and 16384 x 576 34.
__device__ __forceinline__ void ln_fetch(const Bwd& p, uint8_t* b, uint64_t* bar, uint32_t rb, int64_t row) {
  mbar_arrive_expect_tx(bar, rb * (p.res ? 3u : 2u));
  bulk_g2s(b, p.x + row * p.d8, rb, bar);
  bulk_g2s(b + rb, p.dy + row * p.d8, rb, bar);
  if (p.res) bulk_g2s(b + 2 * rb, p.res + row * p.d8, rb, bar);
}

// a row per warp, V words a lane
constexpr int LNW = 8;
template <int V, bool GRADS>
__global__ void __launch_bounds__(LNW * 32, 2) ln_bwd_warp_kernel(const __grid_constant__ Bwd p, int nst, int stage) {
  extern __shared__ __align__(128) uint8_t smem[];  // per warp [nst][x | dy | res], then every stage's barrier
  __shared__ float comb[LNW * 32 * 9];
  __shared__ int gave_up[LNW];  // stage and parity of a wait that did (in registers it costs the loop 1%)
  const int t = (int)(threadIdx.x & 31), w = (int)(threadIdx.x >> 5);
  uint8_t* ring = smem + (size_t)w * nst * stage;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)LNW * nst * stage) + w * nst;
  const int d8 = p.d8;
  const uint32_t rb = (uint32_t)d8 * 16;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  const int64_t first = (int64_t)blockIdx.x * LNW + w, step = (int64_t)gridDim.x * LNW;
  if (t == 0) {
    for (int s = 0; s < nst; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  grid_release();
  grid_wait();
  if (t == 0)
    for (int s = 0; s < nst; ++s)
      if (first + s * step < p.rows) ln_fetch(p, ring + (size_t)s * stage, &full[s], rb, first + s * step);
  __syncwarp();
  uint4 gv[V];
  uint64_t sg[GRADS ? V : 1][4], sb[GRADS ? V : 1][4];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    gv[i] = t + i * 32 < d8 ? p.g[t + i * 32] : z;
#pragma unroll
    for (int j = 0; j < 4; ++j) sg[GRADS ? i : 0][j] = sb[GRADS ? i : 0][j] = 0ull;
  }
  int s = 0;
  uint32_t ph = 0;
  bool ok = true;  // after a wait that gave up, the rest of the rows is neither fetched nor waited for
  for (int64_t row = first; row < p.rows; row += step) {
    const float mu = p.mean[row], r = p.rstd[row];
    if (ok && !(ok = mbar_wait(&full[s], ph, 461)) && t == 0) gave_up[w] = 2 * s + (int)ph;
    const uint4* b = reinterpret_cast<const uint4*>(ring + (size_t)s * stage);
    const uint64_t nmu = f2(-mu, -mu), rs = f2(r, r);
    uint64_t xh[4], a[4], s1 = 0ull, s2 = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i) {  // padded words: dy = g = 0
      const int c = t + i * 32;
      const bool in = c < d8;
      ln_bwd_word<GRADS>(in ? b[c] : z, in ? b[d8 + c] : z, gv[i], nmu, rs, xh, a, s1, s2, sg[GRADS ? i : 0],
                         sb[GRADS ? i : 0]);
    }
    const float k1 = -r * warp_sum(pair_sum(s1)) * p.inv_d, k2 = -r * warp_sum(pair_sum(s2)) * p.inv_d;
#pragma unroll
    for (int i = 0; i < V; ++i) {  // xh and a again: kept for every word they would not fit the registers
      const int c = t + i * 32;
      if (c >= d8) break;
      uint64_t u1 = 0ull, u2 = 0ull;
      ln_bwd_word<false>(b[c], b[d8 + c], gv[i], nmu, rs, xh, a, u1, u2, nullptr, nullptr);
      p.out[row * d8 + c] = ln_bwd_out(xh, a, p.res ? b[2 * d8 + c] : z, rs, f2(k1, k1), f2(k2, k2));
    }
    __syncwarp();  // the warp is done with the stage: refill it
    if (t == 0 && ok && row + nst * step < p.rows)
      ln_fetch(p, ring + (size_t)s * stage, &full[s], rb, row + nst * step);
    if (++s == nst) s = 0, ph ^= 1;
  }
  if (!ok && t == 0) mbar_drain(full, nst, gave_up[w] >> 1, (uint32_t)gave_up[w] & 1u, 462);
  if constexpr (GRADS) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the warps' sums, in warp order; row stride 9 keeps the banks apart
        float v[8];
        split8(h ? sb[GRADS ? i : 0] : sg[GRADS ? i : 0], v);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) comb[(w * 32 + t) * 9 + j] = v[j];
        __syncthreads();
        const int c = t + i * 32;
        if (w != 0 || c >= d8) continue;
        for (int k = 1; k < LNW; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += comb[(k * 32 + t) * 9 + j];
        ln_put_sums(p, (int)blockIdx.x, h, c, v);
      }
    }
  }
}

// a row per block, V words a thread.  A stage is refilled once the barrier of the following row has passed:
// every thread is then done with it.
template <int V, bool GRADS>
__global__ void __launch_bounds__(V == 4 ? 512 : 320, V == 4 ? 1 : 2)
    ln_bwd_block_kernel(const __grid_constant__ Bwd p, int nst, int stage) {
  extern __shared__ __align__(128) uint8_t ring[];  // [nst][x | dy | res], then the stages' barriers
  __shared__ float2 red[2][16];
  __shared__ int gave_up;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)nst * stage);
  const int T = (int)blockDim.x, t = (int)threadIdx.x, d8 = p.d8, nw = T >> 5, lane = t & 31;
  const uint32_t rb = (uint32_t)d8 * 16;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  const int64_t first = blockIdx.x, step = gridDim.x;
  if (t == 0) {
    for (int s = 0; s < nst; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  grid_release();
  grid_wait();
  if (t == 0)
    for (int s = 0; s < nst; ++s)
      if (first + s * step < p.rows) ln_fetch(p, ring + (size_t)s * stage, &full[s], rb, first + s * step);
  __syncthreads();
  uint64_t sg[GRADS ? V : 1][4], sb[GRADS ? V : 1][4];
  uint4 gv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    gv[i] = t + i * T < d8 ? p.g[t + i * T] : z;
#pragma unroll
    for (int j = 0; j < 4; ++j) sg[GRADS ? i : 0][j] = sb[GRADS ? i : 0][j] = 0ull;
  }
  int s = 0, flip = 0;
  uint32_t ph = 0;
  bool ok = true;  // after a wait that gave up, the rest of the rows is neither fetched nor waited for
  for (int64_t row = first; row < p.rows; row += step, flip ^= 1) {
    const float mu = p.mean[row], r = p.rstd[row];
    if (ok && !(ok = mbar_wait(&full[s], ph, 461)) && t == 0) gave_up = 2 * s + (int)ph;
    const uint4* b = reinterpret_cast<const uint4*>(ring + (size_t)s * stage);
    const uint64_t nmu = f2(-mu, -mu), rs = f2(r, r);
    uint64_t xh[4], a[4], s1 = 0ull, s2 = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      const bool in = c < d8;
      ln_bwd_word<GRADS>(in ? b[c] : z, in ? b[d8 + c] : z, gv[i], nmu, rs, xh, a, s1, s2, sg[GRADS ? i : 0],
                         sb[GRADS ? i : 0]);
    }
    // the row's two sums: warps by shuffles, then every thread adds the warps' (two buffers, one barrier a row)
    const float w1 = warp_sum(pair_sum(s1)), w2 = warp_sum(pair_sum(s2));
    if (lane == 0) red[flip][t >> 5] = make_float2(w1, w2);
    __syncthreads();
    if (t == 0 && ok && row != first) {  // the previous row's stage
      const int64_t next = row + (nst - 1) * step;
      const int prev = s == 0 ? nst - 1 : s - 1;
      if (next < p.rows) ln_fetch(p, ring + (size_t)prev * stage, &full[prev], rb, next);
    }
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < nw; ++i) {
      const float2 v = red[flip][i];
      sum.x += v.x;
      sum.y += v.y;
    }
    const float k1 = -r * sum.x * p.inv_d, k2 = -r * sum.y * p.inv_d;
#pragma unroll
    for (int i = 0; i < V; ++i) {  // xh and a again: kept for every word they would not fit the registers
      const int c = t + i * T;
      if (c >= d8) break;
      uint64_t u1 = 0ull, u2 = 0ull;
      ln_bwd_word<false>(b[c], b[d8 + c], gv[i], nmu, rs, xh, a, u1, u2, nullptr, nullptr);
      p.out[row * d8 + c] = ln_bwd_out(xh, a, p.res ? b[2 * d8 + c] : z, rs, f2(k1, k1), f2(k2, k2));
    }
    if (++s == nst) s = 0, ph ^= 1;
  }
  if (!ok && t == 0) mbar_drain(full, nst, gave_up >> 1, (uint32_t)gave_up & 1u, 462);
  if constexpr (GRADS) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c >= d8) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
        split8(h ? sb[i] : sg[i], v);
        ln_put_sums(p, (int)blockIdx.x, h, c, v);
      }
    }
  }
}

// Few rows: the statistics are inputs, so the column sums need no row reduction, and a second reading of x and dy
// (from L2) costs less than partial sums and their kernel.  One launch: the first col_blocks blocks add 8 << seg
// columns each over all rows (1 << seg lanes hold a row's words of them; the groups' sums join by shuffles, then
// the warps' in shared memory, in order), the others take a row each, or (WARP) eight.  Wide column blocks for the
// fewest rows: 10 x 16384 3.1 us, not 6.6 with 32 columns in each.
constexpr int FEW_PITCH = 17;  // sixteen sums a word, apart in the banks
template <int V, bool WARP>
__global__ void __launch_bounds__(512) ln_bwd_few_kernel(const __grid_constant__ Bwd p, int col_blocks, int seg) {
  extern __shared__ float comb[];  // [warps][1 << seg][FEW_PITCH]
  __shared__ float2 red[16];
  grid_release();
  grid_wait();
  const int w = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, nw = (int)blockDim.x >> 5, d8 = p.d8;
  if ((int)blockIdx.x < col_blocks) {
    const int wide = 1 << seg, at = lane & (wide - 1), step = nw << (5 - seg);
    const int64_t c = ((int64_t)blockIdx.x << seg) + at;
    uint64_t sg[4] = {0ull, 0ull, 0ull, 0ull}, sb[4] = {0ull, 0ull, 0ull, 0ull};
    if (c < d8) {
#pragma unroll 4
      for (int64_t r = (int)threadIdx.x >> seg; r < p.rows; r += step) {
        uint64_t x[4], d[4];
        const float mu = p.mean[r], rs = p.rstd[r];
        unpack_pairs(p.x[r * d8 + c], x);
        unpack_pairs(p.dy[r * d8 + c], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sg[j] = fma2(d[j], mul2(add2(x[j], f2(-mu, -mu)), f2(rs, rs)), sg[j]);
          sb[j] = add2(sb[j], d[j]);
        }
      }
    }
    float* mine = comb + ((w << seg) + at) * FEW_PITCH;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = f2split(j < 4 ? sg[j & 3] : sb[j & 3]);
      float a = v.x, b = v.y;
      for (int o = wide; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      if (lane < wide) {
        mine[2 * j] = a;
        mine[2 * j + 1] = b;
      }
    }
    __syncthreads();
    for (int it = (int)threadIdx.x; it < 16 << seg; it += (int)blockDim.x) {  // a column's sum: dg's, then db's
      const int h = it >> (seg + 3), k = it & ((8 << seg) - 1);
      const int64_t col = ((int64_t)blockIdx.x << (seg + 3)) + k;
      float* o = h ? p.db : p.dg;
      if (!o || col >= (int64_t)d8 * 8) continue;
      float v = 0.0f;
      for (int i = 0; i < nw; ++i) v += comb[((i << seg) + (k >> 3)) * FEW_PITCH + h * 8 + (k & 7)];
      o[col] = p.accumulate ? o[col] + v : v;
    }
    return;
  }
  const int T = WARP ? 32 : (int)blockDim.x, t = WARP ? lane : (int)threadIdx.x;
  const int64_t blk = (int64_t)blockIdx.x - col_blocks, row = WARP ? blk * nw + w : blk;
  if (WARP && row >= p.rows) return;  // whole warps; no block barrier follows
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  const int64_t base = row * d8;
  uint4 xv[V], dv[V], gv[V], rv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {  // padded words: dy = g = 0
    const int c = t + i * T;
    const bool in = c < d8;
    xv[i] = in ? p.x[base + c] : z;
    dv[i] = in ? p.dy[base + c] : z;
    gv[i] = in ? p.g[c] : z;
    rv[i] = in && p.res ? p.res[base + c] : z;
  }
  const float mu = p.mean[row], r = p.rstd[row];
  const uint64_t nmu = f2(-mu, -mu), rs = f2(r, r);
  uint64_t xh[4], a[4], s1 = 0ull, s2 = 0ull;
#pragma unroll
  for (int i = 0; i < V; ++i) ln_bwd_word<false>(xv[i], dv[i], gv[i], nmu, rs, xh, a, s1, s2, nullptr, nullptr);
  float2 sum = make_float2(warp_sum(pair_sum(s1)), warp_sum(pair_sum(s2)));
  if (!WARP) {
    if (lane == 0) red[w] = sum;
    __syncthreads();
    sum = make_float2(0.0f, 0.0f);
    for (int k = 0; k < nw; ++k) {
      sum.x += red[k].x;
      sum.y += red[k].y;
    }
  }
  const float k1 = -r * sum.x * p.inv_d, k2 = -r * sum.y * p.inv_d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (c >= d8) break;
    uint64_t u1 = 0ull, u2 = 0ull;
    ln_bwd_word<false>(xv[i], dv[i], gv[i], nmu, rs, xh, a, u1, u2, nullptr, nullptr);
    p.out[base + c] = ln_bwd_out(xh, a, rv[i], rs, f2(k1, k1), f2(k2, k2));
  }
}

// out0[c] (+)= sum over the G rows of part[.][c] for c < n0, out1[c - n0] for the columns from n0 on
// (either may be null; n0 and ncols even); part has row stride ld.  Warp w of 32 takes rows w, w + 32, ...,
// ten loads in flight (two blocks' rows on 148 SMs are one batch); then warp w adds column pair w's 32 sums.
__global__ void __launch_bounds__(1024) col_sum_kernel(const float* part, int G, int64_t ld, int64_t n0,
                                                       int64_t ncols, float* out0, float* out1, int accumulate) {
  __shared__ float2 s[32][33];
  grid_release();
  grid_wait();
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t c0 = (int64_t)blockIdx.x * 64, c = c0 + l * 2;
  float2 v = make_float2(0.0f, 0.0f);
  if (c < ncols)
    for (int r0 = w; r0 < G; r0 += 320) {
      float2 u[10];
#pragma unroll
      for (int i = 0; i < 10; ++i)
        u[i] = r0 + i * 32 < G ? *reinterpret_cast<const float2*>(part + (r0 + i * 32) * ld + c)
                               : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        v.x += u[i].x;
        v.y += u[i].y;
      }
    }
  s[w][l] = v;
  __syncthreads();
  const float2 x = s[l][w];
  float2 tot = make_float2(warp_sum(x.x), warp_sum(x.y));
  const int64_t cw = c0 + w * 2;
  if (l != 0 || cw >= ncols) return;
  float* o = cw < n0 ? (out0 ? out0 + cw : nullptr) : (out1 ? out1 + (cw - n0) : nullptr);
  if (!o) return;
  if (accumulate) {
    tot.x += o[0];
    tot.y += o[1];
  }
  o[0] = tot.x;
  o[1] = tot.y;
}

lsq_status col_sum(const float* part, int G, int64_t ld, int64_t n0, int64_t ncols, float* out0, float* out1,
                   int accumulate, cudaStream_t stream) {
  return launch_chained("col_sum_kernel", col_sum_kernel, dim3((unsigned)((ncols + 63) / 64)), 1024, 0, 1, stream, part,
                        G, ld, n0, ncols, out0, out1, accumulate);
}

// ---------------------------------------------------------------- geometry
// WARP rows up to d = 1024 (V words a lane); block rows with V words a thread.  One word a thread (the row's
// latency decides) while the rows run in about one round: norm and checkpoint of 1000 x 2048 3.1 us with one
// word, 4.3 with two; 1500 x 2048 (1.3 rounds) 3.8 and 4.4, 700 x 5120 (1.5) 4.7 and 4.5; LayerNorm of
// 600 x 4096 (1.0) 3.8 and 3.7 with four.  More rows, for 8192 x 5120 with 1 / 2 / 4 words: norm and checkpoint
// 46.7 / 35.0 / 36.4 us, restore and norm 42.7 / 34.2 / 34.9; LayerNorm's two reductions a row ask for fewer
// threads in each (46.7 / 37.8 / 31.7), the backward's three arrays for fewer registers (50.8 / 57.9 / 60.3).
// Gain and bias are fetched ahead where the row's latency decides, one row of 4096 1.6 us for 1.8, 64 x 576 1.5 for
// 2.0; among many rows the registers cost more (16384 x 576 11.1 for 10.6, norm and checkpoint of 200 x 16384 5.7 for
// 4.8 and of 8192 x 5120 39.5 for 34.8).
enum Pass { FORWARD, LAYERNORM, BACKWARD };
struct Geo {
  int v, threads, warp, ahead;
  unsigned blocks;
};
static Geo row_geo(int64_t rows, int d8, Pass pass) {
  Geo g;
  g.warp = d8 <= 128;
  if (g.warp) {
    g.v = d8 <= 32 ? 1 : d8 <= 64 ? 2 : 4;
    g.threads = rows >= 4 * num_sms() ? 256 : 64;
    g.ahead = g.v == 1 || g.threads == 64;
    const int per = g.threads / 32;
    g.blocks = (unsigned)((rows + per - 1) / per);
    return g;
  }
  const int64_t round = 2048ll * num_sms();  // threads that run at once
  const bool many =
      rows >= 2 * num_sms() && (pass == LAYERNORM ? rows * d8 > round : pass == FORWARD && 3 * rows * d8 > 4 * round);
  g.v = d8 > 1024 ? (many ? 4 : 2) : many && d8 >= 512 && pass == LAYERNORM ? 4 : many && d8 >= 256 ? 2 : 1;
  g.threads = (((d8 + g.v - 1) / g.v) + 31) / 32 * 32;
  g.ahead = g.v == 1 || (!many && rows <= num_sms() * (1120 / g.threads));  // the registers' one round
  g.blocks = (unsigned)rows;
  return g;
}
// Backward: a row a warp (eight warps a block) or a row a block; `occ` blocks per SM hide one another's row
// reductions (two blocks of 320 threads: 61 us for 8192 x 5120; one block of two such groups, which halves
// the partial sums: 72) and share its registers and shared memory (rings of nst stages of `stage` bytes).
struct BwdGeo {
  int v, threads, warp, nst, stage;
  unsigned blocks;
};
// Rows for the one kernel of few rows, with dg and db against the rings and their second kernel: 333 x 576 3.1 us for
// 6.6, 130 x 2048 3.3 for 5.4, 10 x 5120 2.0 for 5.6, 1000 x 5120 11.6 for 16.6, 1500 x 2048 9.9 for 12.7; but 1500 x
// 64 7.3 for 5.5, 2000 x 576 8.2 for 7.1, 1000 x 9912 29.8 for 27.2.  The host saves 2.4 us.
static bool few_rows(int64_t rows, int d8) { return rows <= (d8 < 64 ? 1024 : 1536) && rows * d8 <= 1 << 20; }
constexpr int RING_BYTES = 200 * 1024;
static BwdGeo ln_bwd_geo(int64_t rows, int d8, bool grads) {
  BwdGeo g{};
  g.stage = (3 * d8 * 16 + 127) / 128 * 128;
  g.warp = d8 <= 96;
  const int per = g.warp ? LNW : 1;
  int occ = 2;
  if (g.warp) {
    g.v = (d8 + 31) / 32;
    g.threads = LNW * 32;
  } else {
    g.v = d8 <= 640 ? 2 : 4;
    g.threads = (((d8 + g.v - 1) / g.v) + 31) / 32 * 32;
    occ = g.v == 4 ? (g.threads <= 256 ? 2 : 1) : std::max(2, std::min(6, 640 / g.threads));
  }
  // each block's sums are 8 d bytes to write and to add: whole rounds of blocks with about four rows each pay for
  // them (1000 x 2048: 9.5 / 8.3 / 9.0 / 10.8 / 12.4 us with 1 to 5 blocks per SM; 10.2 with 250 blocks)
  if (grads && !g.warp) occ = (int)std::min<int64_t>(occ, (rows + 4 * num_sms() - 1) / (4 * num_sms()));
  g.nst = std::max(2, std::min(8, RING_BYTES / occ / per / g.stage));
  g.blocks = (unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)occ * num_sms());
  return g;
}

template <typename K>
static lsq_status ring_smem(K kernel, int* configured) {
  int dev = 0;
  LSQ_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64 || configured[dev]) return LSQ_OK;
  LSQ_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES + 1024));
  configured[dev] = 1;
  return LSQ_OK;
}
template <int SRC, int NORM, bool PACK>
static lsq_status run_fwd(Fwd p, int64_t rows, int64_t d, const char* what, cudaStream_t s) {
  p.rows = rows;
  p.d8 = (int)(d / 8);
  p.nb = (int)((d + 63) / 64);
  p.inv_d = 1.0f / (float)d;
  const Geo g = row_geo(rows, p.d8, NORM == LAYER ? LAYERNORM : FORWARD);
  constexpr bool N = NORM != NONE;  // without a norm there is nothing to fetch ahead
  auto k = g.warp ? (g.v == 1   ? row_fwd_kernel<1, true, SRC, NORM, PACK, N>
                     : g.v == 2 ? (g.ahead ? row_fwd_kernel<2, true, SRC, NORM, PACK, N>
                                           : row_fwd_kernel<2, true, SRC, NORM, PACK, false>)
                                : (g.ahead ? row_fwd_kernel<4, true, SRC, NORM, PACK, N>
                                           : row_fwd_kernel<4, true, SRC, NORM, PACK, false>))
                  : (g.v == 1   ? row_fwd_kernel<1, false, SRC, NORM, PACK, N>
                     : g.v == 2 ? (g.ahead ? row_fwd_kernel<2, false, SRC, NORM, PACK, N>
                                           : row_fwd_kernel<2, false, SRC, NORM, PACK, false>)
                                : row_fwd_kernel<4, false, SRC, NORM, PACK, false>);
  return launch_chained(what, k, dim3(g.blocks), (unsigned)g.threads, 0, 1, s, p);
}
template <int V, bool WARP, bool GRADS>
static lsq_status run_ln_bwd(const Bwd& p, const BwdGeo& g, cudaStream_t s) {
  static int configured[64] = {0};
  const size_t smem = (size_t)g.nst * (g.stage + 8) * (WARP ? LNW : 1);
  if constexpr (WARP) {
    lsq_status st = ring_smem(ln_bwd_warp_kernel<V, GRADS>, configured);
    if (st != LSQ_OK) return st;
    return launch_chained("ln_bwd_warp_kernel", ln_bwd_warp_kernel<V, GRADS>, dim3(g.blocks), (unsigned)g.threads, smem,
                          1, s, p, g.nst, g.stage);
  } else {
    lsq_status st = ring_smem(ln_bwd_block_kernel<V, GRADS>, configured);
    if (st != LSQ_OK) return st;
    return launch_chained("ln_bwd_block_kernel", ln_bwd_block_kernel<V, GRADS>, dim3(g.blocks), (unsigned)g.threads,
                          smem, 1, s, p, g.nst, g.stage);
  }
}
template <int V, bool WARP>
static lsq_status run_ln_bwd(const Bwd& p, bool grads, const BwdGeo& g, cudaStream_t s) {
  return grads ? run_ln_bwd<V, WARP, true>(p, g, s) : run_ln_bwd<V, WARP, false>(p, g, s);
}

static lsq_status run_ln_bwd_few(const Bwd& p, bool grads, cudaStream_t s) {
  const int d8 = p.d8;
  const bool warp = d8 <= 128;
  const unsigned threads = d8 > 1024 ? 512 : 256;
  auto k = warp ? (d8 <= 32   ? ln_bwd_few_kernel<1, true>
                   : d8 <= 64 ? ln_bwd_few_kernel<2, true>
                              : ln_bwd_few_kernel<4, true>)
                : (d8 <= 256   ? ln_bwd_few_kernel<1, false>
                   : d8 <= 512 ? ln_bwd_few_kernel<2, false>
                               : ln_bwd_few_kernel<4, false>);
  // Column blocks of 32 to 256 columns (64 bytes of a row at least): a block costs its place about 2.5 us, a row of
  // a thread 0.12.  With 32 / 64 / 128 / 256 columns: 333 x 576 3.1 / 3.5 / 4.4 / 6.8 us, 333 x 5120 5.5 / 4.2 / 5.1 /
  // 7.3, 130 x 16384 11.7 / 7.8 / 5.6 / 5.7.
  const int slots = num_sms() * (threads == 512 ? 1 : d8 > 512 || (warp && d8 > 64) ? 2 : 4);
  int seg = 2;
  double least = 1e30;
  for (int i = 2; i <= 5; ++i) {
    const double us = 2.5 * ((d8 + (1 << i) - 1) >> i) / slots + 0.12 * (double)(p.rows << i) / threads;
    if (us < least) least = us, seg = i;
  }
  const int cols = grads ? (d8 + (1 << seg) - 1) >> seg : 0;
  const size_t smem = (size_t)(threads / 32) * FEW_PITCH * sizeof(float) << seg;
  const unsigned rows = (unsigned)(warp ? (p.rows + 7) / 8 : p.rows);
  const char* what = "ln_bwd_few_kernel";
  // in place over dy or x the sums have to be read first
  if (grads && (p.out == p.dy || p.out == p.x)) {
    lsq_status st = launch_chained(what, k, dim3((unsigned)cols), threads, smem, 1, s, p, cols, seg);
    return st != LSQ_OK ? st : launch_chained(what, k, dim3(rows), threads, 0, 1, s, p, 0, seg);
  }
  return launch_chained(what, k, dim3((unsigned)cols + rows), threads, smem, 1, s, p, cols, seg);
}

// the shape and alignment rules of the section, with this file's limits
static lsq_status check_rows(const char* who, int64_t rows, int64_t d) {
  if (rows < 1 || rows > 0x7fffffffll || d < 8 || d % 8 != 0)
    return fail(LSQ_EINVAL, "%s: need 1 <= rows < 2^31, d a positive multiple of 8 (got %lld, %lld)", who,
                (long long)rows, (long long)d);
  if (d > MAX_D) return fail(LSQ_EUNSUPPORTED, "%s: d <= %lld (got %lld)", who, (long long)MAX_D, (long long)d);
  return LSQ_OK;
}
template <typename... P>
static bool aligned16(P... p) {
  return (... && aligned(p, 16));
}
template <typename... P>
static bool aligned4(P... p) {
  return (... && aligned(p, 4));
}
struct Range {
  const void* p;  // null: none
  size_t n;
};
// an output shares bytes with an input or another output
template <size_t O, size_t I>
static bool clash(const Range (&out)[O], const Range (&in)[I]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Range& r : in)
      if (overlap(out[i].p, out[i].n, r.p, r.n)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}
// an output over its input's bytes at another place: a row would be written before another reads it
static bool shifted(const void* in, const void* out, size_t bytes) {
  return in != out && overlap(in, bytes, out, bytes);
}

}  // namespace nrm
}  // namespace lsq

using namespace lsq;

extern "C" lsq_status lsq_layernorm_fwd(const void* x, const void* g, const void* b, void* y, float* mean, float* rstd,
                                        int64_t rows, int64_t d, float eps, lsq_cuda_stream stream) {
  const char* who = "lsq_layernorm_fwd";
  if (!x || !g || !y) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, g, b, y) || !nrm::aligned4(mean, rstd)) return fail(LSQ_EINVAL, "%s: alignment", who);
  const size_t xb = (size_t)rows * d * 2, gb = (size_t)d * 2, sb = (size_t)rows * 4;
  const nrm::Range out[] = {{y, xb}, {mean, sb}, {rstd, sb}}, in[] = {{x == y ? nullptr : x, xb}, {g, gb}, {b, gb}};
  if (nrm::clash(out, in)) return fail(LSQ_EINVAL, "%s: overlapping arguments (y may be x itself)", who);
  if ((st = check_device()) != LSQ_OK) return st;
  nrm::Fwd p{};
  p.x = (const uint4*)x;
  p.g = (const uint4*)g;
  p.b = (const uint4*)b;
  p.y = (uint4*)y;
  p.mean = mean;
  p.rstd = rstd;
  p.eps = eps;
  return nrm::run_fwd<nrm::BF16, nrm::LAYER, false>(p, rows, d, "row_fwd_kernel (layernorm)", (cudaStream_t)stream);
}

extern "C" size_t lsq_layernorm_bwd_workspace_size(int64_t rows, int64_t d) {
  if (rows < 1 || d < 8 || d > nrm::MAX_D) return 256;
  if (nrm::few_rows(rows, (int)(d / 8))) return 256;
  const nrm::BwdGeo g = nrm::ln_bwd_geo(rows, (int)(d / 8), true);
  return ((size_t)g.blocks * 2 * (size_t)d * sizeof(float) + 255) / 256 * 256;
}

extern "C" lsq_status lsq_layernorm_bwd(const void* dy, const void* x, const void* g, const float* mean,
                                        const float* rstd, const void* dres_in, void* dres_out, float* dg, float* db,
                                        int32_t accumulate, int64_t rows, int64_t d, void* workspace,
                                        size_t workspace_bytes, lsq_cuda_stream stream) {
  const char* who = "lsq_layernorm_bwd";
  if (!dy || !x || !g || !mean || !rstd || !dres_out) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(dy, x, g, dres_in, dres_out, dg, db) || !nrm::aligned4(mean, rstd))
    return fail(LSQ_EINVAL, "%s: alignment", who);
  const size_t xb = (size_t)rows * d * 2, gb = (size_t)d * 4, sb = (size_t)rows * 4;
  const bool grads = dg || db;
  const size_t wb = grads ? lsq_layernorm_bwd_workspace_size(rows, d) : 0;
  if (grads && (!workspace || !aligned(workspace, 256) || workspace_bytes < wb))
    return fail(LSQ_EINVAL, "%s: workspace missing, misaligned or too small", who);
  auto in_place = [&](const void* v) { return v == dres_out ? nullptr : v; };
  const nrm::Range out[] = {{dres_out, xb}, {dg, gb}, {db, gb}, {grads ? workspace : nullptr, wb}};
  const nrm::Range in[] = {{in_place(dy), xb}, {in_place(x), xb}, {in_place(dres_in), xb},
                           {g, gb / 2},        {mean, sb},        {rstd, sb}};
  if (nrm::clash(out, in))
    return fail(LSQ_EINVAL, "%s: overlapping arguments (dres_out may be dy, x or dres_in itself)", who);
  if ((st = check_device()) != LSQ_OK) return st;
  if (grads && workspace_bytes < lsq_layernorm_bwd_workspace_size(rows, d))  // now that the device's SMs are known
    return fail(LSQ_EINVAL, "%s: workspace too small for this device", who);
  nrm::Bwd p{};
  p.dy = (const uint4*)dy;
  p.x = (const uint4*)x;
  p.g = (const uint4*)g;
  p.mean = mean;
  p.rstd = rstd;
  p.res = (const uint4*)dres_in;
  p.out = (uint4*)dres_out;
  p.part = static_cast<float*>(workspace);
  p.dg = dg;
  p.db = db;
  p.rows = rows;
  p.d8 = (int)(d / 8);
  p.accumulate = accumulate ? 1 : 0;
  p.inv_d = 1.0f / (float)d;
  cudaStream_t s = (cudaStream_t)stream;
  if (nrm::few_rows(rows, p.d8)) return nrm::run_ln_bwd_few(p, grads, s);
  const nrm::BwdGeo ge = nrm::ln_bwd_geo(rows, p.d8, grads);
  if (ge.warp)
    st = ge.v == 1   ? nrm::run_ln_bwd<1, true>(p, grads, ge, s)
         : ge.v == 2 ? nrm::run_ln_bwd<2, true>(p, grads, ge, s)
                     : nrm::run_ln_bwd<3, true>(p, grads, ge, s);
  else
    st = ge.v == 2 ? nrm::run_ln_bwd<2, false>(p, grads, ge, s) : nrm::run_ln_bwd<4, false>(p, grads, ge, s);
  if (st != LSQ_OK) return st;
  if (!grads) return LSQ_OK;
  return nrm::col_sum(p.part, (int)ge.blocks, 2 * d, d, 2 * d, dg, db, p.accumulate, s);
}

// ---------------------------------------------------------------- 8-bit checkpoints
extern "C" size_t lsq_ckpt8_size(int64_t rows, int64_t d) {
  if (rows < 1 || d < 1) return 256;
  return (nrm::ckpt_used(rows, d) + 255) / 256 * 256;
}

extern "C" lsq_status lsq_ckpt8_pack(const void* x, void* ckpt, int64_t rows, int64_t d, lsq_cuda_stream stream) {
  const char* who = "lsq_ckpt8_pack";
  if (!x || !ckpt) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, ckpt)) return fail(LSQ_EINVAL, "%s: alignment", who);
  if (overlap(x, (size_t)rows * d * 2, ckpt, nrm::ckpt_used(rows, d)))
    return fail(LSQ_EINVAL, "%s: x overlaps the checkpoint", who);
  if ((st = check_device()) != LSQ_OK) return st;
  nrm::Fwd p{};
  p.x = (const uint4*)x;
  p.out = nrm::ckpt_of(ckpt, rows, d);
  return nrm::run_fwd<nrm::BF16, nrm::NONE, true>(p, rows, d, "row_fwd_kernel (pack8)", (cudaStream_t)stream);
}

extern "C" lsq_status lsq_ckpt8_unpack(const void* ckpt, void* x, int64_t rows, int64_t d, lsq_cuda_stream stream) {
  const char* who = "lsq_ckpt8_unpack";
  if (!x || !ckpt) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, ckpt)) return fail(LSQ_EINVAL, "%s: alignment", who);
  if (overlap(x, (size_t)rows * d * 2, ckpt, nrm::ckpt_used(rows, d)))
    return fail(LSQ_EINVAL, "%s: x overlaps the checkpoint", who);
  if ((st = check_device()) != LSQ_OK) return st;
  nrm::Fwd p{};
  p.xo = (uint4*)x;
  p.in = nrm::ckpt_of(ckpt, rows, d);
  return nrm::run_fwd<nrm::CKPT8, nrm::NONE, false>(p, rows, d, "row_fwd_kernel (unpack8)", (cudaStream_t)stream);
}

extern "C" lsq_status lsq_rmsnorm_fwd_pack8(const void* x, const void* g, void* y, float* rstd, void* ckpt,
                                            int64_t rows, int64_t d, float eps, lsq_cuda_stream stream) {
  const char* who = "lsq_rmsnorm_fwd_pack8";
  if (!x || !g || !y || !ckpt) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, g, y, ckpt) || !nrm::aligned4(rstd)) return fail(LSQ_EINVAL, "%s: alignment", who);
  const size_t xb = (size_t)rows * d * 2, cb = nrm::ckpt_used(rows, d);
  const nrm::Range out[] = {{y, xb}, {rstd, (size_t)rows * 4}, {ckpt, cb}};
  const nrm::Range in[] = {{x == y ? nullptr : x, xb}, {g, (size_t)d * 2}};
  if (nrm::clash(out, in)) return fail(LSQ_EINVAL, "%s: overlapping arguments (y may be x itself)", who);
  if ((st = check_device()) != LSQ_OK) return st;
  nrm::Fwd p{};
  p.x = (const uint4*)x;
  p.g = (const uint4*)g;
  p.y = (uint4*)y;
  p.rstd = rstd;
  p.out = nrm::ckpt_of(ckpt, rows, d);
  p.eps = eps;
  return nrm::run_fwd<nrm::BF16, nrm::RMS, true>(p, rows, d, "row_fwd_kernel (rmsnorm pack8)", (cudaStream_t)stream);
}

extern "C" lsq_status lsq_rmsnorm_fwd_unpack8(const void* ckpt, const void* g, void* x, void* y, float* rstd,
                                              int64_t rows, int64_t d, float eps, lsq_cuda_stream stream) {
  const char* who = "lsq_rmsnorm_fwd_unpack8";
  if (!x || !g || !y || !ckpt) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, g, y, ckpt) || !nrm::aligned4(rstd)) return fail(LSQ_EINVAL, "%s: alignment", who);
  const size_t xb = (size_t)rows * d * 2;
  const nrm::Range out[] = {{x, xb}, {y, xb}, {rstd, (size_t)rows * 4}};
  const nrm::Range in[] = {{ckpt, nrm::ckpt_used(rows, d)}, {g, (size_t)d * 2}};
  if (nrm::clash(out, in)) return fail(LSQ_EINVAL, "%s: overlapping arguments", who);
  if ((st = check_device()) != LSQ_OK) return st;
  nrm::Fwd p{};
  p.in = nrm::ckpt_of(ckpt, rows, d);
  p.g = (const uint4*)g;
  p.xo = (uint4*)x;
  p.y = (uint4*)y;
  p.rstd = rstd;
  p.eps = eps;
  return nrm::run_fwd<nrm::CKPT8, nrm::RMS, false>(p, rows, d, "row_fwd_kernel (rmsnorm unpack8)",
                                                   (cudaStream_t)stream);
}

extern "C" lsq_status lsq_rmsnorm_bwd_unpack8(const void* dy, const void* ckpt, const void* g, const float* rstd,
                                              const void* dres_in, void* dres_out, int64_t rows, int64_t d,
                                              lsq_cuda_stream stream) {
  const char* who = "lsq_rmsnorm_bwd_unpack8";
  if (!dy || !ckpt || !g || !rstd || !dres_out) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(dy, ckpt, g, dres_in, dres_out) || !nrm::aligned4(rstd))
    return fail(LSQ_EINVAL, "%s: alignment", who);
  const size_t xb = (size_t)rows * d * 2;
  const nrm::Range out[] = {{dres_out, xb}};
  const nrm::Range in[] = {{dy == dres_out ? nullptr : dy, xb},
                           {dres_in == dres_out ? nullptr : dres_in, xb},
                           {ckpt, nrm::ckpt_used(rows, d)},
                           {g, (size_t)d * 2},
                           {rstd, (size_t)rows * 4}};
  if (nrm::clash(out, in))
    return fail(LSQ_EINVAL, "%s: overlapping arguments (dres_out may be dy or dres_in itself)", who);
  if ((st = check_device()) != LSQ_OK) return st;
  nrm::Bwd p{};
  p.dy = (const uint4*)dy;
  p.g = (const uint4*)g;
  p.in = nrm::ckpt_of(ckpt, rows, d);
  p.rstd = rstd;
  p.res = (const uint4*)dres_in;
  p.out = (uint4*)dres_out;
  p.rows = rows;
  p.d8 = (int)(d / 8);
  p.nb = (int)((d + 63) / 64);
  p.inv_d = 1.0f / (float)d;
  cudaStream_t s = (cudaStream_t)stream;
  const nrm::Geo ge = nrm::row_geo(rows, p.d8, nrm::BACKWARD);
  auto k = ge.warp ? (ge.v == 1   ? nrm::rms_bwd_unpack8_kernel<1, true>
                      : ge.v == 2 ? nrm::rms_bwd_unpack8_kernel<2, true>
                                  : nrm::rms_bwd_unpack8_kernel<4, true>)
                   : (ge.v == 1 ? nrm::rms_bwd_unpack8_kernel<1, false> : nrm::rms_bwd_unpack8_kernel<2, false>);
  return launch_chained("rms_bwd_unpack8_kernel", k, dim3(ge.blocks), (unsigned)ge.threads, 0, 1, s, p);
}
