// LayerNorm (forward, backward, gradients of gain and bias) and the 8-bit
// activation checkpoint with the RMSNorm passes that write and read it.
//
// All are HBM-bound row passes over bf16 [rows, d].  A row belongs to one warp
// (WARP, d <= 1024) or to one block; each thread holds V 16-byte words of it
// in registers from the one load to the last use, so every input is read once.
// Word c of a row belongs to thread c % T (T threads per row, a multiple of
// 32), so eight neighbouring lanes hold one 64-column block of the checkpoint.
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
// (the caller alternates between two buffers, so no second one)
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (WARP) return v;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (l == 0) red[w] = v;
  __syncthreads();
  return warp_sum(l < (int)(blockDim.x >> 5) ? red[l] : 0.0f);
}
template <bool WARP>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (WARP) return make_float2(a, b);
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  if (l == 0) red[w] = make_float2(a, b);
  __syncthreads();
  const float2 t = l < (int)(blockDim.x >> 5) ? red[l] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(t.x), warp_sum(t.y));
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
  float f[8];
  unpack8(w, f);
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(fmaf(f[i], inv, CODE_MAGIC));
  return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
}
__device__ __forceinline__ uint4 decode8(uint2 codes, uint32_t amax) {
  const float s = __uint_as_float(amax << 16) * INV_127;
  float f[8];
  const uint32_t a = codes.x ^ 0x80808080u, b = codes.y ^ 0x80808080u;  // q + 128, unsigned
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = (__uint_as_float(__byte_perm(a, 0x4b000000u, 0x7440 + i)) - 8388736.0f) * s;  // 2^23 + q + 128
    f[4 + i] = (__uint_as_float(__byte_perm(b, 0x4b000000u, 0x7440 + i)) - 8388736.0f) * s;
  }
  return pack8(f);
}

struct Ckpt {
  uint8_t* codes;   // int8 [rows][d]
  uint16_t* amax;   // bf16 [rows][ceil(d / 64)]
};
static size_t ckpt_amax_off(int64_t rows, int64_t d) { return (size_t)(rows * d + 15) / 16 * 16; }
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

template <int V, bool WARP, int SRC, int NORM, bool PACK>
__global__ void __launch_bounds__(WARP ? 256 : V == 4 ? 512 : 1024) row_fwd_kernel(const __grid_constant__ Fwd p) {
  __shared__ float red[2][32];
  const int T = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
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
  if (NORM == NONE) return;
  float mu = 0.0f, ss = 0.0f;
  if (NORM == LAYER) {  // the mean first, then the centred squares: no cancellation
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8(xv[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
    }
    mu = row_sum<WARP>(s, red[0]) * p.inv_d;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (NORM == LAYER && t + i * T >= d8) break;  // the padding is not centred
    float f[8];
    unpack8(xv[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j] - mu, f[j] - mu, ss);
  }
  const float rs = 1.0f / sqrtf(row_sum<WARP>(ss, red[1]) * p.inv_d + p.eps);
  if (t == 0) {
    if (p.mean) p.mean[row] = mu;
    if (p.rstd) p.rstd[row] = rs;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (c >= d8) break;
    float f[8], gv[8], bv[8];
    unpack8(xv[i], f);
    unpack8(p.g[c], gv);
    if (NORM == LAYER && p.b) {
      unpack8(p.b[c], bv);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf((f[j] - mu) * rs, gv[j], bv[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (f[j] - mu) * rs * gv[j];
    }
    p.y[base + c] = pack8(f);
  }
}

// ---------------------------------------------------------------- row passes, backward
struct Bwd {
  const uint4 *dy, *x, *g;
  Ckpt in;
  const float *mean, *rstd;
  const uint4* res;   // dres_in or null; may alias out
  uint4* out;
  float* part;        // [gridDim.x][2][d]: this block's sums of dy xhat and dy (GRADS)
  float *dg, *db;     // written here when the grid is one block
  int64_t rows;
  int d8, nb, accumulate;
  float inv_d;
};

// RMSNorm from a checkpoint: out = res + rs (dy g) - x rs^3 mean(dy g x), one row per warp or block
template <int V, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : V == 4 ? 512 : 1024) rms_bwd_unpack8_kernel(const __grid_constant__ Bwd p) {
  __shared__ float red[32];
  const int T = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
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
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[8], d[8], g[8];
    unpack8(decode8(cv[i], av[i]), f);
    unpack8(dv[i], d);
    unpack8(gv[i], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) dot = fmaf(d[j] * g[j], f[j], dot);
  }
  const float k = rs * rs * rs * row_sum<WARP>(dot, red) * p.inv_d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = t + i * T;
    if (c >= d8) break;
    float f[8], d[8], g[8], o[8];
    unpack8(decode8(cv[i], av[i]), f);
    unpack8(dv[i], d);
    unpack8(gv[i], g);
    unpack8(rv[i], o);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] += rs * d[j] * g[j] - f[j] * k;
    p.out[base + c] = pack8(o);
  }
}

// LayerNorm: out = res + rs (a - mean(a) - xh mean(a xh)), a = dy g, xh = (x - mean) rs.  Blocks walk
// the rows in strides and a thread's columns stay the same, so the sums over rows of dy xh and dy
// (dg, db) collect in registers and leave once per block; col_sum_kernel adds the blocks in order.
template <int V, bool WARP, bool GRADS>
__global__ void __launch_bounds__(WARP ? 256 : 512) ln_bwd_kernel(const __grid_constant__ Bwd p) {
  __shared__ float2 red[2][32];
  __shared__ float comb[WARP ? 8 * 32 * 9 : 1];
  const int T = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int nw = (int)(blockDim.x >> 5), w = (int)(threadIdx.x >> 5);
  const int64_t first = WARP ? (int64_t)blockIdx.x * nw + w : (int64_t)blockIdx.x;
  const int64_t step = WARP ? (int64_t)gridDim.x * nw : (int64_t)gridDim.x;
  const int d8 = p.d8;
  const uint4 z = make_uint4(0u, 0u, 0u, 0u);
  // V = 4 (block rows): the sums take 64 registers, so gain and residual are loaded at their use
  constexpr bool LATE = !WARP && V == 4;
  uint4 gk[LATE ? 1 : V];
  if (!LATE) {
#pragma unroll
    for (int i = 0; i < V; ++i) gk[LATE ? 0 : i] = t + i * T < d8 ? p.g[t + i * T] : z;
  }
  auto gain = [&](int i) { return LATE ? (t + i * T < d8 ? p.g[t + i * T] : z) : gk[LATE ? 0 : i]; };
  float sg[GRADS ? V : 1][8], sb[GRADS ? V : 1][8];
  if (GRADS) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sg[i][j] = sb[i][j] = 0.0f;
  }
  int flip = 0;
  for (int64_t row = first; row < p.rows; row += step, flip ^= 1) {
    const int64_t base = row * d8;
    uint4 xv[V], dv[V], rv[LATE ? 1 : V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      const bool in = c < d8;
      xv[i] = in ? p.x[base + c] : z;
      dv[i] = in ? p.dy[base + c] : z;
      if (!LATE) rv[LATE ? 0 : i] = (in && p.res) ? p.res[base + c] : z;
    }
    const float mu = p.mean[row], rs = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8], d[8], g[8];
      unpack8(xv[i], f);
      unpack8(dv[i], d);
      unpack8(gain(i), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // padded columns: d = g = 0
        const float xh = (f[j] - mu) * rs, a = d[j] * g[j];
        s1 += a;
        s2 = fmaf(a, xh, s2);
        if (GRADS) {
          sg[i][j] = fmaf(d[j], xh, sg[i][j]);
          sb[i][j] += d[j];
        }
      }
    }
    const float2 s = row_sum2<WARP>(s1, s2, red[flip]);
    const float m1 = s.x * p.inv_d, m2 = s.y * p.inv_d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = t + i * T;
      if (c >= d8) break;
      float f[8], d[8], g[8], o[8];
      unpack8(xv[i], f);
      unpack8(dv[i], d);
      unpack8(gain(i), g);
      unpack8(LATE ? (p.res ? p.res[base + c] : z) : rv[LATE ? 0 : i], o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += rs * (d[j] * g[j] - m1 - (f[j] - mu) * rs * m2);
      p.out[base + c] = pack8(o);
    }
  }
  if (!GRADS) return;
  const int d = d8 * 8;
  const bool one = gridDim.x == 1;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = h ? sb[i][j] : sg[i][j];
      if (WARP) {  // the warps' sums, in warp order; row stride 9 keeps the banks apart
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) comb[(w * 32 + t) * 9 + j] = v[j];
        __syncthreads();
        if (w != 0) continue;
        for (int k = 1; k < nw; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += comb[(k * 32 + t) * 9 + j];
      }
      const int c = t + i * T;
      if (c >= d8) continue;
      float* o = one ? (h ? p.db : p.dg) : p.part + ((int64_t)blockIdx.x * 2 + h) * d;
      if (!o) continue;
      float4* o4 = reinterpret_cast<float4*>(o + c * 8);
      if (one && p.accumulate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += o[c * 8 + j];
      }
      o4[0] = make_float4(v[0], v[1], v[2], v[3]);
      o4[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

// out0[c] (+)= sum over the G rows of part[.][c] for c < n0, out1[c - n0] for the columns from n0 on
// (either may be null); part has row stride ld.  16 warps take rows w, w + 16, ..., added in warp order.
__global__ void __launch_bounds__(512) col_sum_kernel(const float* __restrict__ part, int G, int64_t ld, int64_t n0,
                                                      int64_t ncols, float* out0, float* out1, int accumulate) {
  __shared__ float s[16][33];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;
  float v = 0.0f;
  if (c < ncols)
    for (int r = w; r < G; r += 16) v += part[r * ld + c];
  s[w][l] = v;
  __syncthreads();
  if (w != 0 || c >= ncols) return;
  float tot = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) tot += s[k][l];
  float* o = c < n0 ? (out0 ? out0 + c : nullptr) : (out1 ? out1 + (c - n0) : nullptr);
  if (o) *o = accumulate ? *o + tot : tot;
}

lsq_status col_sum(const float* part, int G, int64_t ld, int64_t n0, int64_t ncols, float* out0, float* out1,
                   int accumulate, cudaStream_t stream) {
  col_sum_kernel<<<(unsigned)((ncols + 31) / 32), 512, 0, stream>>>(part, G, ld, n0, ncols, out0, out1, accumulate);
  LSQ_LAUNCH_CHECK("col_sum_kernel");
  return LSQ_OK;
}

// ---------------------------------------------------------------- geometry
// WARP rows up to d = 1024 (V words a lane); block rows with V words a thread.  Few rows: one word a
// thread (the row's latency decides); many: more words a thread (fewer threads per reduction).
struct Geo {
  int v, threads, warp;
  unsigned blocks;
};
static Geo fwd_geo(int64_t rows, int d8) {
  Geo g;
  g.warp = d8 <= 128;
  if (g.warp) {
    g.v = d8 <= 32 ? 1 : d8 <= 64 ? 2 : 4;
    g.threads = rows >= 4 * num_sms() ? 256 : 64;
    const int per = g.threads / 32;
    g.blocks = (unsigned)((rows + per - 1) / per);
    return g;
  }
  g.v = rows >= 2 * num_sms() ? (d8 >= 512 ? 4 : d8 >= 256 ? 2 : 1) : (d8 > 1024 ? 2 : 1);
  g.threads = (((d8 + g.v - 1) / g.v) + 31) / 32 * 32;
  g.blocks = (unsigned)rows;
  return g;
}
static Geo ln_bwd_geo(int64_t rows, int d8) {
  Geo g;
  g.warp = d8 <= 128;
  int per = 1, occ;
  if (g.warp) {
    g.v = d8 <= 32 ? 1 : d8 <= 64 ? 2 : 4;
    g.threads = 256;
    per = 8;
    occ = 2;
  } else {
    g.v = d8 <= 512 ? 1 : d8 <= 1024 ? 2 : 4;
    g.threads = (((d8 + g.v - 1) / g.v) + 31) / 32 * 32;
    occ = g.threads <= 256 ? 4 : 2;
  }
  g.blocks = (unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)occ * num_sms());
  return g;
}

template <int SRC, int NORM, bool PACK>
static lsq_status run_fwd(Fwd p, int64_t rows, int64_t d, const char* what, cudaStream_t s) {
  p.rows = rows;
  p.d8 = (int)(d / 8);
  p.nb = (int)((d + 63) / 64);
  p.inv_d = 1.0f / (float)d;
  const Geo g = fwd_geo(rows, p.d8);
  if (g.warp) {
    if (g.v == 1) row_fwd_kernel<1, true, SRC, NORM, PACK><<<g.blocks, g.threads, 0, s>>>(p);
    else if (g.v == 2) row_fwd_kernel<2, true, SRC, NORM, PACK><<<g.blocks, g.threads, 0, s>>>(p);
    else row_fwd_kernel<4, true, SRC, NORM, PACK><<<g.blocks, g.threads, 0, s>>>(p);
  } else {
    if (g.v == 1) row_fwd_kernel<1, false, SRC, NORM, PACK><<<g.blocks, g.threads, 0, s>>>(p);
    else if (g.v == 2) row_fwd_kernel<2, false, SRC, NORM, PACK><<<g.blocks, g.threads, 0, s>>>(p);
    else row_fwd_kernel<4, false, SRC, NORM, PACK><<<g.blocks, g.threads, 0, s>>>(p);
  }
  LSQ_LAUNCH_CHECK(what);
  return LSQ_OK;
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

}  // namespace nrm
}  // namespace lsq

using namespace lsq;

extern "C" lsq_status lsq_layernorm_fwd(const void* x, const void* g, const void* b, void* y, float* mean, float* rstd,
                                        int64_t rows, int64_t d, float eps, lsq_cuda_stream stream) {
  const char* who = "lsq_layernorm_fwd";
  if (!x || !g || !y) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, g, b, y)) return fail(LSQ_EINVAL, "%s: alignment", who);
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
  const nrm::Geo g = nrm::ln_bwd_geo(rows, (int)(d / 8));
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
  if (!nrm::aligned16(dy, x, g, dres_in, dres_out, dg, db)) return fail(LSQ_EINVAL, "%s: alignment", who);
  const bool grads = dg || db;
  if (grads && (!workspace || !aligned(workspace, 256) || workspace_bytes < lsq_layernorm_bwd_workspace_size(rows, d)))
    return fail(LSQ_EINVAL, "%s: workspace missing, misaligned or too small", who);
  if ((st = check_device()) != LSQ_OK) return st;
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
  const nrm::Geo ge = nrm::ln_bwd_geo(rows, p.d8);
  cudaStream_t s = (cudaStream_t)stream;
#define LSQ_LN_BWD(V, W)                                                                     \
  (grads ? nrm::ln_bwd_kernel<V, W, true><<<ge.blocks, ge.threads, 0, s>>>(p)                \
         : nrm::ln_bwd_kernel<V, W, false><<<ge.blocks, ge.threads, 0, s>>>(p))
  if (ge.warp) {
    if (ge.v == 1) LSQ_LN_BWD(1, true);
    else if (ge.v == 2) LSQ_LN_BWD(2, true);
    else LSQ_LN_BWD(4, true);
  } else {
    if (ge.v == 1) LSQ_LN_BWD(1, false);
    else if (ge.v == 2) LSQ_LN_BWD(2, false);
    else LSQ_LN_BWD(4, false);
  }
#undef LSQ_LN_BWD
  LSQ_LAUNCH_CHECK("ln_bwd_kernel");
  if (!grads || ge.blocks == 1) return LSQ_OK;
  return nrm::col_sum(p.part, (int)ge.blocks, 2 * d, d, 2 * d, dg, db, p.accumulate, s);
}

// ---------------------------------------------------------------- 8-bit checkpoints
extern "C" size_t lsq_ckpt8_size(int64_t rows, int64_t d) {
  if (rows < 1 || d < 1) return 256;
  return (nrm::ckpt_amax_off(rows, d) + (size_t)rows * (size_t)((d + 63) / 64) * 2 + 255) / 256 * 256;
}

extern "C" lsq_status lsq_ckpt8_pack(const void* x, void* ckpt, int64_t rows, int64_t d, lsq_cuda_stream stream) {
  const char* who = "lsq_ckpt8_pack";
  if (!x || !ckpt) return fail(LSQ_EINVAL, "%s: NULL argument", who);
  lsq_status st = nrm::check_rows(who, rows, d);
  if (st != LSQ_OK) return st;
  if (!nrm::aligned16(x, ckpt)) return fail(LSQ_EINVAL, "%s: alignment", who);
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
  if (!nrm::aligned16(x, g, y, ckpt)) return fail(LSQ_EINVAL, "%s: alignment", who);
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
  if (!nrm::aligned16(x, g, y, ckpt)) return fail(LSQ_EINVAL, "%s: alignment", who);
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
  if (!nrm::aligned16(dy, ckpt, g, dres_in, dres_out)) return fail(LSQ_EINVAL, "%s: alignment", who);
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
  const nrm::Geo ge = nrm::fwd_geo(rows, p.d8);
  cudaStream_t s = (cudaStream_t)stream;
  if (ge.warp) {
    if (ge.v == 1) nrm::rms_bwd_unpack8_kernel<1, true><<<ge.blocks, ge.threads, 0, s>>>(p);
    else if (ge.v == 2) nrm::rms_bwd_unpack8_kernel<2, true><<<ge.blocks, ge.threads, 0, s>>>(p);
    else nrm::rms_bwd_unpack8_kernel<4, true><<<ge.blocks, ge.threads, 0, s>>>(p);
  } else {
    if (ge.v == 1) nrm::rms_bwd_unpack8_kernel<1, false><<<ge.blocks, ge.threads, 0, s>>>(p);
    else if (ge.v == 2) nrm::rms_bwd_unpack8_kernel<2, false><<<ge.blocks, ge.threads, 0, s>>>(p);
    else nrm::rms_bwd_unpack8_kernel<4, false><<<ge.blocks, ge.threads, 0, s>>>(p);
  }
  LSQ_LAUNCH_CHECK("rms_bwd_unpack8_kernel");
  return LSQ_OK;
}
