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
#include <algorithm>

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

// ---------------------------------------------------------------- activations
// act(z) and act'(z) in fp32 on the fp32 pre-activation.  GELU: z Phi(z), Phi by erfcf on the side where
// it does not cancel; its tanh form and SiLU are z sigmoid(u), the logistic through expf, which under- and
// overflows to the right limits.
__device__ __forceinline__ float logistic(float u) { return 1.0f / (1.0f + expf(-u)); }
__device__ __forceinline__ float phi_cdf_f(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }
constexpr float GT_C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float GT_A = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if (ACT == LSQ_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if (ACT == LSQ_ACT_GELU) return z == -INFINITY ? 0.0f : z * phi_cdf_f(z);
  if (ACT == LSQ_ACT_GELU_TANH) return z == -INFINITY ? 0.0f : z * logistic(GT_C * (z + GT_A * z * z * z));
  if (ACT == LSQ_ACT_SILU) return z == -INFINITY ? 0.0f : z * logistic(z);
  return z;
}
template <int ACT>
__device__ __forceinline__ float dact_f(float z) {
  if (ACT == LSQ_ACT_RELU) return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
  // beyond |z| = 1e4 every derivative here is 0 or 1 in fp32, and the products below would meet inf * 0
  if (ACT != LSQ_ACT_NONE && fabsf(z) > 1e4f) return z > 0.0f ? 1.0f : 0.0f;
  if (ACT == LSQ_ACT_GELU) return phi_cdf_f(z) + z * 0.3989422804014327f * expf(-0.5f * z * z);
  if (ACT == LSQ_ACT_GELU_TANH) {
    const float s = logistic(GT_C * (z + GT_A * z * z * z));
    return s + z * s * (1.0f - s) * GT_C * (1.0f + 3.0f * GT_A * z * z);
  }
  if (ACT == LSQ_ACT_SILU) {
    const float s = logistic(z);
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}
__device__ __forceinline__ float act_of(int act, float z) {
  switch (act) {
    case LSQ_ACT_RELU: return act_f<LSQ_ACT_RELU>(z);
    case LSQ_ACT_GELU: return act_f<LSQ_ACT_GELU>(z);
    case LSQ_ACT_GELU_TANH: return act_f<LSQ_ACT_GELU_TANH>(z);
    case LSQ_ACT_SILU: return act_f<LSQ_ACT_SILU>(z);
    default: return z;
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
  int tp, splits;  // 128-column tiles; cluster size (contraction split)
  Epi e;
};
struct Maps {
  CUtensorMap p, q;
};

// eight neighbouring columns of one output row: bias, z, activation, residual, one rounding, one store
__device__ __forceinline__ void finish8(float (&v)[8], const Epi& e, int64_t off, int col) {
  if (e.f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(e.out) + off);
    if (e.accumulate) {
      const float4 a = o[0], b = o[1];
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  if (e.bias) {
    float b[8];
    unpack8(*reinterpret_cast<const uint4*>(e.bias + col), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (e.z) *reinterpret_cast<uint4*>(e.z + off) = pack8(v);
  if (e.act != LSQ_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_of(e.act, v[i]);
  }
  if (e.residual) {
    float r[8];
    unpack8(*reinterpret_cast<const uint4*>(e.residual + off), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(e.out) + off) = pack8(v);
}

// ---------------------------------------------------------------- one tile per cluster
// 128 output columns (the tensor core's M, so few output rows waste none of it) x BT output rows; the S
// CTAs of a cluster split the contraction, each leaves its fp32 partial tile in the shared memory of the
// CTA that finishes those rows (BT / S of them), and that CTA adds them in rank order: no atomics, no
// second kernel, no workspace.
constexpr int BP = 128, BK = 64, NTHREADS = 192, MAX_S = 8;
constexpr int P_BYTES = BP * BK * 2;

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
__global__ void __launch_bounds__(NTHREADS, 1) linear_split_kernel(const __grid_constant__ Maps maps,
                                                                   const __grid_constant__ Params p) {
  using C = Cfg<BT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NST;
  uint64_t* afull = empty + C::NST;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits, rank = (int)(blockIdx.x % S), tile = (int)(blockIdx.x / S);
  const int p0 = (tile % p.tp) * BP, q0 = (tile / p.tp) * BT;
  const int kb0 = (int)((int64_t)p.nkb * rank / S), kb1 = (int)((int64_t)p.nkb * (rank + 1) / S);

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
  // the cluster's CTAs have started once this phase completes (waited for before the exchange)
  if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  if (warp == 4) {
    if (lane == 0) {
      for (int i = kb0; i < kb1; ++i) {
        const int j = i - kb0, s = j % C::NST;
        if (!mbar_wait(&empty[s], ((uint32_t)(j / C::NST) & 1u) ^ 1u, 431)) break;
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
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t id = idesc_bf16(BP, BT, PMN, QMN);
      for (int i = kb0; i < kb1; ++i) {
        const int j = i - kb0, s = j % C::NST;
        if (!mbar_wait(&full[s], (uint32_t)(j / C::NST) & 1u, 531)) break;
        tc_fence_after();
        const uint32_t pb = smem_u32(smem + s * C::STAGE), qb = pb + P_BYTES;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint64_t pd = PMN ? smem_desc(pb + kk * 2048, 8192, 1024, 2) : smem_desc(pb + kk * 32, 16, 1024, 2);
          const uint64_t qd = QMN ? smem_desc(qb + kk * 2048, 8192, 1024, 2) : smem_desc(qb + kk * 32, 16, 1024, 2);
          tc_mma(tmem, pd, qd, id, (j | kk) != 0);
        }
        tc_commit(&empty[s]);
      }
      tc_commit(afull);  // also when a wait gave up: the epilogue is not left waiting
    }
    __syncwarp();
  }
  if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int per = BT / S;  // output rows this CTA finishes
  if (warp < 4) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(afull, 0, 731));
    tc_fence_after();
    if (ok) {
      const uint32_t lb = (uint32_t)(warp * 32) << 16;
      const int col = warp * 32 + lane;
#pragma unroll
      for (int c = 0; c < BT; c += 16) {
        float v[16];
        tmem_ld16(tmem + lb + (uint32_t)c, v);
        tc_wait_ld();
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const int r = c + t;  // row of the tile: finished by rank r / per
          float* dst = reinterpret_cast<float*>(smem + C::OFF_X) + (rank * per + r % per) * BP + col;
          if (S == 1) {
            *dst = v[t];
          } else {
            uint32_t a;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(dst)), "r"(r / per));
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v[t]) : "memory");
          }
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
  for (int it = threadIdx.x; it < per * (BP / 8); it += NTHREADS) {
    const int r = it / (BP / 8), c = (it % (BP / 8)) * 8;
    const int q = q0 + rank * per + r, col = p0 + c;
    if (q >= p.Q || col >= p.P) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    for (int k = 0; k < S; ++k) {  // rank order
      const float4* a = reinterpret_cast<const float4*>(xs + (k * per + r) * BP + c);
      const float4 lo = a[0], hi = a[1];
      v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
      v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
    }
    finish8(v, p.e, (int64_t)q * p.P + col, col);
  }
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
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(clusters * p.splits));
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = Cfg<BT>::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)p.splits;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  LSQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, linear_split_kernel<PMN, QMN, BT>, maps, p));
  return LSQ_OK;
}

// out[Q, P] = sum over C of the operands (see the top), with the epilogue e
template <int PMN, int QMN>
static lsq_status product(const void* pop, const void* qop, int64_t P, int64_t Q, int64_t C, const Epi& e,
                          cudaStream_t stream) {
  const int bt = QMN ? (Q <= 64 ? 64 : 128) : Q <= 16 ? 16 : Q <= 32 ? 32 : Q <= 64 ? 64 : 128;
  Params p{};
  p.P = (int)P;
  p.Q = (int)Q;
  p.nkb = (int)((C + BK - 1) / BK);  // the tail reads as zeros (TMA out-of-bounds fill)
  p.tp = (int)((P + BP - 1) / BP);
  p.e = e;
  const int64_t tiles = (int64_t)p.tp * ((Q + bt - 1) / bt);
  p.splits = 1;
  while (p.splits < MAX_S && tiles * p.splits * 2 <= num_sms() && p.nkb >= p.splits * 4) p.splits *= 2;
  Maps maps;
  memset(&maps, 0, sizeof(maps));
  lsq_status st = map_operand(&maps.p, pop, PMN, P, C, BP);
  if (st == LSQ_OK) st = map_operand(&maps.q, qop, QMN, Q, C, bt);
  if (st != LSQ_OK) return st;
  if constexpr (!QMN) {
    if (bt == 16) return launch_split<PMN, QMN, 16>(maps, p, tiles, stream);
    if (bt == 32) return launch_split<PMN, QMN, 32>(maps, p, tiles, stream);
  }
  if (bt == 64) return launch_split<PMN, QMN, 64>(maps, p, tiles, stream);
  return launch_split<PMN, QMN, 128>(maps, p, tiles, stream);
}

// ---------------------------------------------------------------- dz and db
// dz = dy act'(z) (bf16: the products' operand type) and, from the fp32 dz, the sums over a strip of rows;
// a warp covers 256 columns of a row (16 bytes a lane), a block's eight warps take rows in turn, and the
// strips' sums are added in order by col_sum_kernel.
template <int ACT>
__global__ void __launch_bounds__(256) dz_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ z,
                                                 uint4* __restrict__ dz, float* __restrict__ part, int64_t rows, int n8,
                                                 int64_t strip) {
  __shared__ float comb[8][32][9];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + l;
  const int64_t r0 = blockIdx.y * strip, r1 = r0 + strip < rows ? r0 + strip : rows;
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.0f;
  if (c < n8) {
#pragma unroll 2
    for (int64_t r = r0 + w; r < r1; r += 8) {
      float d[8];
      unpack8(dy[r * n8 + c], d);
      if (ACT != LSQ_ACT_NONE) {
        float zv[8];
        unpack8(z[r * n8 + c], zv);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= dact_f<ACT>(zv[j]);
        dz[r * n8 + c] = pack8(d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += d[j];
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) comb[w][l][j] = s[j];
  __syncthreads();
  if (w != 0 || c >= n8) return;
#pragma unroll
  for (int k = 1; k < 8; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += comb[k][l][j];
  float4* o = reinterpret_cast<float4*>(part + ((int64_t)blockIdx.y * n8 + c) * 8);
  o[0] = make_float4(s[0], s[1], s[2], s[3]);
  o[1] = make_float4(s[4], s[5], s[6], s[7]);
}

// row strips of dz_kernel: about eight blocks per SM, at least 8 rows each
static int64_t strips_of(int64_t M, int64_t N) {
  const int64_t cb = (N + 255) / 256;
  const int64_t want = std::max<int64_t>(1, (8 * num_sms() + cb - 1) / cb);
  const int64_t rows = std::max<int64_t>(8, (M + want - 1) / want);
  return (M + rows - 1) / rows;
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
  if (z && (z == y || z == residual)) return fail(LSQ_EINVAL, "%s: z must not alias y or residual", who);
  if ((st = check_device()) != LSQ_OK) return st;
  lin::Epi e{};
  e.bias = static_cast<const __nv_bfloat16*>(bias);
  e.residual = static_cast<const __nv_bfloat16*>(residual);
  e.z = static_cast<__nv_bfloat16*>(z);
  e.out = y;
  e.act = act;
  return lin::product<0, 0>(w, x, N, M, K, e, (cudaStream_t)stream);
}

extern "C" size_t lsq_linear_bwd_workspace_size(int64_t M, int64_t N, int64_t K, int32_t act) {
  if (M < 1 || N < 8 || K < 8) return 256;
  return (act == LSQ_ACT_NONE ? 0 : lin::round256((size_t)M * (size_t)N * 2)) +
         lin::round256((size_t)lin::strips_of(M, N) * (size_t)N * sizeof(float));
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
  if ((st = check_device()) != LSQ_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const void* dz = dy;
  if (pass) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (act != LSQ_ACT_NONE) {
      dz = ws;
      ws += lin::round256((size_t)M * (size_t)N * 2);
    }
    float* part = dbias ? reinterpret_cast<float*>(ws) : nullptr;
    const int64_t strips = lin::strips_of(M, N), strip = (M + strips - 1) / strips;
    const int ns = (int)((M + strip - 1) / strip);
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)ns);
    const uint4 *a = (const uint4*)dy, *b = (const uint4*)z;
    uint4* o = (uint4*)dz;
    const int n8 = (int)(N / 8);
    switch (act) {
      case LSQ_ACT_RELU: lin::dz_kernel<LSQ_ACT_RELU><<<grid, 256, 0, s>>>(a, b, o, part, M, n8, strip); break;
      case LSQ_ACT_GELU: lin::dz_kernel<LSQ_ACT_GELU><<<grid, 256, 0, s>>>(a, b, o, part, M, n8, strip); break;
      case LSQ_ACT_GELU_TANH: lin::dz_kernel<LSQ_ACT_GELU_TANH><<<grid, 256, 0, s>>>(a, b, o, part, M, n8, strip); break;
      case LSQ_ACT_SILU: lin::dz_kernel<LSQ_ACT_SILU><<<grid, 256, 0, s>>>(a, b, o, part, M, n8, strip); break;
      default: lin::dz_kernel<LSQ_ACT_NONE><<<grid, 256, 0, s>>>(a, b, nullptr, part, M, n8, strip); break;
    }
    LSQ_LAUNCH_CHECK("dz_kernel");
    if (dbias && (st = nrm::col_sum(part, ns, N, N, N, dbias, nullptr, accumulate ? 1 : 0, s)) != LSQ_OK) return st;
  }
  if (dx) {
    lin::Epi e{};
    e.out = dx;
    if ((st = lin::product<1, 0>(w, dz, K, M, N, e, s)) != LSQ_OK) return st;
  }
  if (dw) {
    lin::Epi e{};
    e.out = dw;
    e.f32 = dw_f32 ? 1 : 0;
    e.accumulate = accumulate ? 1 : 0;
    if ((st = lin::product<1, 1>(x, dz, K, N, M, e, s)) != LSQ_OK) return st;
  }
  return LSQ_OK;
}
