// Host-side helpers of the lsq library: error reporting, device checks, the
// NF4 codebook and its decision thresholds, TMA tensor-map encoding.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>

#include <atomic>

#include "../../include/lsq.h"

namespace lsq {

// Sets the thread's last-error message and returns s.
lsq_status fail(lsq_status s, const char* fmt, ...);
lsq_status cuda_fail(cudaError_t e, const char* what);

// Checks the current device is sm_100 (B200) once per device.
lsq_status check_device();

// Library codebook (16 ascending fp32 levels) and the 15 fp32 decision
// thresholds: code(x) = number of i with x >= thr[i].
const float* codebook();
const float* thresholds();

// 2-D tiled tensor map: dims {inner, outer} in elements, row pitch in bytes,
// box {box_inner, box_outer}; out-of-bounds elements read as zero.
lsq_status encode_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
                          uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                          CUtensorMapSwizzle swz);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// whether [a, a + na) and [b, b + nb) share a byte (no: either is NULL)
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

int num_sms();

extern std::atomic<uint64_t> g_launches;  // kernels that launch_chained has enqueued

// Launch with programmatic stream serialization (and a cluster size, where above 1): the kernel may be set up
// while its predecessor on the stream still runs, so it must call grid_wait (common.cuh).
template <typename... P, typename... A>
lsq_status launch_chained(const char* what, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                          unsigned cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e != cudaSuccess) return cuda_fail(e, what);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return LSQ_OK;
}

}  // namespace lsq

#define LSQ_CUDA_TRY(call)                                        \
  do {                                                            \
    cudaError_t e_ = (call);                                      \
    if (e_ != cudaSuccess) return ::lsq::cuda_fail(e_, #call);    \
  } while (0)

#define LSQ_LAUNCH_CHECK(what)                                          \
  do {                                                                  \
    cudaError_t e_ = cudaGetLastError();                                \
    if (e_ != cudaSuccess) return ::lsq::cuda_fail(e_, what);           \
  } while (0)
