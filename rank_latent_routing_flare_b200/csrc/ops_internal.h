// Argument checks shared by the entry points of include/flare_ops.h.
#pragma once

#include <atomic>
#include <cstdint>

#include "attention.h"
#include "flare_ops.h"
#include "host_internal.h"

namespace flare {

constexpr int64_t kMaxInt = 2147483647;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool row_width_ok(int64_t D) { return D == 16 || D == 32 || D == 64 || D == 128; }

// Strides of a [B][H][N][D] tensor of bf16 rows: every row starts on a
// 16-byte boundary; a dimension of size one has no stride (0 is stored); rows
// of an output do not share memory through a zero stride.
inline flare_status fill_strides(long (&out)[3], const void* base, const int64_t* s, int64_t B, int64_t H, int64_t N,
                                 int64_t D, bool is_output) {
  const int64_t n[3] = {B, H, N};
  if (!aligned16(base)) return FLARE_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    out[i] = n[i] == 1 ? 0 : static_cast<long>(s[i]);
    if (n[i] == 1) continue;
    if (s[i] % 8 != 0) return FLARE_ERR_ALIGN;
    if (s[i] < 0 || (s[i] != 0 && s[i] < D) || (is_output && s[i] == 0)) return FLARE_ERR_SHAPE;
    if (s[i] > (int64_t(1) << 38)) return FLARE_ERR_UNSUPPORTED;
  }
  return FLARE_OK;
}

// Lets a kernel use `bytes` of dynamic shared memory; set once per kernel and
// device (`Tag` is the kernel's own type), since setting it takes as long as
// half a launch.
template <typename Tag, typename Kernel>
inline cudaError_t allow_smem(Kernel* kern, int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launch of a kernel whose splits along the keys are a cluster (where there
// are few enough), or are joined by a kernel behind it.
template <typename Kernel, typename... Args>
inline cudaError_t launch_splits(Kernel* kern, dim3 grid, int threads, size_t smem, cudaStream_t s, dim3 cluster, int splits,
                                 const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster.x;
  attr.val.clusterDim.y = cluster.y;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = splits > 1 && splits <= kAttnClusterSplits ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace flare
