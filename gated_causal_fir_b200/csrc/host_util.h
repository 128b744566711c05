// host_util.h -- host-side helpers shared by the translation units of the library.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

namespace hyena {
namespace host {

// The current device's status word (device memory of the library) and SM count, looked up once
// per device; HYENA_OK or HYENA_ERR_CUDA.  Defined in hyena_conv.cu.
struct DeviceInfo {
  unsigned int *status;
  int sm_count;
};
__attribute__((visibility("hidden"))) int device_info(DeviceInfo *out);

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
__attribute__((visibility("hidden"))) EncodeTiledFn encode_tiled();

inline bool aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Whether [a, a + na) and [b, b + nb) share a byte (null pointers share none).
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

inline int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Launch with programmatic stream serialisation: the kernel waits (griddepcontrol.wait) before
// its first access to global memory.  In clusters of `cluster` CTAs where that is not 1.
template <typename... Exp, typename... Act>
cudaError_t launch_in_clusters(unsigned cluster, void (*kernel)(Exp...), dim3 grid, dim3 block,
                               size_t smem, cudaStream_t s, Act &&...args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Act>(args)...);
}
template <typename... Exp, typename... Act>
cudaError_t launch(void (*kernel)(Exp...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                   Act &&...args) {
  return launch_in_clusters(1, kernel, grid, block, smem, s, std::forward<Act>(args)...);
}

}  // namespace host
}  // namespace hyena
