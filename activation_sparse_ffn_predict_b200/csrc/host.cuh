// Host-side helpers shared by the library's source files: the launch every
// kernel goes through, the device's SM count, and the argument checks.
#pragma once

#include <cuda.h>            // CUtensorMap and its encoder's types (the encoder comes from the runtime)
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "asffn.h"
#include "common.cuh"

namespace asf {

struct DevCache {
  int sms = 0;
};
inline std::mutex g_mu;
inline DevCache g_dev[64];

inline int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_dev[dev].sms == 0) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
    g_dev[dev].sms = v;
  }
  return g_dev[dev].sms;
}

// The attributes a kernel was last given on a device, so that a launch does not
// set them again (1 us of host time per launch).
struct KernelAttrs {
  size_t smem = 0;
};
inline std::map<std::pair<const void *, int>, KernelAttrs> g_attrs;

// Every kernel prefers the largest shared-memory carveout: an SM then never
// has to be reconfigured between the chained kernels, and a kernel can start
// beside one that uses less than all of it (the layer-2 predictor beside the
// layer-1 slice kernel: +1.7% tokens/s at the 70B shape).
inline cudaError_t prepare_kernel(const void *kern, size_t smem, bool again) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_attrs.find({kern, dev});
  const bool known = it != g_attrs.end();
  if (known && !again && it->second.smem >= smem) return cudaSuccess;
  if (smem > 40 * 1024) {   // 48 KB without asking, a kernel's static part included
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
  try {
    KernelAttrs &k = g_attrs[{kern, dev}];
    k.smem = again ? smem : std::max(k.smem, smem);
  } catch (...) {              // no memory to note it: set again by the next launch
  }
  return cudaSuccess;
}

// cluster: CTAs of a thread-block cluster along x (1: none)
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, int cluster,
                            Args... args) {
  cudaError_t e = prepare_kernel((const void *)kern, smem, false);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  if (e == cudaErrorInvalidValue || e == cudaErrorLaunchOutOfResources) {
    // a device that was reset has forgotten the attributes: once more with them
    cudaGetLastError();
    e = prepare_kernel((const void *)kern, smem, true);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  }
  return e;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  return launch_clusters(kern, grid, block, smem, st, 1, args...);
}

inline bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
inline size_t r256(size_t v) { return (v + 255) & ~size_t(255); }
inline asf_status check_ws(void *ws, size_t ws_bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return ASF_ERR_WORKSPACE;
  if (ws_bytes < need) return ASF_ERR_WORKSPACE;
  return ASF_OK;
}

inline asf_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ASF_OK : ASF_ERR_CUDA; }

// cuTensorMapEncodeTiled, from the driver through the runtime (no link to the
// driver library).
using TmapEncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline TmapEncodeFn tmap_encoder() {
  static TmapEncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (TmapEncodeFn) nullptr;
    return reinterpret_cast<TmapEncodeFn>(p);
  }();
  return fn;
}

}  // namespace asf
