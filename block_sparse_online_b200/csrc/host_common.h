// host_common.h -- host helpers that the entry points share: alignment, the device's
// properties, the tensor-map encoder, checks of pointers, and profiler ranges.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "solattn.h"

namespace solattn {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// NVTX range around the host code that enqueues one stage ("solattn pool", "solattn route",
// "solattn attention", ...), for timeline tools; without a tool attached it costs a few ns.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

struct DeviceInfo {
  int sms = 0;
  int major = 0;
  int devices = 0;  // GPUs of the process
  bool known = false;
};

inline std::mutex g_mu;
inline DeviceInfo g_dev[64];

inline int device_info(DeviceInfo *out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SOLATTN_ECUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_dev[dev].known) {
    int sms = 0, major = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SOLATTN_ECUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return SOLATTN_ECUDA;
    int devices = 0;
    if (cudaGetDeviceCount(&devices) != cudaSuccess) return SOLATTN_ECUDA;
    g_dev[dev].devices = devices;
    g_dev[dev].sms = sms;
    g_dev[dev].major = major;
    g_dev[dev].known = true;
  }
  *out = g_dev[dev];
  return SOLATTN_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// A device pointer that belongs to another GPU than the current one (the kernels would
// read or write it from the wrong device). Host, managed and unregistered pointers pass:
// the alignment and null checks above cover them, and managed memory is reachable.
inline bool foreign_device_pointer(const void *p, int dev) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();  // clear the sticky-free error of an unknown pointer
    return false;
  }
  return a.type == cudaMemoryTypeDevice && a.device != dev;
}

}  // namespace solattn
