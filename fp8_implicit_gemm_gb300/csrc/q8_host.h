// q8_host.h -- host-side checks and lookups shared by the C entry points of the quantised transformer path.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "q8.h"

namespace c3d {

inline bool value_type_ok(int t) { return t == Q8_F32 || t == Q8_BF16 || t == Q8_F16; }
inline bool code_type_ok(int t) { return t == Q8_INT8 || t == Q8_E4M3; }
inline int value_bytes(int t) { return t == Q8_F32 ? 4 : 2; }
inline long long round_up(long long a, long long b) { return (a + b - 1) / b * b; }
inline bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Puts the current device back at the end of a scope.
struct DeviceRestore {
  int prev = -1;
  DeviceRestore() {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
  }
  ~DeviceRestore() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

// Whether `device` is the current device and an sm_103.
inline conv3d_status check_device(int device) {
  int cur = -1, major = 0, minor = 0;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  if (cur != device) return CONV3D_EINVAL;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, cur) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, cur) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  return major == 10 && minor == 3 ? CONV3D_OK : CONV3D_EUNSUPPORTED;
}

// The status of a launch; its error, if any, is not left behind for the caller's next CUDA call.
inline conv3d_status launched(cudaError_t e) {
  if (e == cudaSuccess) return CONV3D_OK;
  cudaGetLastError();
  return CONV3D_ECUDA;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

}  // namespace c3d
