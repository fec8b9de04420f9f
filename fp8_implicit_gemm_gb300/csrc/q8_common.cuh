// q8_common.cuh -- device pieces shared by the kernels of the 8-bit transformer path.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "q8_internal.h"

namespace c3d {

__device__ __forceinline__ float q8_to_float(float v) { return v; }
__device__ __forceinline__ float q8_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float q8_to_float(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T q8_from_float(float v);
template <>
__device__ __forceinline__ float q8_from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 q8_from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half q8_from_float<__half>(float v) { return __float2half_rn(v); }

// The value of one element whose type is known only at run time (a bias, a norm's weight).
__device__ __forceinline__ float q8_load_value(const void* p, int type, long long i) {
  if (type == Q8_F32) return __ldg(static_cast<const float*>(p) + i);
  if (type == Q8_BF16) return q8_to_float(static_cast<const __nv_bfloat16*>(p)[i]);
  return q8_to_float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void q8_store_value(void* p, int type, long long i, float v) {
  if (type == Q8_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == Q8_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

}  // namespace c3d
