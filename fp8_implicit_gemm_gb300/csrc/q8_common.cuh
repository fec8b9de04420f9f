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

// Four int8 codes as f16 pairs in order. A code's byte with the sign bit flipped is u = code + 128;
// under the exponent byte 0x64 it is the f16 1024 + u, and 1024 + u - 1152 = code exactly.
__device__ __forceinline__ void int8_to_f16(uint32_t codes, uint32_t* h) {
  const __half2 bias = __floats2half2_rn(1152.0f, 1152.0f);
  const uint32_t u = codes ^ 0x80808080u;
  const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140);
  const uint32_t hi = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
  h[0] = *reinterpret_cast<const uint32_t*>(&a);
  h[1] = *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void int8_to_f16(const uint4& c, uint32_t* h) {
  int8_to_f16(c.x, h);
  int8_to_f16(c.y, h + 2);
  int8_to_f16(c.z, h + 4);
  int8_to_f16(c.w, h + 6);
}

// y's element from its sum: scaled by token and channel, the bias added (0 without one).
struct ScaleBias {
  float w, bias;
  __device__ __forceinline__ float operator()(float acc, float sx) const {
    return fmaf(acc * sx, w, bias);
  }
};

}  // namespace c3d
