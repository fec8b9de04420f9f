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

// Two fp32 operations by one instruction, for code that is bound by its issue.
__device__ __forceinline__ float2 q8_add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 q8_mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 q8_fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Two values rounded to a 16-bit type, the first in the low half.
template <typename Y>
__device__ __forceinline__ uint32_t q8_pack2(float2 v);
template <>
__device__ __forceinline__ uint32_t q8_pack2<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t q8_pack2<__half>(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// y's element from its sum: scaled by token and channel, the bias added (0 without one).
struct ScaleBias {
  float w, bias;
  __device__ __forceinline__ float operator()(float acc, float sx) const {
    return fmaf(acc * sx, w, bias);
  }
};

}  // namespace c3d
