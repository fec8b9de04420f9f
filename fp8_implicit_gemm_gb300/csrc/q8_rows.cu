// q8_rows.cu -- the two operators that turn rows of values into 8-bit codes with a scale each: the
// root-mean-square norm with the residual's addition, and the gated activation.
//
// One reduction serves the norm. With v = h * weight and r = 1 / sqrt(sum(h^2)/cols + eps), the
// normed value is y = v * r, so amax(y) = r * amax(v) and the code y / (amax(y) / T) = v * T /
// amax(v): r cancels out of the codes and enters only the scale. The sum of squares and amax(v) are
// therefore taken in the same pass and reduced together.
#include "q8_common.cuh"

namespace c3d {

constexpr int kRowsThreads = 256;

// amax(|v|) as bits: unsigned order is the order of the magnitudes, and a NaN is above them all, so
// that one NaN or infinity marks the row.
struct RowStat {
  float sum;
  unsigned amax;
};

__device__ __forceinline__ RowStat row_reduce(RowStat s) {
  __shared__ RowStat warp_stat[kRowsThreads / 32];
  for (int o = 16; o > 0; o >>= 1) s.sum += __shfl_xor_sync(0xFFFFFFFFu, s.sum, o);
  s.amax = __reduce_max_sync(0xFFFFFFFFu, s.amax);
  if ((threadIdx.x & 31) == 0) warp_stat[threadIdx.x >> 5] = s;
  __syncthreads();
  s = warp_stat[0];
  for (int w = 1; w < kRowsThreads / 32; ++w) {
    s.sum += warp_stat[w].sum;
    s.amax = max(s.amax, warp_stat[w].amax);
  }
  return s;
}

__device__ __forceinline__ uint8_t row_code(float v, float inv, int code_type) {
  if (code_type == Q8_E4M3) return __nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, __NV_E4M3);
  return (uint8_t)(int8_t)max(-127, min(127, __float2int_rn(v * inv)));
}

// Codes and scale of the row of values v in shared memory; `gain` is what the codes' scale is
// multiplied by (the norm's r). A row that is not finite gets the scale NaN and codes 0.
__device__ __forceinline__ void row_write(const float* v, const RowStat& st, float gain,
                                          const RowsParams& p, long long row, int code_type) {
  const float top = code_type == Q8_E4M3 ? 448.0f : 127.0f;
  const bool bad = st.amax >= 0x7F800000u || !(st.sum < INFINITY);
  const float amax = __uint_as_float(st.amax);
  // a tiny amax is lifted first: top / amax would overflow
  const float lift = amax < 0x1p-100f ? 0x1p100f : 1.0f;
  const float inv = bad || amax == 0.0f ? 0.0f : top / (amax * lift);
  uint8_t* q = p.q + row * p.q_pitch;
  for (int c = threadIdx.x; c < p.cols; c += kRowsThreads)
    q[c] = bad ? 0 : row_code(v[c] * lift, inv, code_type);
  if (threadIdx.x == 0)
    p.scale[row] = bad ? __int_as_float(0x7FC00000) : (amax > 0.0f ? amax * gain / top : 1.0f);
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads)
    rmsnorm_q8_kernel(const RowsParams p, int weight_type, int code_type) {
  extern __shared__ float v[];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.a) + row * p.a_pitch;
  const T* res = p.b ? static_cast<const T*>(p.b) + row * p.b_pitch : nullptr;
  T* sum_out = p.b ? static_cast<T*>(p.sum_out) + row * p.sum_pitch : nullptr;
  RowStat st{0.0f, 0u};
  for (int c = threadIdx.x; c < p.cols; c += kRowsThreads) {
    float h = q8_to_float(x[c]);
    if (res) {
      h += q8_to_float(res[c]);
      sum_out[c] = q8_from_float<T>(h);
    }
    v[c] = h * q8_load_value(p.weight, weight_type, c);
    st.sum += h * h;
    st.amax = max(st.amax, __float_as_uint(fabsf(v[c])));
  }
  st = row_reduce(st);
  row_write(v, st, rsqrtf(st.sum / (float)p.cols + p.eps), p, row, code_type);
}

template <typename T>
__global__ void __launch_bounds__(kRowsThreads)
    silu_mul_q8_kernel(const RowsParams p, int code_type) {
  extern __shared__ float v[];
  const long long row = blockIdx.x;
  const T* gate = static_cast<const T*>(p.a) + row * p.a_pitch;
  const T* up = static_cast<const T*>(p.b) + row * p.b_pitch;
  RowStat st{0.0f, 0u};
  for (int c = threadIdx.x; c < p.cols; c += kRowsThreads) {
    const float g = q8_to_float(gate[c]);
    v[c] = g / (1.0f + __expf(-g)) * q8_to_float(up[c]);
    st.amax = max(st.amax, __float_as_uint(fabsf(v[c])));
  }
  st = row_reduce(st);
  row_write(v, st, 1.0f, p, row, code_type);
}

template <typename T>
static cudaError_t rmsnorm_typed(const RowsParams& p, int weight_type, int code_type,
                                 cudaStream_t stream) {
  const int smem = p.cols * 4;
  const cudaError_t e = cudaFuncSetAttribute(
      rmsnorm_q8_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8_MAX_COLS * 4);
  if (e != cudaSuccess) return e;
  rmsnorm_q8_kernel<T><<<(unsigned)p.rows, kRowsThreads, smem, stream>>>(p, weight_type, code_type);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t silu_mul_typed(const RowsParams& p, int code_type, cudaStream_t stream) {
  const int smem = p.cols * 4;
  const cudaError_t e = cudaFuncSetAttribute(
      silu_mul_q8_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8_MAX_COLS * 4);
  if (e != cudaSuccess) return e;
  silu_mul_q8_kernel<T><<<(unsigned)p.rows, kRowsThreads, smem, stream>>>(p, code_type);
  return cudaGetLastError();
}

cudaError_t launch_rmsnorm_q8(const RowsParams& p, int value_type, int weight_type, int code_type,
                              cudaStream_t stream) {
  if (value_type == Q8_F32) return rmsnorm_typed<float>(p, weight_type, code_type, stream);
  if (value_type == Q8_BF16) return rmsnorm_typed<__nv_bfloat16>(p, weight_type, code_type, stream);
  return rmsnorm_typed<__half>(p, weight_type, code_type, stream);
}

cudaError_t launch_silu_mul_q8(const RowsParams& p, int value_type, int code_type,
                               cudaStream_t stream) {
  if (value_type == Q8_F32) return silu_mul_typed<float>(p, code_type, stream);
  if (value_type == Q8_BF16) return silu_mul_typed<__nv_bfloat16>(p, code_type, stream);
  return silu_mul_typed<__half>(p, code_type, stream);
}

}  // namespace c3d
