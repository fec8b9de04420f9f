// q8_linear.cu -- products of 8-bit codes: y = scale_x * scale_w * (x * w^T) + bias.
#include "q8_common.cuh"

namespace c3d {

constexpr int kLinTile = 64, kLinK = 32;

// A 64 x 64 tile of y by 16 x 16 threads, 4 x 4 elements each, over K in steps of 32 codes.
template <bool kInt8>
__global__ void __launch_bounds__(256) linear_q8_kernel(const LinearParams p) {
  using Acc = typename std::conditional<kInt8, int, float>::type;
  __shared__ Acc sx[kLinK][kLinTile + 1], sw[kLinK][kLinTile + 1];
  const int tn = threadIdx.x & 15, tm = threadIdx.x >> 4;
  const long long m0 = (long long)blockIdx.y * kLinTile, n0 = (long long)blockIdx.x * kLinTile;
  Acc acc[4][4] = {};
  auto code = [](uint8_t c) -> Acc {
    if constexpr (kInt8) return (int)(int8_t)c;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
  };
  for (int k0 = 0; k0 < p.K; k0 += kLinK) {
    for (int i = threadIdx.x; i < kLinTile * kLinK; i += 256) {
      const int r = i / kLinK, k = i % kLinK;
      const bool in_k = k0 + k < p.K;
      sx[k][r] = in_k && m0 + r < p.M ? code(p.x[(m0 + r) * p.x_pitch + k0 + k]) : Acc(0);
      sw[k][r] = in_k && n0 + r < p.N ? code(p.w[(n0 + r) * p.w_pitch + k0 + k]) : Acc(0);
    }
    __syncthreads();
    for (int k = 0; k < kLinK; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += sx[k][tm + 16 * i] * sw[k][tn + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      float v = (float)acc[i][j] * p.scale_x[m] * p.scale_w[n];
      if (p.bias) v += q8_load_value(p.bias, p.bias_type, n);
      q8_store_value(p.y, p.y_type, m * p.y_pitch + n, v);
    }
}

cudaError_t launch_linear_q8(const LinearParams& p, int code_type, cudaStream_t stream) {
  const dim3 grid((p.N + kLinTile - 1) / kLinTile, (p.M + kLinTile - 1) / kLinTile);
  if (code_type == Q8_INT8)
    linear_q8_kernel<true><<<grid, 256, 0, stream>>>(p);
  else
    linear_q8_kernel<false><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace c3d
