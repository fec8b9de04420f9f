// q8_linear_few.cu -- products of 8-bit codes for few tokens (a decoding step): w is read once,
// straight from global memory into registers, and its bytes are what bounds the time. Neither TMEM
// nor a workspace is used: allocating TMEM alone costs more than these products take.
//
// A block takes 16 channels; its warps share K in steps of 128 codes, so that one warp's loads cover
// 128 consecutive bytes of 8 rows, and add up through shared memory in a fixed order. A warp's
// product of 16 channels by 8 tokens is mma.sync m16n8k16 on f16, in which every code of either
// type is exact; the accumulator is fp32. The instruction's order of k is free as long as both
// operands use the same: thread t of a row takes 16 consecutive bytes, and MMA j of the four they
// feed takes bytes 4j..4j+3 of each.
#include "ptx.cuh"
#include "q8_common.cuh"

namespace c3d {

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewChannels = 16;
constexpr int kFewStep = 128;  // codes of K a warp takes at a time

// Two e4m3 codes to f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

template <bool kInt8>
__device__ __forceinline__ void codes_to_f16(const uint4& c, uint32_t* h) {
  if (kInt8) {
    int8_to_f16(c, h);
  } else {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[2 * i] = e4m3x2_to_f16(w[i] & 0xFFFFu);
      h[2 * i + 1] = e4m3x2_to_f16(w[i] >> 16);
    }
  }
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 16 bytes at column k of a row, zero past K (codes behind a row's end are not used, whatever
// they hold). k is a multiple of 16 and rows start on 16-byte boundaries, so a load that takes in a
// row's last code stays inside that code's aligned 16 bytes.
__device__ __forceinline__ uint4 load_codes(const uint8_t* row, int k, int K, bool ok) {
  if (!ok || k >= K) return make_uint4(0, 0, 0, 0);
  uint4 c = __ldg(reinterpret_cast<const uint4*>(row + k));
  const int left = K - k;
  if (left < 16) {
    uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int keep = left - 4 * i;
      if (keep <= 0)
        w[i] = 0;
      else if (keep < 4)
        w[i] &= (1u << (8 * keep)) - 1u;
    }
    c = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return c;
}

// kTiles: groups of 8 tokens.
template <bool kInt8, int kTiles>
__global__ void __launch_bounds__(kFewThreads) linear_q8_few_kernel(const LinearParams p) {
  __shared__ float part[kFewWarps][kTiles * 8][kFewChannels + 1];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const long long n0 = (long long)blockIdx.x * kFewChannels;
  const bool ok0 = n0 + g < p.N, ok1 = n0 + g + 8 < p.N;
  const uint8_t* w0 = p.w + (n0 + g) * p.w_pitch;
  const uint8_t* w1 = w0 + 8 * p.w_pitch;
  const uint8_t* xr[kTiles];
  bool xok[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    xok[i] = 8 * i + g < p.M;
    xr[i] = p.x + (long long)(8 * i + g) * p.x_pitch;
  }
  float acc[kTiles][4] = {};
  for (int k0 = warp * kFewStep; k0 < p.K; k0 += kFewWarps * kFewStep) {
    uint4 a[2][2], b[kTiles][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 64 * h + 16 * t;
      a[0][h] = load_codes(w0, k, p.K, ok0);
      a[1][h] = load_codes(w1, k, p.K, ok1);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) b[i][h] = load_codes(xr[i], k, p.K, xok[i]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t fa[2][8];
      codes_to_f16<kInt8>(a[0][h], fa[0]);
      codes_to_f16<kInt8>(a[1][h], fa[1]);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        uint32_t fb[8];
        codes_to_f16<kInt8>(b[i][h], fb);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_16816(acc[i], fa[0][2 * j], fa[1][2 * j], fa[0][2 * j + 1], fa[1][2 * j + 1],
                    fb[2 * j], fb[2 * j + 1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    part[warp][8 * i + 2 * t][g] = acc[i][0];
    part[warp][8 * i + 2 * t + 1][g] = acc[i][1];
    part[warp][8 * i + 2 * t][g + 8] = acc[i][2];
    part[warp][8 * i + 2 * t + 1][g + 8] = acc[i][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kTiles * 8 * kFewChannels; e += kFewThreads) {
    const int c = e & (kFewChannels - 1), m = e / kFewChannels;
    const long long n = n0 + c;
    if (m >= p.M || n >= p.N) continue;
    float v = part[0][m][c];
#pragma unroll
    for (int w = 1; w < kFewWarps; ++w) v += part[w][m][c];
    const ScaleBias sc{__ldg(p.scale_w + n),
                       p.bias ? q8_load_value(p.bias, p.bias_type, n) : 0.0f};
    q8_store_value(p.y, p.y_type, m * p.y_pitch + n, sc(v, __ldg(p.scale_x + m)));
  }
}

cudaError_t launch_linear_few(const LinearParams& p, int code_type, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.N + kFewChannels - 1) / kFewChannels));
  cfg.blockDim = dim3(kFewThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bool int8 = code_type == Q8_INT8;
  if (p.M <= 8)
    return int8 ? cudaLaunchKernelEx(&cfg, linear_q8_few_kernel<true, 1>, p)
                : cudaLaunchKernelEx(&cfg, linear_q8_few_kernel<false, 1>, p);
  return int8 ? cudaLaunchKernelEx(&cfg, linear_q8_few_kernel<true, 2>, p)
              : cudaLaunchKernelEx(&cfg, linear_q8_few_kernel<false, 2>, p);
}

}  // namespace c3d
