// q8_linear_few.cu -- products of 8-bit codes for few tokens (a decoding step): w is read once,
// straight from global memory into registers, and its bytes are what bounds the time. Neither TMEM
// nor a workspace is used: allocating TMEM alone costs more than these products take.
//
// A block takes 16 or 32 channels; its 4 to 16 warps share K in steps of 128 codes, so that one warp's
// loads cover 128 consecutive bytes of 8 rows, and add up through shared memory in a fixed order. The
// loads of a warp's next step are issued before this step's products. A warp's product of 16
// channels by 8 tokens is mma.sync m16n8k16 on f16, in which every code of either type is exact; the
// accumulator is fp32. The instruction's order of k is free as long as both operands use the same:
// thread t of a row takes 16 consecutive bytes, and MMA j of the four they feed takes bytes
// 4j..4j+3 of each.
#include "ptx.cuh"
#include "q8_common.cuh"

namespace c3d {

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
__device__ __forceinline__ uint4 load_codes_tail(const uint8_t* row, int k, int K) {
  if (k >= K) return make_uint4(0, 0, 0, 0);
  const uint4 c = __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const int left = K - k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int keep = left - 4 * i;
    if (keep <= 0)
      w[i] = 0;
    else if (keep < 4)
      w[i] &= (1u << (8 * keep)) - 1u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One step's codes of a warp: kCh x 16 channels and kTok x 8 tokens by 128 codes of K.
template <int kCh, int kTok>
struct FewStep {
  uint4 w[kCh][2][2], x[kTok][2];
};

// kCh: 16-channel groups of a block; kTok: 8-token groups of the product.
template <bool kInt8, int kCh, int kTok, int kFewWarps>
__global__ void __launch_bounds__(kFewWarps * 32) linear_q8_few_kernel(const LinearParams p) {
  constexpr int kChannels = 16 * kCh, kTokens = 8 * kTok;
  __shared__ float part[kFewWarps][kTokens][kChannels + 1];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const long long n0 = (long long)blockIdx.x * kChannels;
  // Rows past the last channel or token read the last one's codes: what they give is not stored, and
  // no load depends on a condition, which would make the compiler wait for it at once.
  const uint8_t* wrow[kCh][2];
  const uint8_t* xrow[kTok];
#pragma unroll
  for (int c = 0; c < kCh; ++c)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      wrow[c][r] = p.w + min(n0 + 16 * c + 8 * r + g, (long long)p.N - 1) * p.w_pitch + 16 * t;
#pragma unroll
  for (int i = 0; i < kTok; ++i) xrow[i] = p.x + (long long)min(8 * i + g, p.M - 1) * p.x_pitch + 16 * t;
  using Step = FewStep<kCh, kTok>;
  auto load = [&](Step& s, int k0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          s.w[c][r][h] = __ldg(reinterpret_cast<const uint4*>(wrow[c][r] + k0 + 64 * h));
#pragma unroll
      for (int i = 0; i < kTok; ++i)
        s.x[i][h] = __ldg(reinterpret_cast<const uint4*>(xrow[i] + k0 + 64 * h));
    }
  };
  float acc[kCh][kTok][4] = {};
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t fx[kTok][8];
#pragma unroll
      for (int i = 0; i < kTok; ++i) codes_to_f16<kInt8>(s.x[i][h], fx[i]);
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        uint32_t fw[2][8];
        codes_to_f16<kInt8>(s.w[c][0][h], fw[0]);
        codes_to_f16<kInt8>(s.w[c][1][h], fw[1]);
#pragma unroll
        for (int i = 0; i < kTok; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_16816(acc[c][i], fw[0][2 * j], fw[1][2 * j], fw[0][2 * j + 1], fw[1][2 * j + 1],
                      fx[i][2 * j], fx[i][2 * j + 1]);
      }
    }
  };
  constexpr int kStride = kFewWarps * kFewStep;
  const int whole = p.K / kFewStep * kFewStep;  // K in whole steps
  int k0 = warp * kFewStep;
  if (k0 < whole) {
    Step a, b;  // one in use, one on its way
    load(a, k0);
    while (true) {
      if (k0 + kStride < whole) load(b, k0 + kStride);
      multiply(a);
      k0 += kStride;
      if (k0 >= whole) break;
      if (k0 + kStride < whole) load(a, k0 + kStride);
      multiply(b);
      k0 += kStride;
      if (k0 >= whole) break;
    }
  }
  if (k0 == whole && whole < p.K) {  // the last, incomplete step, by the warp whose turn it is
    Step s;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = whole + 64 * h;  // the rows' pointers are 16 t bytes in
#pragma unroll
      for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) s.w[c][r][h] = load_codes_tail(wrow[c][r], k, p.K - 16 * t);
#pragma unroll
      for (int i = 0; i < kTok; ++i) s.x[i][h] = load_codes_tail(xrow[i], k, p.K - 16 * t);
    }
    multiply(s);
  }
#pragma unroll
  for (int c = 0; c < kCh; ++c)
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      part[warp][8 * i + 2 * t][16 * c + g] = acc[c][i][0];
      part[warp][8 * i + 2 * t + 1][16 * c + g] = acc[c][i][1];
      part[warp][8 * i + 2 * t][16 * c + g + 8] = acc[c][i][2];
      part[warp][8 * i + 2 * t + 1][16 * c + g + 8] = acc[c][i][3];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < kTokens * kChannels; e += kFewWarps * 32) {
    const int c = e % kChannels, m = e / kChannels;
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

template <bool kInt8, int kCh, int kTok, int kFewWarps>
static cudaError_t launch_one(const LinearParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.N + 16 * kCh - 1) / (16 * kCh)));
  cfg.blockDim = dim3(kFewWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_q8_few_kernel<kInt8, kCh, kTok, kFewWarps>, p);
}

template <bool kInt8>
static cudaError_t launch_few(const LinearParams& p, cudaStream_t stream) {
  // Channels and warps of a block, from sweeps of K = 256 to 16384 and N = 512 to 28672. 4864 and 9728
  // channels are a wave of 32-channel blocks, one and two an SM. Up to a wave, more warps share K where
  // it is long; past it, the last blocks of a wave leave SMs idle, the less the smaller a block is.
  // Up to 8 tokens, us, N x K int8, 16 channels on 4 warps / 32 on 4 / 32 on 8 / 32 on 16:
  //   4096 x 512  1.9 / 1.9 / 1.9 / 2.2      8192 x 2048  3.6 / 3.5 / 3.6 / 5.2
  //   4096 x 8192 13.1 / 14.2 / 8.5 / 6.7    8192 x 4096  8.0 / 8.6 / 6.7 / 8.3
  //   10240 x 1024 3.1 / 3.4 / 3.9 / 5.8     16384 x 4096 13.0 / 13.4 / 14.4 / 18.1
  // and 16 channels on 16 warps 2048 x 4096 3.2, where those take 3.8 / 4.3 / 3.5 / 3.7.
  const bool long_n = p.N > 9728;
  if (p.M <= 8) {
    if (p.N <= 2432)
      return p.K <= 1024 ? launch_one<kInt8, 1, 1, 4>(p, stream)
                         : launch_one<kInt8, 1, 1, 16>(p, stream);
    if (long_n && (kInt8 || p.K <= 512)) return launch_one<kInt8, 1, 1, 4>(p, stream);
    if (long_n || p.K <= 2048) return launch_one<kInt8, 2, 1, 4>(p, stream);
    return p.N <= 4864 ? launch_one<kInt8, 2, 1, 16>(p, stream) : launch_one<kInt8, 2, 1, 8>(p, stream);
  }
  // More tokens, whose x takes registers. 16 tokens, 16 channels on 4 warps / 16 on 8 / 32 on 4:
  //   4096 x 4096 4.7 / 4.5 / 5.1    8192 x 1024 3.4 / 4.4 / 3.9    10240 x 4096 15.6 / 14.4 / 11.4
  // and 2048 x 16384 16 on 8 / 16 on 16 13.4 / 8.9. 32 tokens, 16 on 8 / 32 on 4: 2048 x 4096 5.0 / 8.0,
  // 8192 x 1024 8.4 / 4.9.
  if (p.M <= 16) {
    if (p.N <= 2432 && p.K > 8192) return launch_one<kInt8, 1, 2, 16>(p, stream);
    if (p.N <= 4864) return launch_one<kInt8, 1, 2, 8>(p, stream);
    if constexpr (kInt8)
      if (long_n) return launch_one<kInt8, 2, 2, 4>(p, stream);
    return launch_one<kInt8, 1, 2, 4>(p, stream);
  }
  if constexpr (kInt8) {
    if (p.M <= 24)
      return p.N <= 4864 ? launch_one<kInt8, 1, 3, 8>(p, stream)
                         : launch_one<kInt8, 1, 3, 4>(p, stream);
    return p.N <= 2432 ? launch_one<kInt8, 1, 4, 8>(p, stream) : launch_one<kInt8, 2, 4, 4>(p, stream);
  }
  return cudaErrorInvalidValue;  // more than few_tokens
}

cudaError_t launch_linear_few(const LinearParams& p, int code_type, cudaStream_t stream) {
  return code_type == Q8_INT8 ? launch_few<true>(p, stream) : launch_few<false>(p, stream);
}

}  // namespace c3d
