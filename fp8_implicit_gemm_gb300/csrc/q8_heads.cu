// q8_heads.cu -- the heads' launch for every value type, the kernels of bfloat16 (q8_heads.cuh), and a cache's rows as values.
#include "q8_heads.cuh"

namespace c3d {

// in q8_heads_f32.cu and q8_heads_f16.cu
extern template cudaError_t launch_heads_in<float>(const HeadsParams&, int, bool, cudaStream_t);
extern template cudaError_t launch_heads_in<__half>(const HeadsParams&, int, bool, cudaStream_t);

cudaError_t launch_heads(const HeadsParams& p, int value_type, int code_type, bool adjacent,
                         cudaStream_t stream) {
  if (value_type == Q8_F32) return launch_heads_in<float>(p, code_type, adjacent, stream);
  if (value_type == Q8_BF16) return launch_heads_in<__nv_bfloat16>(p, code_type, adjacent, stream);
  return launch_heads_in<__half>(p, code_type, adjacent, stream);
}

// ------------------------------------------------------------------ rows of a cache as values
// A lane reads eight codes and writes eight values; a block takes one head's k or v of consecutive tokens,
// so that neighbouring rows of a page are read together.
constexpr int kReadRows = 4;  // rows a lane has under way

template <typename T, int CODE, int L>
__global__ void __launch_bounds__(kHeadsThreads) cache_read_kernel(const ReadParams p) {
  constexpr int kRows = kHeadsThreads / L;
  const Cache& c = p.cache;
  // k and v of all heads by turns: blocks that run at the same time write neighbouring rows
  const unsigned side = blockIdx.x % (2u * c.kv_heads), tokens = blockIdx.x / (2u * c.kv_heads);
  const bool is_v = (int)side >= c.kv_heads;
  const int head = side - (is_v ? c.kv_heads : 0);
  const uint8_t* codes = is_v ? c.v_codes : c.k_codes;
  const float* scales = is_v ? c.v_scale : c.k_scale;
  const Heads& out = is_v ? p.v : p.k;
  const int chunk = threadIdx.x % L;
  const long long t0 = (long long)tokens * (kRows * kReadRows) + threadIdx.x / L;
  long long row[kReadRows];
  uint2 word[kReadRows];
  float2 scale[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const long long t = t0 + i * kRows;
    const long long slot = t < p.tokens ? p.slots[t] : -1;
    row[i] = -1;
    if (slot >= 0 && slot < (long long)c.slots) {
      const unsigned page = (unsigned)slot / (unsigned)c.page_size;
      row[i] = ((long long)page * c.kv_heads + head) * c.page_size +
               ((unsigned)slot - page * c.page_size);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (row[i] < 0) continue;
    if constexpr (CODE == Q8_INT4) {
      word[i].x = *reinterpret_cast<const unsigned*>(codes + (row[i] * L + chunk) * (kLane / 2));
      scale[i] = *reinterpret_cast<const float2*>(scales + 2 * row[i]);
    } else {
      word[i] = *reinterpret_cast<const uint2*>(codes + (row[i] * L + chunk) * kLane);
      scale[i].x = scales[row[i]];
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (row[i] < 0) continue;
    float f[kLane];
    if constexpr (CODE == Q8_INT4) {
#pragma unroll
      for (int e = 0; e < kLane; ++e)
        f[e] = fmaf((float)((word[i].x >> (4 * e)) & 15u), scale[i].x, scale[i].y);
    } else if constexpr (CODE == Q8_INT8) {
#pragma unroll
      for (int e = 0; e < kLane; ++e) {
        const unsigned w = e < 4 ? word[i].x : word[i].y;
        f[e] = (float)(int8_t)(w >> (8 * (e % 4))) * scale[i].x;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLane; e += 2) {
        const unsigned w = e < 4 ? word[i].x : word[i].y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (8 * (e % 4))),
                                                         __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        f[e] = v.x * scale[i].x;
        f[e + 1] = v.y * scale[i].x;
      }
    }
    store8(static_cast<T*>(out.p) + (t0 + i * kRows) * out.pitch + head * out.head_pitch +
               chunk * kLane, f);
  }
}

template <typename T, int CODE>
cudaError_t launch_read_of(const ReadParams& p, cudaStream_t stream) {
  const int lanes = p.cache.head_dim / kLane, rows = kHeadsThreads / lanes * kReadRows;
  const long long blocks = ((long long)p.tokens + rows - 1) / rows * 2 * p.cache.kv_heads;
  const unsigned grid = (unsigned)blocks;
  if (lanes == 8)
    cache_read_kernel<T, CODE, 8><<<grid, kHeadsThreads, 0, stream>>>(p);
  else if (lanes == 16)
    cache_read_kernel<T, CODE, 16><<<grid, kHeadsThreads, 0, stream>>>(p);
  else
    cache_read_kernel<T, CODE, 32><<<grid, kHeadsThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_read_in(const ReadParams& p, cudaStream_t stream) {
  switch (p.cache.code_type) {
    case Q8_INT8: return launch_read_of<T, Q8_INT8>(p, stream);
    case Q8_E4M3: return launch_read_of<T, Q8_E4M3>(p, stream);
    default: return launch_read_of<T, Q8_INT4>(p, stream);
  }
}

cudaError_t launch_cache_read(const ReadParams& p, int value_type, cudaStream_t stream) {
  if (value_type == Q8_F32) return launch_read_in<float>(p, stream);
  if (value_type == Q8_BF16) return launch_read_in<__nv_bfloat16>(p, stream);
  return launch_read_in<__half>(p, stream);
}

}  // namespace c3d
