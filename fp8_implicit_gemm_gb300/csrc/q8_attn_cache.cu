// q8_attn_cache.cu -- attention of each sequence's newest tokens over a paged cache of codes.
//
// A warp a row of q: its lanes hold the head's elements, each key's score is a sum over the warp, and the
// softmax runs along with it (a running maximum and sum).
#include "q8_attn_internal.h"
#include "q8_common.cuh"

namespace c3d {

constexpr int kRowThreads = 128;

__device__ __forceinline__ float cache_value(const Cache& c, const uint8_t* codes, const float* scales,
                                             long long row, int i) {
  if (c.code_type == Q8_INT4) {
    const unsigned b = codes[(row * c.head_dim + i) / 2];
    return fmaf((float)((i & 1) ? b >> 4 : b & 15u), scales[2 * row], scales[2 * row + 1]);
  }
  const uint8_t b = codes[row * c.head_dim + i];
  if (c.code_type == Q8_INT8) return (float)(int8_t)b * scales[row];
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3))) * scales[row];
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) cache_attn_kernel(const CacheAttnParams p) {
  const long long id = (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31, dim = p.cache.head_dim;
  if (id >= (long long)p.seqs * p.tokens * p.q_heads) return;
  const int head = (int)(id % p.q_heads);
  const long long row = id / p.q_heads;
  const int seq = (int)(row / p.tokens), t = (int)(row % p.tokens);
  const int kv = head / (p.q_heads / p.cache.kv_heads), size = p.cache.page_size;
  const T* q = static_cast<const T*>(p.q.p) + row * p.q.pitch + head * p.q.head_pitch;
  float qf[8], o[8] = {};
  for (int i = 0; i < dim / 32; ++i) qf[i] = q8_to_float(q[32 * i + lane]) * p.scale * 1.44269504f;
  const int length = p.lengths[seq];
  bool bad = length < 0 || length > (long long)p.table_width * size;
  float top = -1e30f, sum = 0.0f;
  for (int s = 0; !bad && s < length - p.tokens + 1 + t; ++s) {
    const int page = p.table[seq * p.table_pitch + s / size];
    if (page < 0 || page >= (int)(p.cache.slots / size)) {
      bad = true;
      break;
    }
    const long long at = ((long long)page * p.cache.kv_heads + kv) * size + s % size;
    float x = 0.0f;
    for (int i = 0; i < dim / 32; ++i)
      x = fmaf(qf[i], cache_value(p.cache, p.cache.k_codes, p.cache.k_scale, at, 32 * i + lane), x);
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
    const float now = fmaxf(top, x), keep = exp2f(top - now), pr = exp2f(x - now);
    top = now;
    sum = sum * keep + pr;
    for (int i = 0; i < dim / 32; ++i)
      o[i] = fmaf(pr, cache_value(p.cache, p.cache.v_codes, p.cache.v_scale, at, 32 * i + lane), o[i] * keep);
  }
  if (bad && lane == 0) atomicOr(p.status, kAttnBadInput);
  T* out = static_cast<T*>(p.o.p) + row * p.o.pitch + head * p.o.head_pitch;
  for (int i = 0; i < dim / 32; ++i)
    out[32 * i + lane] =
        q8_from_float<T>(bad ? __int_as_float(0x7FFFFFFF) : sum == 0.0f ? 0.0f : o[i] / sum);
}

cudaError_t launch_cache_attn(const CacheAttnParams& p, int value_type, cudaStream_t stream) {
  const long long rows = (long long)p.seqs * p.tokens * p.q_heads;
  const unsigned blocks = (unsigned)((rows + kRowThreads / 32 - 1) / (kRowThreads / 32));
  if (value_type == Q8_BF16)
    cache_attn_kernel<__nv_bfloat16><<<blocks, kRowThreads, 0, stream>>>(p);
  else
    cache_attn_kernel<__half><<<blocks, kRowThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace c3d
