// q8_attn_prompt.cu -- attention over whole prompts, packed one behind the other.
//
// A warp a row of q: its lanes hold the head's elements, each key's score is a sum over the warp, and the
// softmax runs along with it (a running maximum and sum).
#include "q8_attn_internal.h"
#include "q8_common.cuh"

namespace c3d {

constexpr int kRowThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kRowThreads) prompt_attn_kernel(const PromptParams p) {
  const long long id = (long long)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31, dim = p.head_dim;
  if (id >= (long long)p.q_rows * p.q_heads) return;
  const int head = (int)(id % p.q_heads), kv = head / (p.q_heads / p.kv_heads);
  const int row = (int)(id / p.q_heads);
  int seq = -1, begin = 0, end = 0;
  for (int b = 0; b < p.seqs && seq < 0; ++b) {
    begin = max(0, p.starts[b]);
    end = min(p.q_rows, p.starts[b + 1]);
    if (row >= begin && row < end) seq = b;
  }
  if (seq < 0) return;
  const int* ks = p.key_starts ? p.key_starts : p.starts;
  const int k0 = min(max(0, ks[seq]), p.k_rows), k1 = min(max(k0, ks[seq + 1]), p.k_rows), keys = k1 - k0;
  const int limit = p.causal ? min(keys, row - begin + 1 + keys - (end - begin)) : keys;
  const T* q = static_cast<const T*>(p.q.p) + row * p.q.pitch + head * p.q.head_pitch;
  float qf[4] = {}, o[4] = {};
  for (int i = 0; 32 * i + lane < dim; ++i) qf[i] = q8_to_float(q[32 * i + lane]) * p.scale * 1.44269504f;
  float top = -1e30f, sum = 0.0f;
  for (int s = 0; s < limit; ++s) {
    const T* k = static_cast<const T*>(p.k.p) + (k0 + s) * p.k.pitch + kv * p.k.head_pitch;
    const T* v = static_cast<const T*>(p.v.p) + (k0 + s) * p.v.pitch + kv * p.v.head_pitch;
    float x = 0.0f;
    for (int i = 0; 32 * i + lane < dim; ++i) x = fmaf(qf[i], q8_to_float(k[32 * i + lane]), x);
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
    const float now = fmaxf(top, x), keep = exp2f(top - now), pr = exp2f(x - now);
    top = now;
    sum = sum * keep + pr;
    for (int i = 0; 32 * i + lane < dim; ++i) o[i] = fmaf(pr, q8_to_float(v[32 * i + lane]), o[i] * keep);
  }
  T* out = static_cast<T*>(p.o.p) + row * p.o.pitch + head * p.o.head_pitch;
  for (int i = 0; 32 * i + lane < dim; ++i)
    out[32 * i + lane] = q8_from_float<T>(sum == 0.0f ? 0.0f : o[i] / sum);
}

cudaError_t launch_prompt_attn(const PromptParams& p, int value_type, cudaStream_t stream) {
  const long long rows = (long long)p.q_rows * p.q_heads;
  const unsigned blocks = (unsigned)((rows + kRowThreads / 32 - 1) / (kRowThreads / 32));
  if (value_type == Q8_BF16)
    prompt_attn_kernel<__nv_bfloat16><<<blocks, kRowThreads, 0, stream>>>(p);
  else
    prompt_attn_kernel<__half><<<blocks, kRowThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace c3d
