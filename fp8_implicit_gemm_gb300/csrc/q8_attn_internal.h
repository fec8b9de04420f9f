// q8_attn_internal.h -- what the host side and the kernels of the attention half of the quantised
// transformer path share.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "q8_attention.h"

namespace c3d {

// A validated cache.
struct Cache {
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  unsigned slots;        // pages * page_size
  int page_size, kv_heads, head_dim, code_type;
};

// A matrix of heads: element (token, head, i) at token * pitch + head * head_pitch + i.
struct Heads {
  void* p;
  long long pitch, head_pitch;
};

struct HeadsParams {
  Heads q, q_out, k, k_out, v;
  const void *q_weight, *k_weight;
  const unsigned long long* turns;
  const unsigned char* axis;
  const long long* positions;
  const long long* slots;
  Cache cache;
  long long positions_pitch;
  int tokens, q_heads, kv_heads, head_dim, rot_dim, axes, weight_type;
  float eps;
};
// code_type 0: no cache.
cudaError_t launch_heads(const HeadsParams& p, int value_type, int code_type, bool adjacent,
                         cudaStream_t stream);

struct ReadParams {
  Cache cache;
  const long long* slots;
  Heads k, v;
  int tokens;
};
cudaError_t launch_cache_read(const ReadParams& p, int value_type, cudaStream_t stream);

// Bits of an attention plan's status word.
constexpr int kAttnBadInput = 1, kAttnTimeout = 2;

struct CacheAttnParams {
  Cache cache;
  Heads q, o;
  const int *table, *lengths;
  long long table_pitch;
  int seqs, tokens, q_heads, table_width;
  float scale;
  int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
// Bytes that the runs of a plan need for the sums of heads that several blocks share.
size_t cache_attn_workspace(int sms, int tokens, int q_heads, int kv_heads, int dim);
cudaError_t cache_attn_setup(int code_type, int dim);  // the kernels' shared-memory grant on this device
cudaError_t launch_cache_attn(const CacheAttnParams& p, int value_type, void* workspace, int sms, cudaStream_t stream);

struct PromptParams {
  Heads q, k, v, o;
  const int *starts, *key_starts;
  int q_rows, k_rows, seqs, q_heads, kv_heads, head_dim, causal;
  int negate;            // the scale is negative
  float scale;           // its magnitude times log2(e)
  int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
cudaError_t prompt_attn_setup();       // the kernels' shared-memory grant on this device
cudaError_t launch_prompt_attn(const PromptParams& p, int value_type, cudaStream_t stream);

}  // namespace c3d
