// q8_internal.h -- what the host side and the kernels of the 8-bit transformer path share.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "q8.h"

namespace c3d {

// Validated arguments of the two row operators (one row of values in, one row of codes out).
struct RowsParams {
  const void* a;         // x, or gate
  const void* b;         // residual (null: none), or up
  const void* weight;    // norm only
  void* sum_out;         // norm with a residual: x + residual
  uint8_t* q;
  float* scale;
  long long a_pitch, b_pitch, sum_pitch, q_pitch;  // elements
  long long rows;
  int cols;
  float eps;
};

cudaError_t launch_rmsnorm_q8(const RowsParams& p, int value_type, int weight_type, int code_type,
                              cudaStream_t stream);
cudaError_t launch_silu_mul_q8(const RowsParams& p, int value_type, int code_type,
                               cudaStream_t stream);

// One product y = (x * w^T) scaled.
struct LinearParams {
  const uint8_t* x;
  const float* scale_x;
  const uint8_t* w;
  const float* scale_w;
  const void* bias;      // null: none
  void* y;
  long long x_pitch, w_pitch, y_pitch;
  int M, N, K;           // tokens, channels, summed length
  int y_type, bias_type;
};

cudaError_t launch_linear_q8(const LinearParams& p, int code_type, cudaStream_t stream);

}  // namespace c3d
