// q8_internal.h -- what the host side and the kernels of the 8-bit transformer path share.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
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
  int code_type, weight_type;
  int row_threads;       // threads that hold one row (set by the launcher)
  float eps;
};

// Where every row of all matrices starts: on 16 bytes (codes on 8), on a pair of elements with an even
// number of columns, or anywhere.
enum class RowsGrid { kChunk, kPair, kElement };
cudaError_t launch_rows_q8(RowsParams p, int value_type, bool norm, RowsGrid grid,
                           cudaStream_t stream);

// One product y = scale_x * scale_w * (x * w^T) + bias.
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
  int y_vec;             // four channels of y may be stored at once
  int y_tma;             // y's tiles may leave by TMA
  // the tensor-core kernel's tiling (linear_tc_decide) and workspace
  int block_t;           // tokens of a tile (a tile has kTcChannels channels)
  int m_tiles, n_tiles;
  int boxes, k_blocks;   // a K block is `boxes` boxes of kTcBlockK codes
  int splits;            // slices of K, one for each pair of a cluster: 1 to kTcMaxSplits
  int stages;
  int w_slots, x_slots;  // int8 only: boxes of w in TMEM and K blocks of x in shared memory, as f16
  uint16_t* xh;          // int8 only: x as f16, [M][xh_pitch]
  long long xh_pitch;
  int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};

// The kernel for few tokens takes up to this many; it needs no workspace.
constexpr int few_tokens(int code_type) { return code_type == Q8_INT8 ? 32 : 16; }
// Whether it is the faster one, from sweeps of K = 256 to 16384 and N = 512 to 28672. us, few tokens /
// tensor cores, N x K: e4m3 8 tokens 4096 x 8192 7.8 / 7.9, 10240 x 2048 5.9 / 5.8, 16384 x 2048 8.5 / 7.3,
// 10240 x 4096 12.3 / 10.1; 16 tokens 4096 x 4096 5.5 / 6.1, 4096 x 8192 11.1 / 8.3, 10240 x 512 3.5 / 3.8,
// 16384 x 1024 5.8 / 4.8. int8 8 tokens 28672 x 8192 39.0 / 44.4; 16 tokens 4096 x 8192 8.7 / 12.4,
// 8192 x 8192 16.1 / 17.8, 16384 x 4096 17.4 / 16.3; 24 tokens 4096 x 4096 6.7 / 8.8, 4096 x 8192 12.4 /
// 12.6; 32 tokens 4096 x 4096 8.1 / 8.9, 4096 x 8192 18.2 / 12.5, 10240 x 512 5.9 / 5.7.
inline bool prefer_few(long long M, long long N, long long K, int code_type) {
  if (M > few_tokens(code_type)) return false;
  const double codes = (double)N * (double)K;
  const bool long_n = N > 9728;  // more than a wave of blocks
  if (code_type == Q8_E4M3) {
    if (M <= 8) return codes <= (long_n ? 15e6 : 24e6);
    return codes <= (N > 4864 ? 10e6 : 20e6);
  }
  if (M <= 8) return true;
  if (M <= 16) return codes <= (long_n ? 60e6 : 70e6);
  if (M <= 24) return codes <= (long_n ? 10e6 : 20e6);
  return codes <= 20e6 && !long_n;
}
cudaError_t launch_linear_few(const LinearParams& p, int code_type, cudaStream_t stream);

// The tensor-core kernel: CTA pairs, tiles of 256 channels by block_t tokens.
constexpr int kTcChannels = 256;
constexpr int kTcBlockK = 128;         // codes of K in a box
constexpr int kTcMaxTokens = 256;
constexpr int kTcMaxSplits = 4;
// The most tokens of a tile: TMEM holds two accumulators, and for int8 two K blocks of w beside them.
// (One accumulator of 256 tokens and four K blocks took 193 us for 4096 x 8192 x 4096, where two of 160
// or 192 take 160: the epilogue's 8 us a tile are then not hidden.)
constexpr int tc_most_tokens(int code_type) { return code_type == Q8_INT8 ? 192 : kTcMaxTokens; }
// What a plan's device and options allow.
struct TcLimits {
  int clusters[kTcMaxSplits];  // clusters of 2, 4, 6 and 8 CTAs held at once
  int block_t, splits;   // 0: the choice of linear_tc_decide
};
// Fills in the tiling of a product of M, N and K; block_t stays 0 where the limits leave none.
void linear_tc_decide(LinearParams& p, int code_type, const TcLimits& lim);
// Boxes of the tensor maps: rows of w one CTA loads at a time (of x: half of block_t).
constexpr int kTcWBoxRows = 128;
// The box of y's map: 32 channels (a warp) of 2 KB worth of tokens.
constexpr int kTcYBoxBytes = 2048;
cudaError_t launch_linear_expand(const LinearParams& p, cudaStream_t stream);  // x -> xh
cudaError_t linear_tc_setup();         // the kernels' shared-memory grant
cudaError_t linear_tc_max_clusters(int (&clusters)[kTcMaxSplits]);
cudaError_t launch_linear_tc(const LinearParams& p, int code_type, const CUtensorMap& wmap,
                             const CUtensorMap& xmap, const CUtensorMap& ymap, const TcLimits& lim,
                             cudaStream_t stream);

}  // namespace c3d
