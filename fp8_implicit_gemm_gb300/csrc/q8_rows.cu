// q8_rows.cu -- the two operators that turn rows of values into 8-bit codes with a scale each: the
// root-mean-square norm with the residual's addition, and the gated activation.
//
// One reduction serves the norm. With v = h * weight and r = 1 / sqrt(sum(h^2)/cols + eps), the
// normed value is y = v * r, so amax(y) = r * amax(v) and the code y / (amax(y) / T) = v * T /
// amax(v): r cancels out of the codes and enters only the scale. The sum of squares and amax(v) are
// therefore taken in the same pass, reduced together, and the row's values stay in registers: every
// input is read once, every output written once, which is the operator's floor (both are bound by
// the memory's bandwidth, and by one row's latency when there are few rows).
#include "ptx.cuh"
#include "q8_common.cuh"

namespace c3d {

constexpr int kChunk = 8;  // values a thread takes at a time: 16 bytes of a 16-bit type

// amax(|v|) as bits: unsigned order is the order of the magnitudes, and a NaN is above them all, so
// that one NaN or infinity marks the row.
struct RowStat {
  float sum;
  unsigned amax;
};

__device__ __forceinline__ RowStat warp_reduce(RowStat s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s.sum += __shfl_xor_sync(0xFFFFFFFFu, s.sum, o);
  s.amax = __reduce_max_sync(0xFFFFFFFFu, s.amax);
  return s;
}

// Over the threads of one row: a warp, or the whole block.
__device__ __forceinline__ RowStat row_reduce(RowStat s, int threads) {
  s = warp_reduce(s);
  if (threads == 32) return s;
  __shared__ RowStat warp_stat[32];
  const int lane = threadIdx.x & 31;
  if (lane == 0) warp_stat[threadIdx.x >> 5] = s;
  __syncthreads();
  s = lane < threads / 32 ? warp_stat[lane] : RowStat{0.0f, 0u};
  return warp_reduce(s);
}

// Eight consecutive values at p (16-byte aligned) as fp32.
__device__ __forceinline__ void load8(const float* p, float (&v)[kChunk]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[kChunk]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[kChunk]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kChunk]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kChunk]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[kChunk]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a thread's kChunk values of step i lie. Aligned rows: consecutive columns, moved by 16-byte
// accesses (the row's last, incomplete chunk by single elements). Other rows (a base, a pitch or a
// weight off the 16-byte grid): columns one row-team apart, moved one by one, so that a warp still
// touches consecutive addresses.
template <bool kAligned>
struct Place {
  int tid, threads, cols;
  __device__ __forceinline__ int col(int i, int e) const {
    return kAligned ? (i * threads + tid) * kChunk + e : (i * kChunk + e) * threads + tid;
  }
  __device__ __forceinline__ bool whole(int i) const {
    return kAligned && col(i, 0) + kChunk <= cols;
  }
  // Columns past the row's end read 0, which changes neither a sum of squares nor an amax.
  template <typename T>
  __device__ __forceinline__ void load(const T* row, int i, float (&v)[kChunk]) const {
    if (whole(i)) {
      load8(row + col(i, 0), v);
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        v[e] = col(i, e) < cols ? q8_to_float(row[col(i, e)]) : 0.0f;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int i, const float (&v)[kChunk]) const {
    if (whole(i)) {
      store8(row + col(i, 0), v);
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col(i, e) < cols) row[col(i, e)] = q8_from_float<T>(v[e]);
    }
  }
  __device__ __forceinline__ void store_codes(uint8_t* row, int i, uint2 c) const {
    if (whole(i)) {
      *reinterpret_cast<uint2*>(row + col(i, 0)) = c;
    } else {
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        if (col(i, e) < cols) row[col(i, e)] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
    }
  }
};

// Four int8 codes of values |v * inv| <= 127 (and a rounding error): adding 1.5 * 2^23 rounds the
// fused product to an integer, ties to even, whose low byte is the code.
__device__ __forceinline__ uint32_t int8_codes(const float* v, float inv) {
  uint32_t n[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) n[i] = __float_as_uint(fmaf(v[i], inv, 12582912.0f));
  return __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t e4m3_codes(const float* v, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv),
                                               __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xFFFFu) | (hi << 16);
}

// Codes and scale of one row whose values the threads hold; `gain` is what the scale is multiplied
// by (the norm's r). A row that is not finite gets the scale NaN and codes 0.
template <int NV, bool kAligned>
__device__ __forceinline__ void row_write(float (&v)[NV][kChunk], const RowStat& st, float gain,
                                          const RowsParams& p, long long row,
                                          const Place<kAligned>& at) {
  const float top = p.code_type == Q8_E4M3 ? 448.0f : 127.0f;
  const bool bad = st.amax >= 0x7F800000u || !(st.sum < INFINITY);
  const float amax = __uint_as_float(st.amax);
  uint8_t* q = p.q + row * p.q_pitch;
  if (at.tid == 0)
    p.scale[row] = bad ? __int_as_float(0x7FC00000) : (amax > 0.0f ? amax * gain / top : 1.0f);
  float inv = top / amax;
  if (bad || amax < 0x1p-100f) {  // rows that are no numbers, zeros, or so small that top / amax
    const bool zero = bad || amax == 0.0f;  // would overflow: those are lifted first
    inv = zero ? 0.0f : top / (amax * 0x1p100f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[i][e] = zero ? 0.0f : v[i][e] * 0x1p100f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint2 c = p.code_type == Q8_E4M3
                        ? make_uint2(e4m3_codes(v[i], inv), e4m3_codes(v[i] + 4, inv))
                        : make_uint2(int8_codes(v[i], inv), int8_codes(v[i] + 4, inv));
    at.store_codes(q, i, c);
  }
}

// The row this thread works on: one a block, or one a warp when a warp holds a row.
__device__ __forceinline__ long long my_row(const RowsParams& p) {
  return p.row_threads == 32 ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                             : (long long)blockIdx.x;
}

template <typename T, int NV, bool kAligned>
__global__ void __launch_bounds__(NV >= 4 ? 512 : 1024) rmsnorm_q8_kernel(const RowsParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const long long row = my_row(p);
  if (row >= p.rows) return;  // whole warps, of blocks that hold a row a warp
  const Place<kAligned> at{p.row_threads == 32 ? (int)(threadIdx.x & 31) : (int)threadIdx.x,
                           p.row_threads, p.cols};
  const T* x = static_cast<const T*>(p.a) + row * p.a_pitch;
  float v[NV][kChunk];
#pragma unroll
  for (int i = 0; i < NV; ++i) at.load(x, i, v[i]);
  if (p.b) {
    const T* res = static_cast<const T*>(p.b) + row * p.b_pitch;
    T* sum_out = static_cast<T*>(p.sum_out) + row * p.sum_pitch;
    // all of the residual's loads in flight at once, where registers hold them
    constexpr int kAhead = kAligned && NV <= 4 ? NV : 1;
    float r[kAhead][kChunk];
#pragma unroll
    for (int i0 = 0; i0 < NV; i0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) at.load(res, i0 + i, r[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[i0 + i][e] += r[i][e];
        at.store(sum_out, i0 + i, v[i0 + i]);  // columns this thread has read, if x's or residual's
      }
    }
  }
  RowStat st{0.0f, 0u};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[kChunk];
    if (p.weight_type == Q8_F32)
      at.load(static_cast<const float*>(p.weight), i, w);
    else if (p.weight_type == Q8_BF16)
      at.load(static_cast<const __nv_bfloat16*>(p.weight), i, w);
    else
      at.load(static_cast<const __half*>(p.weight), i, w);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      st.sum = fmaf(v[i][e], v[i][e], st.sum);
      v[i][e] *= w[e];
      st.amax = max(st.amax, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
    }
  }
  st = row_reduce(st, p.row_threads);
  row_write<NV, kAligned>(v, st, rsqrtf(st.sum / (float)p.cols + p.eps), p, row, at);
}

template <typename T, int NV, bool kAligned>
__global__ void __launch_bounds__(NV >= 4 ? 512 : 1024) silu_mul_q8_kernel(const RowsParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const long long row = my_row(p);
  if (row >= p.rows) return;
  const Place<kAligned> at{p.row_threads == 32 ? (int)(threadIdx.x & 31) : (int)threadIdx.x,
                           p.row_threads, p.cols};
  const T* gate = static_cast<const T*>(p.a) + row * p.a_pitch;
  const T* up = static_cast<const T*>(p.b) + row * p.b_pitch;
  float v[NV][kChunk], u[NV][kChunk];
#pragma unroll
  for (int i = 0; i < NV; ++i) at.load(gate, i, v[i]);
#pragma unroll
  for (int i = 0; i < NV; ++i) at.load(up, i, u[i]);
  RowStat st{0.0f, 0u};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const float g = v[i][e];
      v[i][e] = __fdividef(g, 1.0f + __expf(-g)) * u[i][e];
      st.amax = max(st.amax, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
    }
  st = row_reduce(st, p.row_threads);
  row_write<NV, kAligned>(v, st, 1.0f, p, row, at);
}

// One row a block of 32..1024 threads, or four rows a block of four warps when a warp holds a row.
template <typename Kernel>
static cudaError_t launch_rows(Kernel kernel, const RowsParams& p, cudaStream_t stream) {
  const bool warp_rows = p.row_threads == 32;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(warp_rows ? (p.rows + 3) / 4 : p.rows));
  cfg.blockDim = dim3(warp_rows ? 128 : p.row_threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, bool kAligned>
static cudaError_t launch_typed(const RowsParams& p, bool norm, int nv, cudaStream_t stream) {
  if (norm) {
    if (nv == 1) return launch_rows(rmsnorm_q8_kernel<T, 1, kAligned>, p, stream);
    if (nv == 2) return launch_rows(rmsnorm_q8_kernel<T, 2, kAligned>, p, stream);
    if (nv == 4) return launch_rows(rmsnorm_q8_kernel<T, 4, kAligned>, p, stream);
    return launch_rows(rmsnorm_q8_kernel<T, 8, kAligned>, p, stream);
  }
  if (nv == 1) return launch_rows(silu_mul_q8_kernel<T, 1, kAligned>, p, stream);
  if (nv == 2) return launch_rows(silu_mul_q8_kernel<T, 2, kAligned>, p, stream);
  if (nv == 4) return launch_rows(silu_mul_q8_kernel<T, 4, kAligned>, p, stream);
  return launch_rows(silu_mul_q8_kernel<T, 8, kAligned>, p, stream);
}

cudaError_t launch_rows_q8(RowsParams p, int value_type, bool norm, bool aligned,
                           cudaStream_t stream) {
  const int chunks = (p.cols + kChunk - 1) / kChunk;
  int nv = p.rows <= 304 ? 1 : 4;
  while (nv > 1 && chunks <= 32 * (nv / 2)) nv >>= 1;
  while (chunks > (nv >= 4 ? 512 : 1024) * nv) nv <<= 1;  // Q8_MAX_COLS is 8 chunks of 512 threads
  p.row_threads = ((chunks + nv - 1) / nv + 31) / 32 * 32;
  if (value_type == Q8_F32)
    return aligned ? launch_typed<float, true>(p, norm, nv, stream)
                   : launch_typed<float, false>(p, norm, nv, stream);
  if (value_type == Q8_BF16)
    return aligned ? launch_typed<__nv_bfloat16, true>(p, norm, nv, stream)
                   : launch_typed<__nv_bfloat16, false>(p, norm, nv, stream);
  return aligned ? launch_typed<__half, true>(p, norm, nv, stream)
                 : launch_typed<__half, false>(p, norm, nv, stream);
}

}  // namespace c3d
