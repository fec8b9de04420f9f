// q8_rows.cu -- the two operators that turn rows of values into 8-bit codes with a scale each: the
// root-mean-square norm with the residual's addition, and the gated activation.
//
// One reduction serves the norm. With v = h * weight and r = 1 / sqrt(sum(h^2)/cols + eps), the
// normed value is y = v * r, so amax(y) = r * amax(v) and the code y / (amax(y) / T) = v * T /
// amax(v): r cancels out of the codes and enters only the scale. The sum of squares and amax(v) are
// therefore taken in the same pass, reduced together, and the row's values stay in registers: every
// input is read once, every output written once, which is the operator's floor (both are bound by
// the memory's bandwidth, and by one row's latency when there are few rows).
#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "q8_common.cuh"

namespace c3d {

constexpr int kChunk = 8;  // values a thread takes at a time: 16 bytes of a 16-bit type

// Squares of values below about 2^-50 lose bits in fp32, or all of them. Beside an eps of kSmallEps or more
// that changes nothing. With a smaller one (0, mostly) small_rows_kernel first takes the sum of values
// lifted by kRowLift, and it counts (kSmall) for rows whose plain sum is below kLiftBelow, where no lifted
// square overflows. It is a launch of its own (1 x 4096 bf16 2.1 -> 3.1 us, 8192 x 4096 37.4 -> 39.4, 40000 x
// 256 13.6 -> 18.9): taken in the norm's kernels, under a condition that other calls do not meet, it
// cost those their registers (8192 x 4098 bf16 42 -> 57 us).
constexpr float kSmallEps = 0x1p-120f, kRowLift = 0x1p100f, kLiftBelow = 0x1p-100f;

// amax(|v|) as bits: unsigned order is the order of the magnitudes, and a NaN is above them all, so
// that one NaN or infinity marks the row.
struct RowStat {
  float sum;
  unsigned amax;
};

// amax with |a| and |b| taken in, a NaN kept (max.NaN gives the positive one).
__device__ __forceinline__ unsigned amax_with(unsigned amax, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;"
      : "=f"(r)
      : "f"(a), "f"(b), "f"(__uint_as_float(amax)));
  return __float_as_uint(r);
}

__device__ __forceinline__ RowStat warp_reduce(RowStat s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s.sum += __shfl_xor_sync(0xFFFFFFFFu, s.sum, o);
  s.amax = __reduce_max_sync(0xFFFFFFFFu, s.amax);
  return s;
}

// Over the threads of one row: a warp, or the whole block. Consecutive rows of a block alternate
// between two buffers, so that one barrier a row is enough.
__device__ __forceinline__ RowStat row_reduce(RowStat s, int threads, int buffer) {
  s = warp_reduce(s);
  if (threads == 32) return s;
  __shared__ RowStat warp_stat[2][32];
  const int lane = threadIdx.x & 31;
  if (lane == 0) warp_stat[buffer][threadIdx.x >> 5] = s;
  __syncthreads();
  s = lane < threads / 32 ? warp_stat[buffer][lane] : RowStat{0.0f, 0u};
  return warp_reduce(s);
}

// Eight values of a row on their way to registers, as they lie in memory: the loads of the next row
// are in flight while this one is worked on, so they are held unconverted.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float v[kChunk];
  __device__ __forceinline__ void load8(const float* p) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void load1(int e, const float* p) { v[e] = *p; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) v[e] = 0.0f;
  }
  __device__ __forceinline__ void values(float (&f)[kChunk]) const {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) f[e] = v[e];
  }
};
template <typename T>
struct Raw16 {
  uint32_t w[4];  // two values each, the first in the low half
  __device__ __forceinline__ void load8(const T* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ __forceinline__ void load1(int e, const T* p) {
    const uint32_t h = *reinterpret_cast<const uint16_t*>(p);
    w[e / 2] = e % 2 ? (w[e / 2] & 0xFFFFu) | (h << 16) : h;
  }
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
};
template <>
struct Raw<__nv_bfloat16> : Raw16<__nv_bfloat16> {
  __device__ __forceinline__ void values(float (&f)[kChunk]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw<__half> : Raw16<__half> {
  __device__ __forceinline__ void values(float (&f)[kChunk]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
};

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

// Where a thread's kChunk values of step i lie in rows on the 16-byte grid: consecutive columns,
// moved by 16-byte accesses. Only a warp that holds a row's last, incomplete chunk (kTail) has code
// for single elements; in the others a chunk is in the row or not.
struct Place {
  int tid, threads, cols;
  __device__ __forceinline__ int col(int i) const { return (i * threads + tid) * kChunk; }
  __device__ __forceinline__ bool whole(int i) const { return col(i) + kChunk <= cols; }
  __device__ __forceinline__ bool partial(int i) const { return !whole(i) && col(i) < cols; }
  // Columns past the row's end read 0, which changes neither a sum of squares nor an amax.
  template <bool kTail, typename T>
  __device__ __forceinline__ void load(const T* row, int i, Raw<T>& r) const {
    r.clear();
    if (whole(i)) r.load8(row + col(i));
    if (kTail && partial(i)) {
#pragma unroll
      for (int e = 0; e < kChunk - 1; ++e)
        if (col(i) + e < cols) r.load1(e, row + col(i) + e);
    }
  }
  template <typename T, bool kTail>
  __device__ __forceinline__ void values(const void* row, int i, float (&v)[kChunk]) const {
    Raw<T> r;
    load<kTail>(static_cast<const T*>(row), i, r);
    r.values(v);
  }
  template <bool kTail, typename T>
  __device__ __forceinline__ void store(T* row, int i, const float (&v)[kChunk]) const {
    if (whole(i)) store8(row + col(i), v);
    if (kTail && partial(i)) {
#pragma unroll
      for (int e = 0; e < kChunk - 1; ++e)
        if (col(i) + e < cols) row[col(i) + e] = q8_from_float<T>(v[e]);
    }
  }
  template <bool kTail>
  __device__ __forceinline__ void store_codes(uint8_t* row, int i, uint2 c) const {
    if (whole(i)) *reinterpret_cast<uint2*>(row + col(i)) = c;
    if (kTail && partial(i)) {
#pragma unroll
      for (int e = 0; e < kChunk - 1; ++e)
        if (col(i) + e < cols)
          row[col(i) + e] = (uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
    }
  }
};

// f with std::true_type or std::false_type.
template <typename F>
__device__ __forceinline__ void with_flag(bool flag, F f) {
  if (flag)
    f(std::true_type{});
  else
    f(std::false_type{});
}

// Four int8 codes of values |v * inv| <= 127 (and a rounding error): adding 1.5 * 2^23 rounds the
// fused product to an integer, ties to even, whose low byte is the code.
__device__ __forceinline__ uint32_t int8_codes(const float* v, float inv) {
  uint32_t n[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float2 r = q8_fma2(make_float2(v[i], v[i + 1]), make_float2(inv, inv),
                          make_float2(12582912.0f, 12582912.0f));
    n[i] = __float_as_uint(r.x);
    n[i + 1] = __float_as_uint(r.y);
  }
  return __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t e4m3_codes(const float* v, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(q8_mul2(make_float2(v[0], v[1]), make_float2(inv, inv)),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(q8_mul2(make_float2(v[2], v[3]), make_float2(inv, inv)),
                                               __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xFFFFu) | (hi << 16);
}

// How a row's values turn into its codes: code = round(v * lift * inv).
struct RowCode {
  float lift, inv;
};

// The row's scale, written by one thread, and its codes' factors. The norm's r goes into the scale
// alone, so only that thread works it out. A row that is not finite gets the scale NaN and codes 0
// (its values must be replaced by 0 before they are multiplied). A row so small that top / amax would
// overflow is lifted first. A code is the rounding of v * (top / amax), two fp32 operations as a quotient
// by the scale is. Next to a tie fp32 decides between two neighbours, in about one code of a million:
// against 64 bits 901 codes of 12 activations of 4096 x 16384 differ, 2458 of 12 norms of 8192 x 4096 and 54
// of 12 of 1501 x 5001 fp32; by elementary fp32 operations and quotients 991, 3395 and 92.
template <bool kNorm, bool kSmall>
__device__ __forceinline__ RowCode row_scale(const RowStat& st, const RowsParams& p, long long row,
                                             bool writer, bool& bad) {
  const float top = p.code_type == Q8_E4M3 ? 448.0f : 127.0f;
  bad = st.amax >= 0x7F800000u || !(st.sum < INFINITY);
  const float amax = __uint_as_float(st.amax);
  if (writer) {
    float root = kNorm ? amax * rsqrtf(st.sum / (float)p.cols + p.eps) : amax;
    if (kSmall && st.sum < kLiftBelow) {
      const float gain = rsqrtf(p.scale[row] / (float)p.cols + p.eps * kRowLift * kRowLift);
      root = amax < 1.0f ? amax * kRowLift * gain : amax * gain * kRowLift;
    }
    p.scale[row] = bad ? __int_as_float(0x7FC00000) : (amax > 0.0f ? root / top : 1.0f);
  }
  RowCode c;
  c.lift = amax < 0x1p-100f ? kRowLift : 1.0f;
  c.inv = bad || amax == 0.0f ? 0.0f : top / (amax * c.lift);
  return c;
}

// Codes and scale of one row whose values the threads hold.
template <int NV, bool kNorm, bool kSmall>
__device__ __forceinline__ void row_write(float (&v)[NV][kChunk], const RowStat& st,
                                          const RowsParams& p, long long row, const Place& at,
                                          bool tail) {
  bool bad;
  const RowCode rc = row_scale<kNorm, kSmall>(st, p, row, at.tid == 0, bad);
  if (bad || rc.lift != 1.0f) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[i][e] = bad ? 0.0f : v[i][e] * rc.lift;
  }
  uint8_t* q = p.q + row * p.q_pitch;
  uint2 c[NV];
  if (p.code_type == Q8_E4M3) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      c[i] = make_uint2(e4m3_codes(v[i], rc.inv), e4m3_codes(v[i] + 4, rc.inv));
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      c[i] = make_uint2(int8_codes(v[i], rc.inv), int8_codes(v[i] + 4, rc.inv));
  }
  with_flag(tail, [&](auto t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) at.template store_codes<decltype(t)::value>(q, i, c[i]);
  });
}

// silu(g) * u with silu(g) = g / (1 + exp(-g)), of two values with |g| <= kSiluNear: nothing over- or
// underflows there, which the approximations need. The reciprocal of a divisor past 2^126 (gates below
// -87.34) would be flushed to 0, where silu, some -1e-36, is an ordinary number.
constexpr float kSiluNear = 80.0f;
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float2 silu_mul_near(float2 g, float2 u) {
  const float2 t = q8_mul2(g, make_float2(-kLog2e, -kLog2e));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const float2 d = q8_add2(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return q8_mul2(q8_mul2(g, r), u);
}
// Any gate: of a negative one, g exp(g) / (1 + exp(g)), whose exponential loses bits below -87 and is 0
// below -104, but whose divisor lies in [1, 2].
__device__ __forceinline__ float silu_mul_far(float g, float u) {
  const float e = __expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * u;
}
// v = silu(v) * u for kChunk values; a NaN takes the second way.
__device__ __forceinline__ void silu_mul(float (&v)[kChunk], const float (&u)[kChunk]) {
  unsigned far = 0;
#pragma unroll
  for (int e = 0; e < kChunk; e += 2) far = amax_with(far, v[e], v[e + 1]);
  if (__uint_as_float(far) <= kSiluNear) {
#pragma unroll
    for (int e = 0; e < kChunk; e += 2) {
      const float2 y = silu_mul_near(make_float2(v[e], v[e + 1]), make_float2(u[e], u[e + 1]));
      v[e] = y.x;
      v[e + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < kChunk; ++e) v[e] = silu_mul_far(v[e], u[e]);
  }
}

// One block (of 32 to 1024 threads) or, for short rows, one warp holds a row, NV chunks a thread, and
// takes every stride-th row. Up to two chunks a thread the next row's loads are issued before this
// row is worked on: without that the memory waits for each block's reduction and stores (norm of
// 8192 x 4096 bf16: 67.5 us with a block a row, 37.3 so). 16-bit rows past 16384 columns take eight
// chunks a thread and no look-ahead, which their registers have no room for (1000 x 32768 32.7 us, 50.4
// by the wide kernel below). fp32 rows past 8192 columns go there: 2368 x 13256 with a residual 66 us, 95
// so, 1000 x 24576 54.5 and 79.7; without a residual 1000 x 32768 loses, 52.9 and 45.5, which one rule for
// both takes. With two chunks a thread a 16-bit norm's 64 registers spill 24 bytes.
template <typename T>
constexpr int rows_max_threads(int nv) {  // 64 registers a thread, or 128
  return nv == 1 || (nv == 2 && sizeof(T) == 2) ? 1024 : 512;
}

template <typename T, int NV, bool kNorm, bool kSmall>
__global__ void __launch_bounds__(rows_max_threads<T>(NV)) rows_q8_kernel(const RowsParams p) {
  constexpr bool kAhead = NV <= 2;
  pdl_wait_primary();
  pdl_launch_dependents();
  const bool warp_rows = p.row_threads == 32;
  const Place at{warp_rows ? (int)(threadIdx.x & 31) : (int)threadIdx.x, p.row_threads,
                           p.cols};
  const long long stride = warp_rows ? (long long)gridDim.x * (blockDim.x >> 5) : gridDim.x;
  long long row = warp_rows ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                            : (long long)blockIdx.x;
  const bool two = !kNorm || p.b;  // a second input: the residual, or up
  bool partial = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) partial |= at.partial(i);
  const bool tail = __any_sync(0xFFFFFFFFu, partial);
  Raw<T> ra[NV], rb[NV];
  auto load_row = [&](long long r) {
    const T* a = static_cast<const T*>(p.a) + r * p.a_pitch;
    const T* b = static_cast<const T*>(p.b) + r * p.b_pitch;
    with_flag(tail, [&](auto t) {
#pragma unroll
      for (int i = 0; i < NV; ++i) at.template load<decltype(t)::value>(a, i, ra[i]);
      if (two) {
#pragma unroll
        for (int i = 0; i < NV; ++i) at.template load<decltype(t)::value>(b, i, rb[i]);
      }
    });
  };
  if (kAhead && row < p.rows) load_row(row);
  for (int buffer = 0; row < p.rows; row += stride, buffer ^= 1) {
    if (!kAhead) load_row(row);
    float v[NV][kChunk];
    RowStat st{0.0f, 0u};
    float2 sum = make_float2(0.0f, 0.0f);
    with_flag(tail, [&](auto t) {
      constexpr bool kTail = decltype(t)::value;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float b[kChunk];
        ra[i].values(v[i]);
        if (two) rb[i].values(b);
        if (kNorm) {
          if (two) {
#pragma unroll
            for (int e = 0; e < kChunk; e += 2) {
              const float2 h = q8_add2(make_float2(v[i][e], v[i][e + 1]), make_float2(b[e], b[e + 1]));
              v[i][e] = h.x;
              v[i][e + 1] = h.y;
            }
            // these columns have been read by this thread, if sum_out is x or the residual
            at.template store<kTail>(static_cast<T*>(p.sum_out) + row * p.sum_pitch, i, v[i]);
          }
          float w[kChunk];
          if (p.weight_type == Q8_F32)
            at.template values<float, kTail>(p.weight, i, w);
          else if (p.weight_type == Q8_BF16)
            at.template values<__nv_bfloat16, kTail>(p.weight, i, w);
          else
            at.template values<__half, kTail>(p.weight, i, w);
#pragma unroll
          for (int e = 0; e < kChunk; e += 2) {
            const float2 h = make_float2(v[i][e], v[i][e + 1]);
            sum = q8_fma2(h, h, sum);
            const float2 y = q8_mul2(h, make_float2(w[e], w[e + 1]));
            v[i][e] = y.x;
            v[i][e + 1] = y.y;
          }
        } else {
          silu_mul(v[i], b);
        }
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) st.amax = amax_with(st.amax, v[i][e], v[i][e + 1]);
      }
    });
    if (kAhead && row + stride < p.rows) load_row(row + stride);
    st.sum = sum.x + sum.y;
    st = row_reduce(st, p.row_threads, buffer);
    row_write<NV, kNorm, kSmall>(v, st, p, row, at, tail);
  }
}

// Rows off the 16-byte grid (a base, a pitch or a weight): elements one by one, or by pairs where every
// row starts on a pair (kPair), consecutive ones by a warp's lanes, kLoose a thread, held in registers
// and loaded one row ahead as above. A warp's columns are a run of 32 * kLoose, the same in every row:
// its accesses are one address and constant offsets, without a mask in all warps but the row's last,
// and its weights are loaded once. Bound by the issue of instructions (1501 x 5001 fp32: 27 us by
// asynchronous copies to shared memory, 21 by 16-byte accesses shifted into place, 14.7 with a block's
// whole width between a thread's elements, each address and mask worked out, 10.6 so; 8192 x 4097 bf16
// with a residual 117 -> 61 us, 3.9 TB/s, and by pairs 8192 x 4098 42 us, 5.6 TB/s).
constexpr int kLoose = 8;
constexpr int kRun = 32 * kLoose;

// kPair (1, 2 or 4) consecutive elements as they lie in memory, in registers of their own.
template <typename T, int kPair>
struct LooseRaw {
  static constexpr int kBytes = kPair * (int)sizeof(T);
  uint32_t w[(kBytes + 3) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ float value(int j) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[j]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    } else {
      return __half2float(__ushort_as_half((unsigned short)(j % 2 ? w[j / 2] >> 16 : w[j / 2])));
    }
  }
};
template <int kPair, typename T>
__device__ __forceinline__ void loose_store(T* p, const float* v) {
  if constexpr (kPair == 1) {
    *p = q8_from_float<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    if constexpr (kPair == 2)
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    const uint32_t lo = q8_pack2<T>(make_float2(v[0], v[1]));
    if constexpr (kPair == 2)
      *reinterpret_cast<uint32_t*>(p) = lo;
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(lo, q8_pack2<T>(make_float2(v[2], v[3])));
  }
}
// The codes e .. e + kPair - 1 of kLoose.
template <int kPair>
__device__ __forceinline__ void loose_store_codes(uint8_t* p, const uint32_t* codes, int e) {
  const uint32_t c = codes[e / 4] >> (8 * (e & 3));
  if constexpr (kPair == 1)
    *p = (uint8_t)c;
  else if constexpr (kPair == 2)
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)c;
  else
    *reinterpret_cast<uint32_t*>(p) = c;
}

// f(e, offset) for the first of each kPair of a thread's kLoose elements, which lies `offset` columns
// behind the thread's first one, `left` columns before the row's end; the mask only where the run
// holds that end.
template <bool kWhole, int kPair, typename F>
__device__ __forceinline__ void for_run(int left, F f) {
#pragma unroll
  for (int e = 0; e < kLoose; e += kPair)
    if (kWhole || 32 * e < left) f(e, 32 * e);
}
template <int kPair, typename F>
__device__ __forceinline__ void for_run(bool whole, int left, F f) {
  if (whole)
    for_run<true, kPair>(left, f);
  else
    for_run<false, kPair>(left, f);
}

__device__ __forceinline__ void loose_codes(const float* f, int code_type, float inv,
                                            uint32_t* codes) {
  if (code_type == Q8_E4M3) {
#pragma unroll
    for (int e = 0; e < kLoose; e += 4) codes[e / 4] = e4m3_codes(f + e, inv);
  } else {
#pragma unroll
    for (int e = 0; e < kLoose; e += 4) codes[e / 4] = int8_codes(f + e, inv);
  }
}

template <typename T, bool kNorm, bool kSmall, int kPair>
__global__ void __launch_bounds__(1024) rows_q8_loose_kernel(const RowsParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int tid = threadIdx.x, threads = blockDim.x;
  const int col = (tid >> 5) * kRun + (tid & 31) * kPair;
  const int left = p.cols - col;
  const bool whole = ((tid >> 5) + 1) * kRun <= p.cols;  // the same for a warp
  const bool two = !kNorm || p.b;
  float w[kLoose] = {};
  if (kNorm)
    for_run<false, kPair>(left, [&](int e, int o) {
#pragma unroll
      for (int j = 0; j < kPair; ++j)
        w[e + j] = q8_load_value(p.weight, p.weight_type, col + o + j);
    });
  // 0 past the row's end, in every row
  LooseRaw<T, kPair> ra[kLoose / kPair] = {}, rb[kLoose / kPair] = {};
  auto load_row = [&](long long r) {
    const T* a = static_cast<const T*>(p.a) + r * p.a_pitch + col;
    const T* b = static_cast<const T*>(p.b) + r * p.b_pitch + col;
    for_run<kPair>(whole, left, [&](int e, int o) { ra[e / kPair].load(a + o); });
    if (two) for_run<kPair>(whole, left, [&](int e, int o) { rb[e / kPair].load(b + o); });
  };
  long long row = blockIdx.x;
  if (row < p.rows) load_row(row);
  for (int buffer = 0; row < p.rows; row += gridDim.x, buffer ^= 1) {
    float v[kLoose];
    RowStat st{0.0f, 0u};
#pragma unroll
    for (int e = 0; e < kLoose; ++e) v[e] = ra[e / kPair].value(e % kPair);
    if (kNorm) {
      if (two) {
        T* sum_out = static_cast<T*>(p.sum_out) + row * p.sum_pitch + col;
#pragma unroll
        for (int e = 0; e < kLoose; ++e) v[e] += rb[e / kPair].value(e % kPair);
        // this thread has read these columns, if sum_out is x or the residual
        for_run<kPair>(whole, left, [&](int e, int o) { loose_store<kPair>(sum_out + o, v + e); });
      }
#pragma unroll
      for (int e = 0; e < kLoose; ++e) {
        st.sum = fmaf(v[e], v[e], st.sum);
        v[e] *= w[e];
      }
    } else {
      float b[kLoose];
#pragma unroll
      for (int e = 0; e < kLoose; ++e) b[e] = rb[e / kPair].value(e % kPair);
      silu_mul(v, b);
    }
#pragma unroll
    for (int e = 0; e < kLoose; e += 2) st.amax = amax_with(st.amax, v[e], v[e + 1]);
    if (row + gridDim.x < p.rows) load_row(row + gridDim.x);
    st = row_reduce(st, threads, buffer);
    bool bad;
    const RowCode rc = row_scale<kNorm, kSmall>(st, p, row, tid == 0, bad);
    if (bad) {
#pragma unroll
      for (int e = 0; e < kLoose; ++e) v[e] = 0.0f;
    }
    if (rc.lift != 1.0f) {
#pragma unroll
      for (int e = 0; e < kLoose; ++e) v[e] *= rc.lift;
    }
    uint32_t codes[kLoose / 4];
    loose_codes(v, p.code_type, rc.inv, codes);
    uint8_t* q = p.q + row * p.q_pitch + col;
    for_run<kPair>(whole, left, [&](int e, int o) { loose_store_codes<kPair>(q + o, codes, e); });
  }
}

// Such rows of more than 8192 columns, and fp32 rows of more on the 16-byte grid (by fours): the row's
// values kept in shared memory between the two passes, a warp working on runs of kRun columns as
// above. 2000 x 12001 bf16 with a residual takes 143 us with single elements of a block's whole width,
// 46 so, 36 by pairs; 60 with 1024 threads, which leave one block an SM; with 256 threads wide rows leave
// too few warps (16383 fp32 columns 75 us against 56).
constexpr int kWideThreads = 512;

template <typename W, bool kWhole, int kPair>
__device__ __forceinline__ void wide_weights(const void* weight, int col, int left, float* w) {
  const W* g = static_cast<const W*>(weight) + col;
  for_run<kWhole, kPair>(left, [&](int e, int o) {
    LooseRaw<W, kPair> r;
    r.load(g + o);
#pragma unroll
    for (int j = 0; j < kPair; ++j) w[e + j] = r.value(j);
  });
}

template <typename T, bool kNorm, bool kWhole, int kPair>
__device__ __forceinline__ void wide_run(const T* a, const T* b, T* sum_out, const RowsParams& p,
                                         int col, float* v, RowStat& st) {
  const int left = p.cols - col;
  LooseRaw<T, kPair> ra[kLoose / kPair] = {}, rb[kLoose / kPair] = {};
  float w[kLoose];
  for_run<kWhole, kPair>(left, [&](int e, int o) { ra[e / kPair].load(a + col + o); });
  if (b) for_run<kWhole, kPair>(left, [&](int e, int o) { rb[e / kPair].load(b + col + o); });
  if (kNorm) {
    if (p.weight_type == Q8_F32)
      wide_weights<float, kWhole, kPair>(p.weight, col, left, w);
    else if (p.weight_type == Q8_BF16)
      wide_weights<__nv_bfloat16, kWhole, kPair>(p.weight, col, left, w);
    else
      wide_weights<__half, kWhole, kPair>(p.weight, col, left, w);
  }
  float f[kLoose];
#pragma unroll
  for (int e = 0; e < kLoose; ++e) f[e] = ra[e / kPair].value(e % kPair);
  if (!kNorm) {
    float u[kLoose];
#pragma unroll
    for (int e = 0; e < kLoose; ++e) u[e] = rb[e / kPair].value(e % kPair);
    silu_mul(f, u);
  }
  for_run<kWhole, kPair>(left, [&](int e, int o) {
    if (kNorm) {
      if (b) {
#pragma unroll
        for (int j = 0; j < kPair; ++j) f[e + j] += rb[e / kPair].value(j);
        loose_store<kPair>(sum_out + col + o, f + e);  // read by this thread, if x or the residual
      }
#pragma unroll
      for (int j = 0; j < kPair; ++j) {
        st.sum = fmaf(f[e + j], f[e + j], st.sum);
        f[e + j] *= w[e + j];
      }
    }
    st.amax = amax_with(st.amax, f[e], f[e + kPair - 1]);
    if constexpr (kPair == 4) st.amax = amax_with(st.amax, f[e + 1], f[e + 2]);
    loose_store<kPair>(v + col + o, f + e);  // read back by this thread alone
  });
}

template <bool kWhole, int kPair>
__device__ __forceinline__ void wide_codes(uint8_t* q, const RowsParams& p, int col, const float* v,
                                           bool bad, const RowCode& rc) {
  const int left = p.cols - col;
  float f[kLoose] = {};
  for_run<kWhole, kPair>(left, [&](int e, int o) {
    LooseRaw<float, kPair> r;
    r.load(v + col + o);
#pragma unroll
    for (int j = 0; j < kPair; ++j) f[e + j] = bad ? 0.0f : r.value(j) * rc.lift;
  });
  uint32_t codes[kLoose / 4];
  loose_codes(f, p.code_type, rc.inv, codes);
  for_run<kWhole, kPair>(left,
                         [&](int e, int o) { loose_store_codes<kPair>(q + col + o, codes, e); });
}

// (The activation is held to the 32 registers that let four blocks share an SM: 4096 x 12002 bf16 48 us,
// 51 with the 40 it takes otherwise.)
template <typename T, bool kNorm, bool kSmall, int kPair>
__global__ void __launch_bounds__(kWideThreads, kNorm ? 0 : 4) rows_q8_wide_kernel(const RowsParams p) {
  extern __shared__ __align__(16) float v[];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int first = (threadIdx.x >> 5) * kRun, lane = (threadIdx.x & 31) * kPair;
  int buffer = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, buffer ^= 1) {
    const T* a = static_cast<const T*>(p.a) + row * p.a_pitch;
    const T* b = p.b ? static_cast<const T*>(p.b) + row * p.b_pitch : nullptr;
    T* sum_out = static_cast<T*>(p.sum_out) + row * p.sum_pitch;
    RowStat st{0.0f, 0u};
    for (int c = first; c < p.cols; c += kWideThreads * kLoose) {
      if (c + kRun <= p.cols)
        wide_run<T, kNorm, true, kPair>(a, b, sum_out, p, c + lane, v, st);
      else
        wide_run<T, kNorm, false, kPair>(a, b, sum_out, p, c + lane, v, st);
    }
    st = row_reduce(st, kWideThreads, buffer);
    bool bad;
    const RowCode rc = row_scale<kNorm, kSmall>(st, p, row, threadIdx.x == 0, bad);
    uint8_t* q = p.q + row * p.q_pitch;
    for (int c = first; c < p.cols; c += kWideThreads * kLoose) {
      if (c + kRun <= p.cols)
        wide_codes<true, kPair>(q, p, c + lane, v, bad, rc);
      else
        wide_codes<false, kPair>(q, p, c + lane, v, bad, rc);
    }
  }
}

// For each row of small values, the sum of their lifted squares in place of its scale, where row_scale
// finds it. A warp takes a row and leaves it at the first value whose square alone makes the plain sum
// good: of ordinary rows no more than the first columns are read.
template <typename T>
__global__ void __launch_bounds__(128) small_rows_kernel(const RowsParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long stride = (long long)gridDim.x * 4;
  for (long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); row < p.rows; row += stride) {
    const T* a = static_cast<const T*>(p.a) + row * p.a_pitch;
    const T* b = p.b ? static_cast<const T*>(p.b) + row * p.b_pitch : nullptr;
    float sum = 0.0f;
    bool small = true;
    for (int c0 = 0, end = 32; small && c0 < p.cols; c0 = end, end += 1024) {
      bool mine = true;
#pragma unroll 8
      for (int c = c0 + lane; c < min(end, p.cols); c += 32) {
        const float h = q8_to_float(a[c]) + (b ? q8_to_float(b[c]) : 0.0f);
        mine = mine && fabsf(h) < 0x1p-49f;
        sum = fmaf(h * kRowLift, h * kRowLift, sum);
      }
      small = __all_sync(0xFFFFFFFFu, mine);
    }
    const RowStat st = warp_reduce(RowStat{sum, 0u});
    if (small && lane == 0) p.scale[row] = st.sum;
  }
}

// A persistent grid: as many blocks as the device holds at once, or as the rows need.
template <typename Kernel>
static cudaError_t launch_rows(Kernel kernel, const RowsParams& p, int threads, size_t smem,
                               cudaStream_t stream) {
  const long long blocks = p.row_threads == 32 ? (p.rows + 3) / 4 : p.rows;
  int dev = 0, sms = 0, held = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && blocks > sms)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&held, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<long long>(blocks, (long long)sms * std::max(1, held)));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The kernel's shared-memory limit is raised to what the widest row needs whatever this row does: the
// limit belongs to the kernel, so were it set to a call's own size, another host thread's call could
// lower it between that and the launch. (A row's values have row_reduce's 512 bytes beside them, and
// the limit that holds unless it is raised counts both.)
template <typename T, bool kNorm, bool kSmall, int kPair>
static cudaError_t launch_wide(RowsParams& p, cudaStream_t stream) {
  constexpr auto kernel = rows_q8_wide_kernel<T, kNorm, kSmall, kPair>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Q8_MAX_COLS * (int)sizeof(float));
  if (e != cudaSuccess) return e;
  p.row_threads = kWideThreads;
  return launch_rows(kernel, p, kWideThreads, p.cols * sizeof(float), stream);
}
template <typename T, bool kNorm, bool kSmall, int kPair>
static cudaError_t launch_loose(RowsParams& p, cudaStream_t stream) {
  if (p.cols > 1024 * kLoose) return launch_wide<T, kNorm, kSmall, kPair>(p, stream);
  p.row_threads = std::max(64, (p.cols + kRun - 1) / kRun * 32);  // one row a block
  return launch_rows(rows_q8_loose_kernel<T, kNorm, kSmall, kPair>, p, p.row_threads, 0, stream);
}

template <typename T, bool kNorm, bool kSmall>
static cudaError_t launch_typed(RowsParams& p, RowsGrid grid, cudaStream_t stream) {
  if (grid == RowsGrid::kElement) return launch_loose<T, kNorm, kSmall, 1>(p, stream);
  if (grid == RowsGrid::kPair) return launch_loose<T, kNorm, kSmall, 2>(p, stream);
  const int chunks = (p.cols + kChunk - 1) / kChunk;
  const bool wide = chunks > 2 * rows_max_threads<T>(2);
  if constexpr (sizeof(T) == 4)
    if (wide)
      return p.cols % 4 == 0   ? launch_wide<T, kNorm, kSmall, 4>(p, stream)
             : p.cols % 2 == 0 ? launch_wide<T, kNorm, kSmall, 2>(p, stream)
                               : launch_wide<T, kNorm, kSmall, 1>(p, stream);
  // One chunk a thread where there are few rows, whose time is one row's latency; otherwise two.
  const int nv = wide ? 8 : chunks > rows_max_threads<T>(1) || (p.rows > 304 && chunks > 32) ? 2 : 1;
  p.row_threads = ((chunks + nv - 1) / nv + 31) / 32 * 32;
  const int threads = p.row_threads == 32 ? 128 : p.row_threads;
  if (nv == 1) return launch_rows(rows_q8_kernel<T, 1, kNorm, kSmall>, p, threads, 0, stream);
  if constexpr (sizeof(T) == 2)
    if (wide) return launch_rows(rows_q8_kernel<T, 8, kNorm, kSmall>, p, threads, 0, stream);
  return launch_rows(rows_q8_kernel<T, 2, kNorm, kSmall>, p, threads, 0, stream);
}

template <typename T>
static cudaError_t launch_type(RowsParams& p, bool norm, RowsGrid grid, cudaStream_t stream) {
  if (!norm) return launch_typed<T, false, false>(p, grid, stream);
  if (p.eps >= kSmallEps) return launch_typed<T, true, false>(p, grid, stream);
  p.row_threads = 32;
  const cudaError_t e = launch_rows(small_rows_kernel<T>, p, 128, 0, stream);
  return e != cudaSuccess ? e : launch_typed<T, true, true>(p, grid, stream);
}

cudaError_t launch_rows_q8(RowsParams p, int value_type, bool norm, RowsGrid grid,
                           cudaStream_t stream) {
  if (value_type == Q8_F32) return launch_type<float>(p, norm, grid, stream);
  if (value_type == Q8_BF16) return launch_type<__nv_bfloat16>(p, norm, grid, stream);
  return launch_type<__half>(p, norm, grid, stream);
}

}  // namespace c3d
