// q8_heads.cuh -- rows of heads on their way into attention: the norm and the rotation of queries and
// keys, their codes in a paged cache (and the cache's rows as values: q8_heads.cu). A value type's kernels take a compiler
// most of a minute, so each has a file of its own (the build takes 60 s instead of 123 on 8 cores).
//
// A row is one token's head. L = 8, 16 or 32 lanes hold it, eight elements each, so that its sums, its
// partners in the rotation and its scale are shuffles, and every element is read once and written once:
// the memory's bandwidth is the bound. A warp takes a token's heads; the sines of its angles are taken once (16384 tokens of
// 16 queries and 16 keys of 128 with three axes: 109 us with a row at a time, 55.4 now, 4.9 TB/s, beside 65% of the issue slots;
// 65536 x 8 rows of 4-bit codes read back: 70.6 us, 4.9 TB/s, 81% of them).
//
// Angles. In turns an angle is frequency / 2 pi * position, and only its fraction matters. With the
// frequency as an integer f of 2^-64 turns the fraction of f * position is the 64-bit product, whose
// overflow drops whole turns: positions of any size cost two integer products and lose nothing, where an
// fp32 product at position 10^5 is off by 4e-3 of a radian. sincospi takes it from there.
//
// Codes. The code of v is T * v / amax, to the nearest, ties to even (for 4 bits 15 * (v - lowest) / (highest -
// lowest)). With 16-bit inputs such quotients lie on ties often, so the quotient has to be right to the
// last bit: q0 = a * r with r = 1 / w rounded, then q0 + r * (a - q0 * w) with both steps fused, which
// is the correctly rounded a / w (Markstein, 1990). (Division by the rounded scale, in fp32 with torch, sends so many 4-bit
// codes of 8192 x 8 x 128 bf16 keys the other way that their values differ by 1.3%.)
#pragma once
#include <algorithm>
#include <type_traits>

#include "q8_attn_internal.h"
#include "q8_common.cuh"

namespace c3d {

constexpr int kHeadsThreads = 256;
constexpr int kLane = 8;             // elements of a row that a lane holds
constexpr int kMostPairs = Q8_MAX_HEAD_DIM / 2;
constexpr int kNoCodes = 0;
constexpr int kBlocksPerSm = 3;      // the kernel's and the grid's: each warp takes the same number of tokens, but for one

// ------------------------------------------------------------------ eight values of a row
__device__ __forceinline__ void store8(float* p, const float (&f)[kLane]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[kLane]) {
  uint4 a;
  a.x = q8_pack2<T>(make_float2(f[0], f[1]));
  a.y = q8_pack2<T>(make_float2(f[2], f[3]));
  a.z = q8_pack2<T>(make_float2(f[4], f[5]));
  a.w = q8_pack2<T>(make_float2(f[6], f[7]));
  *reinterpret_cast<uint4*>(p) = a;
}

// ------------------------------------------------------------------ sums over the lanes of a row
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// Extremes that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int L>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
// The largest magnitude, NaN if there is one.
template <int L>
__device__ __forceinline__ float row_amax(const float (&f)[kLane]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < kLane; e += 2)
    asm("max.NaN.abs.f32 %0, %1, %2, %0;" : "+f"(m) : "f"(f[e]), "f"(f[e + 1]));
  return row_max<L>(m);
}

constexpr float kLargest = 3.4028234e38f;
constexpr float kInteger = 12582912.0f;  // 1.5 * 2^23: added to a small number it leaves its nearest integer in the low bits

// a / w rounded once, for two, given r = 1 / w rounded.
__device__ __forceinline__ float2 quotients(float2 a, float w, float r) {
  const float2 r2 = make_float2(r, r), q = q8_mul2(a, r2);
  return q8_fma2(q8_fma2(make_float2(-q.x, -q.y), make_float2(w, w), a), r2, q);
}

// A power of two that takes w (not 0) to where neither its reciprocal nor 448 times it leaves fp32's normal range.
__device__ __forceinline__ float lift_of(float w) {
  return w < 0x1p-100f ? 0x1p100f : w > 0x1p100f ? 0x1p-100f : 1.0f;
}

// ------------------------------------------------------------------ codes
// One row's codes into the cache at row `row` of its codes; f is 0 in lanes behind the row's end, which
// there are none of with a cache (head_dim is L * 8).
template <int CODE, int L>
__device__ __forceinline__ void write_codes(uint8_t* codes, float* scales, long long row, int chunk,
                                            const float (&f)[kLane], bool store) {
  const float nan = __int_as_float(0x7FFFFFFF);
  if constexpr (CODE == Q8_INT4) {
    float lo = f[0], hi = f[0];
#pragma unroll
    for (int e = 1; e < kLane; ++e) {
      lo = min_nan(lo, f[e]);
      hi = max_nan(hi, f[e]);
    }
    hi = row_max<L>(hi);
    lo = -row_max<L>(-lo);
    const float width = hi - lo;
    const bool bad = !(width <= kLargest), flat = bad || width == 0.0f;
    const float lift = lift_of(width);
    const float w = width * lift, r = __frcp_rn(w);
    const float2 times = make_float2(15.0f * lift, 15.0f * lift), least = make_float2(-lo, -lo);
    unsigned bytes[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = q8_mul2(q8_add2(make_float2(f[2 * e], f[2 * e + 1]), least), times);
      const float2 t = q8_add2(quotients(a, w, r), make_float2(kInteger, kInteger));
      bytes[e] = __float_as_uint(fmaf(16.0f, t.y - kInteger, t.x));  // in the low byte: both codes
    }
    const unsigned word = __byte_perm(__byte_perm(bytes[0], bytes[1], 0x0040), __byte_perm(bytes[2], bytes[3], 0x0040), 0x5410);
    if (!store) return;
    *reinterpret_cast<unsigned*>(codes + (row * L + chunk) * (kLane / 2)) = flat ? 0u : word;
    if (chunk == 0)
      *reinterpret_cast<float2*>(scales + 2 * row) =
          make_float2(bad ? nan : flat ? 1.0f : __fdiv_rn(width, 15.0f), bad ? 0.0f : lo);
  } else {
    constexpr float kTop = CODE == Q8_INT8 ? 127.0f : 448.0f;
    const float amax = row_amax<L>(f);
    const bool bad = !(amax <= kLargest), flat = bad || amax == 0.0f;
    const float lift = lift_of(amax);
    const float w = amax * lift, r = __frcp_rn(w);
    const float2 times = make_float2(kTop * lift, kTop * lift);
    float2 q[kLane / 2];
#pragma unroll
    for (int e = 0; e < kLane / 2; ++e) q[e] = quotients(q8_mul2(make_float2(f[2 * e], f[2 * e + 1]), times), w, r);
    uint2 word;
    if constexpr (CODE == Q8_INT8) {
      unsigned half[4];  // two codes in the low bytes
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = q8_add2(q[e], make_float2(kInteger, kInteger));
        half[e] = __byte_perm(__float_as_uint(t.x), __float_as_uint(t.y), 0x0040);
      }
      word = make_uint2(__byte_perm(half[0], half[1], 0x5410), __byte_perm(half[2], half[3], 0x5410));
    } else {
      unsigned half[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) half[e] = __nv_cvt_float2_to_fp8x2(q[e], __NV_SATFINITE, __NV_E4M3);
      word = make_uint2(half[0] | half[1] << 16, half[2] | half[3] << 16);
    }
    if (!store) return;
    *reinterpret_cast<uint2*>(codes + (row * L + chunk) * kLane) = flat ? make_uint2(0, 0) : word;
    if (chunk == 0) scales[row] = bad ? nan : flat ? 1.0f : __fdiv_rn(amax, kTop);
  }
}

// ------------------------------------------------------------------ the rows of heads
// How pairs lie: next to each other, in whole lanes; the same, where the last rotated lane has elements behind them, which stay
// whatever lies beside them (with that test in every form: 56.6 instead of 55.4 us for 16384 x 32 x 128 with three axes); half of the
// rotated part apart, in whole lanes; the same, not in whole lanes (the partner is then read a second time).
enum { kAdjacent, kLooseAdjacent, kHalves, kLooseHalves };

// What a lane holds of a row as it lies in memory: a row ahead is under way while one is worked on.
template <typename T>
struct RawLane {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float (&f)[kLane]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < kLane; ++e) f[e] = reinterpret_cast<const float*>(w)[e];
    } else if constexpr (std::is_same_v<T, __half>) {
#pragma unroll
      for (int e = 0; e < kLane; e += 2) {
        const float2 v = __half22float2(reinterpret_cast<const __half2*>(w)[e / 2]);
        f[e] = v.x, f[e + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kLane; e += 2) {
        const uint32_t v = reinterpret_cast<const uint32_t*>(w)[e / 2];
        f[e] = __uint_as_float(v << 16), f[e + 1] = __uint_as_float(v & 0xFFFF0000u);
      }
    }
  }
};

// A warp takes a token, or a share of its heads where there are few tokens: 32 / L rows of one kind (queries, keys, values) at a
// time, all of the kind's, with the angles' sines and cosines in its lanes' registers.
template <typename T, int CODE, int L, int PAIRS>
__global__ void __launch_bounds__(kHeadsThreads, kBlocksPerSm) heads_kernel(const HeadsParams p, int shares) {
  constexpr bool kNextTo = PAIRS == kAdjacent || PAIRS == kLooseAdjacent;
  constexpr int kRows = 32 / L;  // of a warp at a time
  constexpr int kAhead = sizeof(T) == 4 ? 1 : 2;  // times that, on their way beside as many that are worked on
  __shared__ float2 turned[kHeadsThreads / 32][kMostPairs];  // cosine and sine
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, chunk = lane % L, e0 = chunk * kLane;
  const bool mine = e0 < p.head_dim;
  const bool rotated = p.turns && e0 < p.rot_dim;
  const int half = p.rot_dim / 2;
  const float one_over_dim = 1.0f / p.head_dim;
  // Rows of each kind, in units of what a warp takes at a time.
  const int q_units = (p.q_heads + kRows - 1) / kRows;
  const int k_units = p.k.p ? (p.kv_heads + kRows - 1) / kRows : 0;
  const int units = q_units + k_units + (CODE != kNoCodes ? (p.kv_heads + kRows - 1) / kRows : 0);
  const int per_share = (units + shares - 1) / shares;
  __shared__ __align__(16) float weights[2][Q8_MAX_HEAD_DIM];  // of queries and of keys
  if (p.q_weight || p.k_weight) {
    for (int i = threadIdx.x; i < p.head_dim; i += kHeadsThreads) {
      if (p.q_weight) weights[0][i] = q8_load_value(p.q_weight, p.weight_type, i);
      if (p.k_weight) weights[1][i] = q8_load_value(p.k_weight, p.weight_type, i);
    }
    __syncthreads();
  }
  const long long items = (long long)p.tokens * shares, step = (long long)gridDim.x * (kHeadsThreads / 32);
  for (long long item = (long long)blockIdx.x * (kHeadsThreads / 32) + warp; item < items; item += step) {
    const int t = shares == 1 ? (int)item : (int)(item / shares);
    const int first = shares == 1 ? 0 : (int)(item - (long long)t * shares) * per_share;
    const int end = min(units, first + per_share);
    // The first queries are on their way while the angles are taken.
    RawLane<T> ahead[kAhead] = {};
    if (first < min(end, q_units)) {
      const T* src = static_cast<const T*>(p.q.p) + t * p.q.pitch + (long long)(first * kRows + lane / L) * p.q.head_pitch + e0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (first + i < end && (first + i) * kRows + lane / L < p.q_heads && mine)
          ahead[i].load(src + i * kRows * p.q.head_pitch);
    }
    long long slot = -1;
    if constexpr (CODE != kNoCodes) slot = p.slots[t];
    float2 turn[kLane];  // of this lane's elements (kNextTo: pairs, of which there are half as many)
    if (p.turns && (first < q_units + k_units)) {
      __syncwarp();
      for (int j = lane; j < half; j += 32) {
        int axis = p.axis ? p.axis[j] : 0;
        if (axis >= p.axes) axis = 0;
        const long long pos = p.positions[axis * p.positions_pitch + t];
        const long long angle = (long long)(p.turns[j] * (unsigned long long)pos);
        float s, c;
        sincospif((float)angle * 0x1p-63f, &s, &c);
        turned[warp][j] = make_float2(c, s);
      }
      __syncwarp();
      if (rotated) {
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
          if (kNextTo && e >= kLane / 2) break;
          const int i = kNextTo ? e0 / 2 + e : e0 + e >= half ? e0 + e - half : e0 + e;
          turn[e] = i < half ? turned[warp][i] : make_float2(1.0f, 0.0f);
        }
      }
    }
    long long at = 0;  // the slot's row of its page's first head
    bool store = false;
    if constexpr (CODE != kNoCodes) {
      store = slot >= 0 && slot < (long long)p.cache.slots;
      const unsigned page = (unsigned)slot / (unsigned)p.cache.page_size;
      at = (long long)page * p.kv_heads * p.cache.page_size + ((unsigned)slot - page * p.cache.page_size);
    }
    // The rows of one kind, of which this share has the units [from, to).
    auto rows = [&](auto kind_of, int from, int to, const Heads& in, const Heads& out, const void* w, int heads) {
      constexpr int kind = decltype(kind_of)::value;
      if (from >= to) return;
      const int head0 = from * kRows + lane / L;
      const T* src = static_cast<const T*>(in.p) + t * in.pitch + head0 * in.head_pitch + e0;
      T* dst = static_cast<T*>(out.p) + t * out.pitch + head0 * out.head_pitch + e0;
      auto load = [&](int u) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (u + i < to && (u + i) * kRows + lane / L < heads && mine) ahead[i].load(src + i * kRows * in.head_pitch);
        src += kAhead * kRows * in.head_pitch;
      };
      if (kind == 0)
        src += kAhead * kRows * in.head_pitch;  // loaded before
      else
        load(from);
      for (int u0 = from; u0 < to; u0 += kAhead) {
        RawLane<T> raws[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) raws[i] = ahead[i];
        [[maybe_unused]] const T* here0 = src - kAhead * kRows * in.head_pitch;
        load(u0 + kAhead);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int u = u0 + i, head = u * kRows + lane / L;
          if (u >= to) break;
          const bool live = head < heads && mine;
          const RawLane<T>& raw = raws[i];
          [[maybe_unused]] const T* here = here0 + i * kRows * in.head_pitch;
          float f[kLane];
          raw.values(f);
          float rms = 1.0f, lift = 1.0f;
          if (kind < 2 && w) {
            float2 two = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < kLane; e += 2) {
              const float2 v = make_float2(f[e], f[e + 1]);
              two = q8_fma2(v, v, two);
            }
            float sum = row_sum<L>(two.x + two.y);
            const bool lifted = !(sum <= 0x1p100f) || (sum < 0x1p-80f && p.eps < 0x1p-100f);
            if (__any_sync(0xFFFFFFFFu, lifted)) {
              if (lifted) lift = sum < 1.0f ? 0x1p100f : 0x1p-100f;
              float again = 0.0f;
#pragma unroll
              for (int e = 0; e < kLane; ++e) {
                if (lifted) f[e] *= lift;
                again = fmaf(f[e], f[e], again);
              }
              again = row_sum<L>(again);
              if (lifted) sum = again;
            }
            const float mean = fmaf(sum, one_over_dim, p.eps * lift * lift);
            rms = mean == 0.0f ? 0.0f : rsqrtf(mean);
            if (mine) {
              const float2 rms2 = make_float2(rms, rms);
#pragma unroll
              for (int e = 0; e < kLane; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(&weights[kind][e0 + e]);
                const float2 a = q8_mul2(make_float2(f[e], f[e + 1]), q8_mul2(rms2, make_float2(v.x, v.y)));
                const float2 b = q8_mul2(make_float2(f[e + 2], f[e + 3]), q8_mul2(rms2, make_float2(v.z, v.w)));
                f[e] = a.x, f[e + 1] = a.y, f[e + 2] = b.x, f[e + 3] = b.y;
              }
            }
          }
          if (kind < 2 && p.turns) {
            if constexpr (kNextTo) {
              if (rotated) {
#pragma unroll
                for (int e = 0; e < kLane; e += 2) {
                  if (PAIRS == kLooseAdjacent && e0 + e >= p.rot_dim) break;
                  const float2 c = turn[e / 2];
                  const float a = f[e], b = f[e + 1];
                  f[e] = a * c.x - b * c.y;
                  f[e + 1] = b * c.x + a * c.y;
                }
              }
            } else if constexpr (PAIRS == kHalves) {
              const bool second = e0 >= half;
              const int from_lane = lane + (rotated ? (second ? -half : half) / kLane : 0);
#pragma unroll
              for (int e = 0; e < kLane; ++e) {
                const float b = __shfl_sync(0xFFFFFFFFu, f[e], from_lane);
                if (rotated) f[e] = fmaf(f[e], turn[e].x, b * (second ? turn[e].y : -turn[e].y));
              }
            } else {
              float g[kLane];
#pragma unroll
              for (int e = 0; e < kLane; ++e) {
                g[e] = f[e];
                const int i = e0 + e;
                if (live && i < p.rot_dim) {
                  const int other = i < half ? i + half : i - half;
                  float b = q8_to_float(here[other - e0]);
                  if (w) b = b * lift * (rms * weights[kind][other]);  // their product may be past fp32's range
                  g[e] = i < half ? f[e] * turn[e].x - b * turn[e].y : f[e] * turn[e].x + b * turn[e].y;
                }
              }
              __syncwarp();  // the output may be the input
#pragma unroll
              for (int e = 0; e < kLane; ++e) f[e] = g[e];
            }
          }
          if (kind < 2) {
            if (live && out.p) store8(dst, f);
            dst += kRows * out.head_pitch;
          }
          if constexpr (CODE != kNoCodes && kind > 0)
            write_codes<CODE, L>(kind == 2 ? p.cache.v_codes : p.cache.k_codes,
                                 kind == 2 ? p.cache.v_scale : p.cache.k_scale, at + (long long)head * p.cache.page_size,
                                 chunk, f, store && live);
        }
      }
    };
    rows(std::integral_constant<int, 0>{}, first, min(end, q_units), p.q, p.q_out, p.q_weight, p.q_heads);
    rows(std::integral_constant<int, 1>{}, max(first - q_units, 0), min(end - q_units, k_units), p.k, p.k_out, p.k_weight,
         p.kv_heads);
    if constexpr (CODE != kNoCodes)
      rows(std::integral_constant<int, 2>{}, max(first - q_units - k_units, 0), end - q_units - k_units, p.v, p.v, nullptr,
           p.kv_heads);
  }
}

template <typename T, int CODE, int L>
cudaError_t launch_heads_as(const HeadsParams& p, bool adjacent, cudaStream_t stream) {
  constexpr int kRows = 32 / L, kWarps = kHeadsThreads / 32;
  auto units_of = [](int heads) { return (heads + kRows - 1) / kRows; };
  const int units = units_of(p.q_heads) + (p.k.p ? units_of(p.kv_heads) : 0) + (CODE != kNoCodes ? units_of(p.kv_heads) : 0);
  // few tokens: their heads are shared out until there are warps for a good part of the device
  const int wanted = 152 * 2 * kWarps;
  const int shares = p.tokens >= wanted ? 1 : std::min(units, (wanted + p.tokens - 1) / p.tokens);
  const long long blocks = ((long long)p.tokens * shares + kWarps - 1) / kWarps;
  const unsigned grid = (unsigned)std::min<long long>(blocks, 152 * kBlocksPerSm);
  if (!p.turns || (adjacent && p.rot_dim % kLane == 0))
    heads_kernel<T, CODE, L, kAdjacent><<<grid, kHeadsThreads, 0, stream>>>(p, shares);
  else if (adjacent)
    heads_kernel<T, CODE, L, kLooseAdjacent><<<grid, kHeadsThreads, 0, stream>>>(p, shares);
  else if (p.rot_dim % (2 * kLane) == 0)
    heads_kernel<T, CODE, L, kHalves><<<grid, kHeadsThreads, 0, stream>>>(p, shares);
  else
    heads_kernel<T, CODE, L, kLooseHalves><<<grid, kHeadsThreads, 0, stream>>>(p, shares);
  return cudaGetLastError();
}

template <typename T, int CODE>
cudaError_t launch_heads_of(const HeadsParams& p, bool adjacent, cudaStream_t stream) {
  if (p.head_dim <= 8 * kLane) return launch_heads_as<T, CODE, 8>(p, adjacent, stream);
  if (p.head_dim <= 16 * kLane) return launch_heads_as<T, CODE, 16>(p, adjacent, stream);
  return launch_heads_as<T, CODE, 32>(p, adjacent, stream);
}

template <typename T>
cudaError_t launch_heads_in(const HeadsParams& p, int code_type, bool adjacent, cudaStream_t stream) {
  switch (code_type) {
    case Q8_INT8: return launch_heads_of<T, Q8_INT8>(p, adjacent, stream);
    case Q8_E4M3: return launch_heads_of<T, Q8_E4M3>(p, adjacent, stream);
    case Q8_INT4: return launch_heads_of<T, Q8_INT4>(p, adjacent, stream);
    default: return launch_heads_of<T, kNoCodes>(p, adjacent, stream);
  }
}

}  // namespace c3d
