// q8_heads.cu -- rows of heads on their way into attention: the norm and the rotation of queries and
// keys, their codes in a paged cache, and the cache's rows as values.
//
// A row is one token's head. L = 8, 16 or 32 lanes hold it, eight elements each, so that its sums, its
// partners in the rotation and its scale are shuffles, and every element is read once and written once:
// the memory's bandwidth is the bound. A block takes a few tokens and all their heads; the sines of
// a token's angles are taken once, into shared memory.
//
// Angles. In turns an angle is frequency / 2 pi * position, and only its fraction matters. With the
// frequency as an integer f of 2^-64 turns the fraction of f * position is the 64-bit product, whose
// overflow drops whole turns: positions of any size cost two integer products and lose nothing, where an
// fp32 product at position 10^5 is off by 4e-3 of a radian. sincospi takes it from there.
//
// Codes. The code of v is T * v / amax, to the nearest, ties to even (for 4 bits 15 * (v - lowest) / (highest -
// lowest)). With 16-bit inputs such quotients lie on ties often, so the quotient has to be right to the
// last bit: q0 = a * r with r = 1 / w rounded, then q0 + r * (a - q0 * w) with both steps fused, which
// is the correctly rounded a / w (Markstein, 1990). The product of a reciprocal alone gave 1.2% of the norm of
// 8192 x 8 x 128 bf16 keys in codes that went the other way.
#include "q8_attn_internal.h"
#include "q8_common.cuh"

namespace c3d {

constexpr int kHeadsThreads = 256;
constexpr int kLane = 8;             // elements of a row that a lane holds
constexpr int kMostPairs = Q8_MAX_HEAD_DIM / 2;
constexpr int kMostTokens = 16;      // of a block
constexpr int kNoCodes = 0;

// ------------------------------------------------------------------ eight values of a row
__device__ __forceinline__ void load8(const float* p, float (&f)[kLane]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[kLane]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const T* h = reinterpret_cast<const T*>(&a);
#pragma unroll
  for (int e = 0; e < kLane; ++e) f[e] = q8_to_float(h[e]);
}
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
// The largest magnitude as bits, whose order is that of the magnitudes with every NaN above them.
template <int L>
__device__ __forceinline__ unsigned row_amax(const float (&f)[kLane]) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < kLane; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

// a / w rounded once, given r = 1 / w rounded.
__device__ __forceinline__ float quotient(float a, float w, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, w, a), r, q);
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
  const unsigned amax_bits = row_amax<L>(f);
  if constexpr (CODE == Q8_INT4) {
    float lo = f[0], hi = f[0];
#pragma unroll
    for (int e = 1; e < kLane; ++e) {
      lo = fminf(lo, f[e]);
      hi = fmaxf(hi, f[e]);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    }
    const float width = hi - lo;
    const bool bad = amax_bits >= 0x7F800000u || width > 3.4028234e38f;
    const bool flat = !(width > 0.0f) || bad;
    const float lift = lift_of(width);
    const float w = flat ? 1.0f : width * lift, r = __frcp_rn(w);
    unsigned word = 0;
#pragma unroll
    for (int e = 0; e < kLane; ++e) {
      const float a = flat ? 0.0f : (f[e] - lo) * lift * 15.0f;
      word |= (unsigned)__float2int_rn(quotient(a, w, r)) << (4 * e);
    }
    if (!store) return;
    *reinterpret_cast<unsigned*>(codes + (row * L + chunk) * (kLane / 2)) = word;
    if (chunk == 0)
      *reinterpret_cast<float2*>(scales + 2 * row) =
          make_float2(bad ? __int_as_float(0x7FFFFFFF) : flat ? 1.0f : __fdiv_rn(width, 15.0f),
                      bad ? 0.0f : lo);
  } else {
    constexpr float kTop = CODE == Q8_INT8 ? 127.0f : 448.0f;
    const float amax = __uint_as_float(amax_bits);
    const bool bad = amax_bits >= 0x7F800000u, flat = bad || amax_bits == 0;
    const float lift = lift_of(amax);
    const float w = flat ? 1.0f : amax * lift, r = __frcp_rn(w);
    float q[kLane];
#pragma unroll
    for (int e = 0; e < kLane; ++e) q[e] = flat ? 0.0f : quotient(f[e] * lift * kTop, w, r);
    uint2 word = make_uint2(0, 0);
    if constexpr (CODE == Q8_INT8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        word.x |= ((unsigned)__float2int_rn(q[e]) & 0xFFu) << (8 * e);
        word.y |= ((unsigned)__float2int_rn(q[4 + e]) & 0xFFu) << (8 * e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        word.x |= (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(q[2 * e], q[2 * e + 1]), __NV_SATFINITE,
                                                     __NV_E4M3) << (16 * e);
        word.y |= (unsigned)__nv_cvt_float2_to_fp8x2(make_float2(q[4 + 2 * e], q[5 + 2 * e]),
                                                     __NV_SATFINITE, __NV_E4M3) << (16 * e);
      }
    }
    if (!store) return;
    *reinterpret_cast<uint2*>(codes + (row * L + chunk) * kLane) = word;
    if (chunk == 0)
      scales[row] = bad ? __int_as_float(0x7FFFFFFF) : flat ? 1.0f : __fdiv_rn(amax, kTop);
  }
}

// ------------------------------------------------------------------ the rows of heads
// How pairs lie: next to each other; half of the rotated part apart, in whole lanes; the same, not in whole
// lanes (the partner is then read a second time).
enum { kAdjacent, kHalves, kLooseHalves };

template <typename T, int CODE, int L, int PAIRS>
__global__ void __launch_bounds__(kHeadsThreads) heads_kernel(const HeadsParams p, int block_tokens) {
  __shared__ float2 turned[kMostTokens * kMostPairs];  // cosine and sine, [token][pair]
  const int t0 = blockIdx.x * block_tokens;
  const int tokens = min(block_tokens, p.tokens - t0);
  const int half = p.rot_dim / 2, pairs = (half + kLane - 1) / kLane * kLane;
  if (p.turns) {
    for (int i = threadIdx.x; i < tokens * pairs; i += kHeadsThreads) {
      const int t = i / pairs, j = i - t * pairs;
      float s = 0.0f, c = 1.0f;
      if (j < half) {
        int axis = p.axis ? p.axis[j] : 0;
        if (axis >= p.axes) axis = 0;
        const long long pos = p.positions[axis * p.positions_pitch + t0 + t];
        const long long turn = (long long)(p.turns[j] * (unsigned long long)pos);
        sincospif((float)turn * 0x1p-63f, &s, &c);
      }
      turned[i] = make_float2(c, s);
    }
  }
  __syncthreads();
  constexpr int kRows = kHeadsThreads / L;
  const int chunk = threadIdx.x % L, e0 = chunk * kLane;
  const bool mine = e0 < p.head_dim;
  const int k_heads = p.k.p ? p.kv_heads : 0, v_heads = CODE != kNoCodes ? p.kv_heads : 0;
  const int heads = p.q_heads + k_heads + v_heads;
  const int rows = tokens * heads;
  const int share = (rows + gridDim.y - 1) / gridDim.y;
  const int first = blockIdx.y * share, end = min(rows, first + share);
  // whole warps go around together
  for (int base = first; base < end; base += kRows) {
    const int row = base + threadIdx.x / L;
    const bool live = row < end;
    const int t = live ? row / heads : 0, h = live ? row - t * heads : 0;
    const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + k_heads;
    const int kv = is_q ? 0 : is_v ? h - p.q_heads - k_heads : h - p.q_heads;
    const Heads& m = is_q ? p.q : is_v ? p.v : p.k;
    const T* src = static_cast<const T*>(m.p) + (t0 + t) * m.pitch + (is_q ? h : kv) * m.head_pitch;
    const void* weight = is_v ? nullptr : is_q ? p.q_weight : p.k_weight;
    float f[kLane] = {};
    if (live && mine) load8(src + e0, f);
    float rms = 1.0f;
    if (p.q_weight || p.k_weight) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < kLane; ++e) sum = fmaf(f[e], f[e], sum);
      sum = row_sum<L>(sum);
      float lift = 1.0f;
      const bool lifted = !(sum <= 0x1p100f) || (sum < 0x1p-80f && p.eps < 0x1p-100f);
      if (__any_sync(0xFFFFFFFFu, lifted)) {
        if (lifted) lift = sum < 1.0f ? 0x1p100f : 0x1p-100f;
        float again = 0.0f;
#pragma unroll
        for (int e = 0; e < kLane; ++e) again = fmaf(f[e] * lift, f[e] * lift, again);
        again = row_sum<L>(again);
        if (lifted) sum = again;
      }
      if (weight) {
        const float mean = sum / p.head_dim + p.eps * lift * lift;
        rms = mean == 0.0f ? 0.0f : rsqrtf(mean);
#pragma unroll
        for (int e = 0; e < kLane; ++e)
          f[e] = f[e] * lift * rms *
                 (mine ? q8_load_value(weight, p.weight_type, e0 + e) : 0.0f);
        rms *= lift;
      }
    }
    if (p.turns) {
      const float2* cs = turned + t * pairs;
      const bool rotated = !is_v && e0 < p.rot_dim;
      if constexpr (PAIRS == kAdjacent) {
        if (rotated) {
#pragma unroll
          for (int e = 0; e < kLane; e += 2) {
            const float2 c = cs[(e0 + e) / 2];
            const float a = f[e], b = f[e + 1];
            f[e] = a * c.x - b * c.y;
            f[e + 1] = b * c.x + a * c.y;
          }
        }
      } else if constexpr (PAIRS == kHalves) {
        const bool second = e0 >= half;
        const int partner = second ? chunk - half / kLane : chunk + half / kLane;
        const int lane = (threadIdx.x & 31) - chunk + (rotated ? partner : chunk);
        const int j0 = second ? e0 - half : e0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
          const float b = __shfl_sync(0xFFFFFFFFu, f[e], lane);
          if (rotated) {
            const float2 c = cs[j0 + e];
            f[e] = second ? f[e] * c.x + b * c.y : f[e] * c.x - b * c.y;
          }
        }
      } else {
        float g[kLane];
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
          g[e] = f[e];
          const int i = e0 + e;
          if (live && rotated && i < p.rot_dim) {
            const int j = i < half ? i : i - half, other = i < half ? i + half : j;
            float b = q8_to_float(src[other]);
            if (weight) b = b * rms * q8_load_value(weight, p.weight_type, other);
            const float2 c = cs[j];
            g[e] = i < half ? f[e] * c.x - b * c.y : f[e] * c.x + b * c.y;
          }
        }
        __syncwarp();  // the output may be the input
#pragma unroll
        for (int e = 0; e < kLane; ++e) f[e] = g[e];
      }
    }
    const Heads& out = is_q ? p.q_out : p.k_out;
    if (live && mine && !is_v && out.p)
      store8(static_cast<T*>(out.p) + (t0 + t) * out.pitch + (is_q ? h : kv) * out.head_pitch + e0, f);
    if constexpr (CODE != kNoCodes) {
      const long long slot = live && !is_q ? p.slots[t0 + t] : -1;
      const bool store = slot >= 0 && slot < (long long)p.cache.slots;
      const unsigned page = (unsigned)slot / (unsigned)p.cache.page_size;
      const long long at = ((long long)page * p.kv_heads + kv) * p.cache.page_size +
                           ((unsigned)slot - page * p.cache.page_size);
      write_codes<CODE, L>(is_v ? p.cache.v_codes : p.cache.k_codes,
                           is_v ? p.cache.v_scale : p.cache.k_scale, at, chunk, f, store);
    }
  }
}

template <typename T, int CODE, int L>
cudaError_t launch_heads_as(const HeadsParams& p, bool adjacent, cudaStream_t stream) {
  const int heads = p.q_heads + (p.k.p ? p.kv_heads : 0) + (CODE != kNoCodes ? p.kv_heads : 0);
  constexpr int kRows = kHeadsThreads / L;
  const int block_tokens = heads >= kRows ? 1 : min(kMostTokens, (kRows + heads - 1) / heads);
  const int blocks = (p.tokens + block_tokens - 1) / block_tokens;
  const int passes = (block_tokens * heads + kRows - 1) / kRows;
  const int split = blocks >= 2 * 152 ? 1 : min(passes, (2 * 152 + blocks - 1) / blocks);
  const dim3 grid(blocks, split);
  if (adjacent || !p.turns)
    heads_kernel<T, CODE, L, kAdjacent><<<grid, kHeadsThreads, 0, stream>>>(p, block_tokens);
  else if (p.rot_dim % (2 * kLane) == 0)
    heads_kernel<T, CODE, L, kHalves><<<grid, kHeadsThreads, 0, stream>>>(p, block_tokens);
  else
    heads_kernel<T, CODE, L, kLooseHalves><<<grid, kHeadsThreads, 0, stream>>>(p, block_tokens);
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
  const bool is_v = (int)blockIdx.y >= c.kv_heads;
  const int head = blockIdx.y - (is_v ? c.kv_heads : 0);
  const uint8_t* codes = is_v ? c.v_codes : c.k_codes;
  const float* scales = is_v ? c.v_scale : c.k_scale;
  const Heads& out = is_v ? p.v : p.k;
  const int chunk = threadIdx.x % L;
  const long long t0 = (long long)blockIdx.x * (kRows * kReadRows) + threadIdx.x / L;
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
  const dim3 grid((p.tokens + rows - 1) / rows, 2 * p.cache.kv_heads);
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
