// q8_linear_tc.cu -- products of 8-bit codes on the tensor cores (tcgen05, CTA pairs):
// y[m][n] = scale_x[m] * scale_w[n] * sum_k x[m][k] * w[n][k] + bias[n].
//
// The channels are the rows of the MMA (M = 256 over the pair, 128 a CTA) and the tokens its columns
// (N = block_t, 32 to 256), so that a batch of any size fills whole rows: the accumulator has a
// channel in each TMEM lane and a token in each column, and a warp's stores of one token cover 32
// consecutive channels of y.
//
// e4m3: both operands go from global memory to shared memory by TMA and into kind::f8f6f4. A stage
// holds 256 codes of K: with 128 the issuing warp's 520 cycles a stage (a wait 160, the MMAs 30 each,
// a commit 60) were as long as the stage's MMAs take at 256 tokens.
//
// int8: sm_103a has no fast integer pipe, but an int8 code is exact in f16 (an 11-bit significand),
// a product of two is an integer of at most 2^14, and the fp32 accumulator holds their sums exactly
// up to 2^24. So the product runs as kind::f16, at the f16 rate, on codes turned into f16:
//   - w stays 8 bits wide as far as shared memory. Converter warps read a stage's codes there, turn
//     them into f16 (a byte under the exponent of 1024, minus 1152 with the sign bit flipped, a
//     permute and a subtraction for each two codes) and write them to TMEM, from where the MMA takes
//     its A operand: in shared memory they would come on top of the codes, x and the MMA's reads,
//     which fill its 128 bytes a cycle at 256 tokens;
//   - x is expanded to f16 by a small kernel first, 3 bytes of traffic a code, and loaded as such.
//     Turned by four or eight more warps of this kernel it is read back into shared memory next to
//     everything else: 256 x 6144 x 4096 takes 26 us so and 22 with the expansion, 64 x 8192 x 4096
//     15.3 and 14.4, 8192 x 4096 x 8192 408 and 328;
//   - a K block has one barrier that says that its w and x are there and one commit that frees both,
//     whatever the depths of their rings, and holds 256 codes in tiles of up to 128 tokens: the
//     issuing warp takes about 160 cycles for a wait, 60 for a commit and 30 for an MMA, as long as
//     those MMAs take. (With a wait and a commit for each 32 codes a box of 128 took 2500 cycles.) For
//     the same reason a converter's visit covers a whole row of a box there, and four groups of four
//     warps take the boxes by turns; in larger tiles, where TMEM holds two or three boxes of w, the
//     shorter way of half a row a thread matters more, and two groups of eight take turns.
//
// Few tiles: a tile is split along K over the pairs of one cluster (4, 6 or 8 CTAs). Each CTA leaves its
// partial sums in its own shared memory and adds up its share of the tokens from all of them over
// distributed shared memory, in the order of the slices: nothing passes through global memory, and
// a result does not depend on which slice is ready first.
//
// Roles of a CTA: warps 0-3 epilogue, then 16 converters of w and the copies of x (int8), the other
// copies, and the MMAs (the leader CTA's).
// Every wait is bounded; one that runs out records a status bit and both CTAs wind down.
#include <algorithm>

#include "conv_common.cuh"
#include "q8_common.cuh"

namespace c3d {

constexpr int kTcWWarps = 16;                       // converters (int8)
constexpr int kTcXWarp = 4 + kTcWWarps;             // x's copies (int8)
template <bool kInt8>
constexpr int kTcTmaWarpOf = kInt8 ? kTcXWarp + 1 : 4;
template <bool kInt8>
constexpr int kTcThreads = (kTcTmaWarpOf<kInt8> + 2) * 32;
// Quartets of warps that share a box's rows by halves, and converter groups that take boxes by turns.
template <int kBoxes>
constexpr int kTcParts = kBoxes == 1 ? 2 : 1;
template <int kBoxes>
constexpr int kTcGroups = kTcWWarps / 4 / kTcParts<kBoxes>;
constexpr int kTcWBytes = kTcWBoxRows * kTcBlockK;  // a box of w's codes: 16 KB a CTA
constexpr int kTcMaxStages = 8;
constexpr int kTcSmemBudget = 208 * 1024;
constexpr int kTcTmemCols = 512;
constexpr int kTcSlotCols = kTcBlockK / 2;          // a box of w as f16 in TMEM: 64 columns
constexpr int kTcDepth = 8;                         // K blocks under way: no ring is deeper
constexpr uint64_t kTcAbortSettleNs = 2ull * 1000 * 1000;  // let copies in flight land on abort

constexpr int kTcBoxBytes = kTcYBoxBytes;           // one staging buffer of an epilogue warp
constexpr int kTcStaging = 4 * 2 * kTcBoxBytes;     // (two boxes of 4 KB and 16 bytes a row otherwise)
constexpr int kTcBars = 2 * kTcMaxStages + 2 * kTcDepth + 5;
constexpr int kTcBarBytes = 512;                    // barriers, the TMEM address, the abort flag
static_assert(kTcBars * 8 + 8 <= kTcBarBytes);

// A box of x's codes of one CTA (half of the tile's tokens), or of half as many as f16. Either way a
// stage (e4m3) or a slot (int8) of x is two.
__host__ __device__ inline uint32_t tc_x_bytes(int block_t) {
  return (uint32_t)(block_t / 2) * kTcBlockK;
}

// What lies in shared memory before the stages, which start on 1024 bytes: the barriers, the staging
// of the epilogue, the scales of two tiles' tokens.
__host__ __device__ inline uint32_t tc_head_bytes(int block_t) {
  return (uint32_t)(kTcBarBytes + kTcStaging + 2 * block_t * 4 + 1023) & ~1023u;
}

// One work unit: a tile and a slice [kb0, kb1) of the K blocks. Tiles are taken in groups of
// kTcGroup channel tiles, tokens before the next group, so that the tiles of one wave share their
// operands in L2 (8 x ~10 of them read 18 operand tiles; in plain order a wide w is read again for
// each tile of tokens).
constexpr int kTcGroup = 8;
struct TcTile {
  int m_tile, n_tile;
};
__device__ __forceinline__ TcTile tc_tile(const LinearParams& p, int tile) {
  TcTile r;
  const int per_group = kTcGroup * p.m_tiles;
  const int group = tile / per_group;
  const int rest = tile - group * per_group;
  const int width = min(kTcGroup, p.n_tiles - group * kTcGroup);
  r.m_tile = rest / width;
  r.n_tile = group * kTcGroup + (rest - r.m_tile * width);
  return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Four consecutive channels of y (element i is a multiple of 4 elements into an aligned row).
__device__ __forceinline__ void store_y4(const LinearParams& p, long long i, const float (&v)[4]) {
  if (p.y_type == Q8_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.y) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (p.y_type == Q8_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<__half*>(p.y) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// Adds up the partial sums that the cluster's CTAs of this rank hold, [token][128 channels] at the
// same offset of their shared memory, for this CTA's share of the tile's tokens. All threads.
__device__ __forceinline__ void tc_join(const LinearParams& p, const TcTile& t, uint32_t part,
                                        int split, uint32_t rank) {
  const int lane = threadIdx.x & 31;
  const long long n = (long long)t.n_tile * kTcChannels + rank * 128 + 4 * lane;
  const long long m0 = (long long)t.m_tile * p.block_t;
  const int tokens = (int)min((long long)p.block_t, p.M - m0);
  const int share = (p.block_t + p.splits - 1) / p.splits;
  if (n >= p.N) return;
  const int have = (int)min(4LL, p.N - n);
  ScaleBias sc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long c = min(n + i, (long long)p.N - 1);
    sc[i] = ScaleBias{__ldg(p.scale_w + c), p.bias ? q8_load_value(p.bias, p.bias_type, c) : 0.0f};
  }
  const int end = min(tokens, (split + 1) * share);
  for (int c = split * share + (threadIdx.x >> 5); c < end; c += blockDim.x / 32) {
    const uint32_t at = part + (uint32_t)(c * 128 + 4 * lane) * 4u;
    float4 a[kTcMaxSplits];
#pragma unroll
    for (int s = 0; s < kTcMaxSplits; ++s)
      if (s < p.splits) a[s] = ld_cluster_f4(map_to_cta(at, 2u * s + rank));
#pragma unroll
    for (int s = 1; s < kTcMaxSplits; ++s)
      if (s < p.splits) {
        a[0].x += a[s].x;
        a[0].y += a[s].y;
        a[0].z += a[s].z;
        a[0].w += a[s].w;
      }
    const float sx = __ldg(p.scale_x + m0 + c);
    const float v[4] = {sc[0](a[0].x, sx), sc[1](a[0].y, sx), sc[2](a[0].z, sx), sc[3](a[0].w, sx)};
    const long long i = (m0 + c) * p.y_pitch + n;
    if (p.y_vec && have == 4) {
      store_y4(p, i, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < have) q8_store_value(p.y, p.y_type, i + e, v[e]);
    }
  }
}

// `rows` rows of y from the staging of the four epilogue warps, for a y off the 16-byte grid. A row's
// 128 channels are staged kShiftPitch bytes apart, as far behind a 16-byte boundary as in y, so that
// both divide into the same 16-byte chunks: one at each end that the row shares with its neighbours
// (as many elements as one chunk together, stored one by one) and those between.
template <typename Y>
constexpr int kShiftPitch = 128 * (int)sizeof(Y) + 16;
template <typename Y>
constexpr int kShiftRows = 4096 / (128 * (int)sizeof(Y));
__device__ __forceinline__ uint32_t behind16(const void* p) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
}
template <typename Y>
__device__ __forceinline__ void store_shifted(Y* first, long long pitch, int rows,
                                              const uint8_t* buf) {
  constexpr int kEdge = 16 / (int)sizeof(Y), kChunks = 128 / kEdge;
#pragma unroll
  for (int i = threadIdx.x; i < kShiftRows<Y> * kChunks; i += 128) {
    const int j = i / kChunks, chunk = i % kChunks;
    if (j >= rows || chunk == 0) continue;
    uint8_t* row = reinterpret_cast<uint8_t*>(first + j * pitch);
    *reinterpret_cast<uint4*>(row - behind16(row) + 16 * chunk) =
        *reinterpret_cast<const uint4*>(buf + j * kShiftPitch<Y> + 16 * chunk);
  }
#pragma unroll
  for (int i = threadIdx.x; i < kShiftRows<Y> * kEdge; i += 128) {
    const int j = i / kEdge, e = i % kEdge;
    if (j >= rows) continue;
    Y* row = first + j * pitch;
    const int behind = (int)behind16(row);
    const int channel = e * (int)sizeof(Y) < 16 - behind ? e : 128 - kEdge + e;
    row[channel] = *reinterpret_cast<const Y*>(buf + j * kShiftPitch<Y> + behind +
                                               channel * (int)sizeof(Y));
  }
}

// One warp's part of the epilogue of a tile of a 16-bit y on the 16-byte grid: channels n0 .. n0 + 31,
// 32 tokens at a time. TMEM is read by 16 lanes x 8 columns, which leaves two tokens of four channels
// with each thread of eight: as pairs they are scaled and rounded two by one instruction, and stmatrix
// transposes them on their way to the staging, eight tokens of the 32 channels by one instruction. A
// thread that held a channel's 32 tokens took 32 two-byte stores and as many roundings for them: 4096 x
// 8192 x 128 e4m3 28.0 us. The staging is a box of y's map, [token][32 channels] with the map's
// 64-byte swizzle (without it the eight rows of a matrix meet in two banks of 16 bytes).
template <typename Y, typename Release>
__device__ __forceinline__ void tc_epilogue16(const LinearParams& p, const CUtensorMap* ymap,
                                              uint32_t trow, const float* scale, ScaleBias sc,
                                              int tokens, long long m0, int n0, uint8_t* own,
                                              uint32_t& boxes, Release release) {
  const int lane = threadIdx.x & 31;
  float2 w[4], bias[4];  // of the channels n0 + 8 q + lane / 4
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float a = __shfl_sync(0xFFFFFFFFu, sc.w, 8 * q + lane / 4);
    const float b = __shfl_sync(0xFFFFFFFFu, sc.bias, 8 * q + lane / 4);
    w[q] = make_float2(a, a);
    bias[q] = make_float2(b, b);
  }
  // this thread's row of the matrix that it addresses: token lane % 8, channels 8 (lane / 8) and on
  const uint32_t row = (uint32_t)((lane % 8) * 64 + (((lane / 8) ^ ((lane % 8) >> 1)) << 4));
  for (int c = 0; c < tokens; c += 32) {
    uint32_t r[2][16];
    tmem_ld_16x256b_x4(trow + c, r[0]);
    tmem_ld_16x256b_x4(trow + c + (16u << 16), r[1]);
    tmem_ld_wait();
    if (c + 32 >= tokens) release();
    const uint32_t buf = smem_u32(own + (boxes++ & 1u) * kTcBoxBytes);
    if (lane == 0) bulk_wait_group_read<1>();  // the store from this buffer, two boxes ago
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // of eight tokens
      const float2 sx = *reinterpret_cast<const float2*>(scale + c + 8 * g + 2 * (lane % 4));
      uint32_t h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* acc = r[q / 2] + 4 * g + 2 * (q % 2);
        const float2 a = make_float2(__uint_as_float(acc[0]), __uint_as_float(acc[1]));
        h[q] = q8_pack2<Y>(q8_fma2(q8_mul2(a, sx), w[q], bias[q]));
      }
      stmatrix_x4_trans(buf + 512u * g + row, h);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(ymap, buf, n0, (int)m0 + c);
      bulk_commit_group();
    }
  }
}

// One warp's part of the epilogue of a tile: a channel a lane, channels n0 .. n0 + 31. A 16-bit y on the
// 16-byte grid goes as above. Of an fp32 one 16 tokens are staged in shared memory as [token][32
// channels], in the warp's two buffers by turns (`boxes` counts them), and leave by a TMA store that
// y's extents bound. A y off the 16-byte grid is staged by the four warps together and stored as
// above; the last channels of a y whose rows end inside 16 bytes leave straight from the lanes (a TMA
// store was seen to write the whole of the 16 bytes that hold a row's last element). With all of y
// stored from the lanes the 67 MB of an e4m3 product of 4096 x 8192 x 4096 took 26 of its 105 us, and
// 6621 x 8192 x 640 to fp32 123 us instead of 81. `release` is called once the accumulator has been read.
template <typename Y, typename Release>
__device__ __forceinline__ void tc_epilogue(const LinearParams& p, const CUtensorMap* ymap,
                                            uint32_t trow, const float* scale, ScaleBias sc,
                                            int tokens, long long m0, int n0, uint8_t* staging,
                                            uint32_t& boxes, Release release) {
  constexpr int kRows = kTcBoxBytes / (32 * (int)sizeof(Y));
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const bool by_tma = p.y_tma && n0 < p.N &&
                      (n0 + 32 <= p.N || (long long)p.N * (int)sizeof(Y) % 16 == 0);
  const bool shifted = !p.y_tma && n0 - 32 * warp + 128 <= p.N;  // the same for the four warps
  uint8_t* own = staging + warp * 2 * kTcBoxBytes;
  if constexpr (sizeof(Y) == 2) {
    if (by_tma) {
      tc_epilogue16<Y>(p, ymap, trow, scale, sc, tokens, m0, n0, own, boxes, release);
      return;
    }
  }
  for (int c = 0; c < tokens; c += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(trow + c, r);
    tmem_ld_wait();
    if (c + 32 >= tokens) release();
    if (n0 >= p.N) continue;
    float v[32];  // before the first store: the compiler cannot tell the staging from the scales
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 sx = *reinterpret_cast<const float4*>(scale + c + j);
      v[j] = sc(__uint_as_float(r[j]), sx.x);
      v[j + 1] = sc(__uint_as_float(r[j + 1]), sx.y);
      v[j + 2] = sc(__uint_as_float(r[j + 2]), sx.z);
      v[j + 3] = sc(__uint_as_float(r[j + 3]), sx.w);
    }
    if (shifted) {
      constexpr int kStep = kShiftRows<Y>;
      Y* first = static_cast<Y*>(p.y) + (m0 + c) * p.y_pitch + (n0 - 32 * warp);
#pragma unroll
      for (int h = 0; h < 32; h += kStep) {
        if (c + h >= tokens) break;
        uint8_t* buf = staging + (boxes++ & 1u) * (kStep * kShiftPitch<Y>);
#pragma unroll
        for (int j = 0; j < kStep; ++j)
          *reinterpret_cast<Y*>(buf + j * kShiftPitch<Y> + behind16(first + (h + j) * p.y_pitch) +
                                threadIdx.x * (int)sizeof(Y)) = q8_from_float<Y>(v[h + j]);
        // the other buffer is written once every warp is past this barrier, and so has read it
        named_barrier_sync(1, 128);
        store_shifted<Y>(first + h * p.y_pitch, p.y_pitch, min(kStep, tokens - c - h), buf);
      }
      continue;
    }
    if (!by_tma) {
      Y* dst = static_cast<Y*>(p.y) + (m0 + c) * p.y_pitch + n0 + lane;
      if (n0 + lane < p.N) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < tokens)
            dst[j * p.y_pitch] = q8_from_float<Y>(v[j]);
      }
      continue;
    }
#pragma unroll
    for (int h = 0; h < 32; h += kRows) {
      if (c + h >= tokens) break;
      uint8_t* buf = own + (boxes++ & 1u) * kTcBoxBytes;
      if (lane == 0) bulk_wait_group_read<1>();  // the store from this buffer, two boxes ago
      __syncwarp();
      Y* to = reinterpret_cast<Y*>(buf) + lane;
#pragma unroll
      for (int j = 0; j < kRows; ++j) to[32 * j] = q8_from_float<Y>(v[h + j]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(ymap, smem_u32(buf), n0, (int)m0 + c + h);
        bulk_commit_group();
      }
    }
  }
}

// kBoxes: boxes of 128 codes that make a K block.
template <bool kInt8, int kBoxes>
__global__ void __launch_bounds__(kTcThreads<kInt8>, 1)
    linear_q8_tc_kernel(const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ CUtensorMap ymap, const LinearParams p) {
  constexpr int kTcTmaWarp = kTcTmaWarpOf<kInt8>, kTcMmaWarp = kTcTmaWarp + 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
  const int S = p.stages;
  // a stage of w's codes is a box (int8) or a K block (e4m3)
  constexpr uint32_t kWStage = kInt8 ? kTcWBytes : 2 * kTcWBytes;
  const uint32_t x_step = (uint32_t)kBoxes * (kInt8 ? 2u : 1u) * tc_x_bytes(p.block_t);
  const uint32_t x_bytes = tc_x_bytes(p.block_t);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint8_t* sBox = smem + kTcBarBytes;                                // the epilogue's staging
  float* sScale = reinterpret_cast<float*>(sBox + kTcStaging);       // [2][block_t]
  uint8_t* sW = smem + tc_head_bytes(p.block_t);
  // x's tiles: codes in the stages (e4m3), or f16 in slots of their own
  uint8_t* sX = sW + (size_t)S * kWStage;
  // Barriers (those marked L: the leader's are used). full[S]: a stage's copies have landed (e4m3 L:
  // both CTAs'; int8: this CTA's). empty[S]: read by the MMAs (e4m3) or the converters (int8).
  // int8, for K block i of all, at i % kTcDepth: ready L: its w and x are there as f16. done: its MMAs
  // have completed. acc_full, acc_empty L. drain.
  const uint32_t bars_u32 = smem_u32(bars);
  auto bar_at = [&](int i) { return bars_u32 + 8u * (uint32_t)i; };
  auto full = [&](int s) { return bar_at(s); };
  auto empty = [&](int s) { return bar_at(kTcMaxStages + s); };
  auto ready = [&](uint32_t i) { return bar_at(2 * kTcMaxStages + (int)(i % kTcDepth)); };
  auto done = [&](uint32_t i) { return bar_at(2 * kTcMaxStages + kTcDepth + (int)(i % kTcDepth)); };
  auto parity = [](uint32_t i) { return (i / kTcDepth) & 1u; };
  auto acc_full = [&](int b) { return bar_at(kTcBars - 5 + b); };
  auto acc_empty = [&](int b) { return bar_at(kTcBars - 3 + b); };
  const uint32_t drain_bar = bar_at(kTcBars - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kTcBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a cluster is 2 * splits CTAs: pair `split` of it takes that slice of a tile's K blocks
  const uint32_t cluster_rank = cluster_ctarank();
  const uint32_t rank = cluster_rank & 1u;  // within the pair
  const int split = (int)(cluster_rank >> 1);
  const bool leader = rank == 0;
  const uint32_t leader_bars = map_to_cta(bars_u32, cluster_rank & ~1u);
  const uint16_t pair_mask = (uint16_t)(0x3u << (cluster_rank & ~1u));
  const int first_tile = blockIdx.x / (2 * p.splits), tile_step = gridDim.x / (2 * p.splits);
  const int num_tiles = p.m_tiles * p.n_tiles;
  const int kb0 = (int)((long long)split * p.k_blocks / p.splits);
  const int kb1 = (int)((long long)(split + 1) * p.k_blocks / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kInt8 ? 4 * kTcParts<kBoxes> : 1);  // a converter group, or a commit
    }
    for (uint32_t i = 0; i < kTcDepth; ++i) {
      // both CTAs' converters, and the copies of x
      mbar_init(ready(i), 2 * 4 * kTcParts<kBoxes> * kBoxes + 1);
      mbar_init(done(i), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 2 * 4);  // an epilogue warp's arrival each, of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTcMmaWarp) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTcTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kTcTmaWarp && lane == 0) {
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&xmap);
    if (p.y_tma) prefetch_tensormap(&ymap);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before anyone signals across the pair
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t slots_base = tmem_base + (uint32_t)(2 * p.block_t);
  pdl_wait_primary();
  pdl_launch_dependents();
  const AbortState ab{abort_flag, p.status, p.timeout_ns};

  if (warp < 4) {
    // ------------------------------------------------------------------------------ epilogue
    Ring acc;
    uint32_t boxes = 0;
    // The scales and biases of the next tile are loaded while this one's sums are stored: a tile of
    // few K blocks otherwise waits for them (4096 x 8192 x 128 e4m3 25.7 us, 24.7 so). For int8 that
    // makes registers spill (36.8 us, 38.1 so).
    constexpr bool kAhead = !kInt8;
    float next_x[2], next_w, next_bias;
    auto load_scales = [&](int u) {
      const TcTile un = tc_tile(p, u);
      const long long n = (long long)un.n_tile * kTcChannels + rank * 128 + threadIdx.x;
      const long long m = (long long)un.m_tile * p.block_t + threadIdx.x;
      const long long end = min((long long)un.m_tile * p.block_t + p.block_t, (long long)p.M);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        next_x[i] = m + 128 * i < end ? __ldg(p.scale_x + m + 128 * i) : 0.0f;
      next_w = next_bias = 0.0f;
      if (n < p.N) {
        next_w = __ldg(p.scale_w + n);
        if (p.bias) next_bias = q8_load_value(p.bias, p.bias_type, n);
      }
    };
    if (kAhead && first_tile < num_tiles) load_scales(first_tile);
    for (int u = first_tile; u < num_tiles; u += tile_step) {
      const TcTile un = tc_tile(p, u);
      const long long m0 = (long long)un.m_tile * p.block_t;
      const int tokens = (int)min((long long)p.block_t, p.M - m0);
      if (!kAhead) load_scales(u);
      // the scales of the tile before the last: that tile lies behind every warp that has come to
      // the last one's barrier
      float* scale = sScale + acc.stage * p.block_t;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if ((int)threadIdx.x + 128 * i < p.block_t) scale[threadIdx.x + 128 * i] = next_x[i];
      const ScaleBias sc{next_w, next_bias};
      if (kAhead && u + tile_step < num_tiles) load_scales(u + tile_step);
      // the four warps go on or stop together: they share the tokens' scales
      const bool ok = tc_wait(acc_full(acc.stage), acc.phase, ab, kStatusWaitAccFull);
      if (!named_barrier_and(1, 128, ok)) break;
      tc_fence_after();
      const uint32_t trow = tmem_base + (uint32_t)(acc.stage * p.block_t) + ((uint32_t)(warp * 32) << 16);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          mbar_arrive_cluster_tmem(leader_bars + (acc_empty(acc.stage) - bars_u32));
      };
      const int n0 = un.n_tile * kTcChannels + (int)rank * 128 + warp * 32;
      if (p.splits > 1) {
        // the pipeline's stages are free: every copy of this pair has been consumed
        float* part = reinterpret_cast<float*>(sW) + threadIdx.x;
        for (int c = 0; c < p.block_t; c += 32) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(trow + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) part[(c + j) * 128] = __uint_as_float(r[j]);
        }
        release();
      } else if (p.y_type == Q8_F32) {
        tc_epilogue<float>(p, &ymap, trow, scale, sc, tokens, m0, n0, sBox, boxes, release);
      } else if (p.y_type == Q8_BF16) {
        tc_epilogue<__nv_bfloat16>(p, &ymap, trow, scale, sc, tokens, m0, n0, sBox, boxes, release);
      } else {
        tc_epilogue<__half>(p, &ymap, trow, scale, sc, tokens, m0, n0, sBox, boxes, release);
      }
      acc.next(2);
    }
    if (lane == 0) bulk_wait_group_all();  // the stores have read their buffers
  } else if (warp < kTcTmaWarp) {
    // ---------------------------------------------------------------------------- converters
    if (kInt8 && warp < kTcXWarp) {
      const int quad = warp & 3;
      constexpr uint32_t kGroups = kTcGroups<kBoxes>;
      constexpr int kParts = kTcParts<kBoxes>, kChunks = 8 / kParts;
      const uint32_t group = (uint32_t)(warp - 4) >> (kParts == 2 ? 3 : 2);
      const int part = kParts == 2 ? ((warp - 4) >> 2) & 1 : 0;
      const int row = quad * 32 + lane;
      const uint32_t dst0 = slots_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(32 * part);
      const uint32_t w_slots = (uint32_t)p.w_slots;
      // The boxes of all tiles are counted through; this group takes every kGroups-th. The number of
      // stages is a multiple of that, so a stage is always the same group's: were it another's next,
      // that group could come to wait for a phase two ahead of the barrier's, which a parity cannot
      // tell from one that is over.
      uint32_t box = group, stage = group, stage_phase = 0, slot = group % w_slots;
      const uint32_t tiles =
          first_tile < num_tiles ? (uint32_t)((num_tiles - 1 - first_tile) / tile_step + 1) : 0u;
      const uint32_t end = tiles * (uint32_t)((kb1 - kb0) * kBoxes);
      for (; box < end; box += kGroups) {
        const uint32_t step = box / kBoxes;
        if (!tc_wait(full((int)stage), stage_phase, ab, kStatusWaitFull)) break;
        const uint8_t* src = sW + stage * kWStage + row * kTcBlockK;
        uint4 c[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)  // 16-byte chunk i, where the swizzle put it
          c[i] = *reinterpret_cast<const uint4*>(src + (((kChunks * part + i) ^ (row & 7)) << 4));
        uint32_t h[kChunks / 4][32];  // the codes as f16, before their slot is free
#pragma unroll
        for (int i = 0; i < kChunks; ++i) int8_to_f16(c[i], h[i / 4] + 8 * (i % 4));
        __syncwarp();  // every lane has its codes
        if (lane == 0) mbar_arrive(empty((int)stage));
        // the K block that had this slot
        if (box >= w_slots) {
          const uint32_t before = (box - w_slots) / kBoxes;
          if (!tc_wait(done(before), parity(before), ab, kStatusWaitEmpty)) break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kChunks / 4; ++i)
          tmem_st_32x32b_x32(dst0 + slot * kTcSlotCols + 32 * i, h[i]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_tmem(leader_bars + (ready(step) - bars_u32));
        stage += kGroups;
        if (stage >= (uint32_t)S) {
          stage -= (uint32_t)S;
          stage_phase ^= 1u;
        }
        slot += kGroups;
        while (slot >= w_slots) slot -= w_slots;
      }
    } else if (kInt8) {
      // x as f16, for the MMAs of the pair
      Ring slots;
      uint32_t it = 0;
      bool aborted = false;
      for (int u = first_tile; u < num_tiles && !aborted; u += tile_step) {
        const int m0 = tc_tile(p, u).m_tile * p.block_t + (int)rank * (p.block_t / 2);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const uint32_t before = it - (uint32_t)p.x_slots;
          if (it >= (uint32_t)p.x_slots &&
              !tc_wait(done(before), parity(before), ab, kStatusWaitEmpty)) {
            aborted = true;
            break;
          }
          if (elect_one()) {
            const uint32_t bar = leader_bars + (ready(it) - bars_u32);
            const uint32_t dst = smem_u32(sX) + (uint32_t)slots.stage * x_step;
            if (leader) mbar_arrive_expect_tx(ready(it), 2 * x_step);
#pragma unroll
            for (int i = 0; i < 2 * kBoxes; ++i)  // 64 f16 wide
              tma_load_2d_pair(dst + (uint32_t)i * x_bytes, &xmap, bar,
                               kb * kBoxes * kTcBlockK + 64 * i, m0);
          }
          __syncwarp();
          slots.next(p.x_slots);
        }
      }
    }
  } else if (warp == kTcTmaWarp) {
    // ------------------------------------------------------------------------------ TMA loader
    Ring ring;
    bool aborted = false;
    const int half_t = p.block_t / 2;
    bool skip = (p.debug_flags & 1) != 0;
    for (int u = first_tile; u < num_tiles && !aborted; u += tile_step) {
      const TcTile un = tc_tile(p, u);
      const int n0 = un.n_tile * kTcChannels + (int)rank * 128;
      const int m0 = un.m_tile * p.block_t + (int)rank * half_t;
      constexpr int per = kInt8 ? kBoxes : 1;  // stages of a K block
      for (int i = kb0 * per; i < kb1 * per; ++i) {
        const int s = ring.stage;
        if (!tc_wait(empty(s), ring.phase ^ 1u, ab, kStatusWaitEmpty)) {
          aborted = true;
          break;
        }
        if (!skip && elect_one()) {
          const uint32_t bar = leader_bars + (full(s) - bars_u32);
          const uint32_t w_dst = smem_u32(sW) + (uint32_t)s * kWStage;
          const uint32_t x_dst = smem_u32(sX) + (uint32_t)s * x_step;
          const int k0 = i * (kInt8 ? kTcBlockK : 2 * kTcBlockK);
          if (kInt8) {  // each CTA's converters wait for its own copies
            mbar_arrive_expect_tx(full(s), kTcWBytes);
            tma_load_2d(w_dst, &wmap, full(s), k0, n0);
          } else {
            const bool both = k0 + kTcBlockK < p.K;  // K may end with the first box
            if (leader) mbar_arrive_expect_tx(full(s), (both ? 4u : 2u) * (kTcWBytes + x_bytes));
            tma_load_2d_pair(w_dst, &wmap, bar, k0, n0);
            tma_load_2d_pair(x_dst, &xmap, bar, k0, m0);
            if (both) {
              tma_load_2d_pair(w_dst + kTcWBytes, &wmap, bar, k0 + kTcBlockK, n0);
              tma_load_2d_pair(x_dst + x_bytes, &xmap, bar, k0 + kTcBlockK, m0);
            }
          }
        }
        skip = false;
        __syncwarp();
        ring.next(S);
      }
    }
  } else if (leader) {
    // ------------------------------------------------------------------------------ MMA issuer
    const uint32_t idesc = kInt8 ? make_idesc_f16_f32(kTcChannels, (uint32_t)p.block_t)
                                 : make_idesc_e4m3_f32(kTcChannels, (uint32_t)p.block_t);
    const uint64_t wdesc0 = make_sw128_kmajor_desc(smem_u32(sW));
    const uint64_t xdesc0 = make_sw128_kmajor_desc(smem_u32(sX));
    Ring ring, wslots;  // the stages (e4m3) or x's slots (int8), w's slots
    const int ring_size = kInt8 ? p.x_slots : S;
    uint32_t it = 0;
    Ring acc;
    bool aborted = false;
    for (int u = first_tile; u < num_tiles && !aborted; u += tile_step) {
      if (!tc_wait(acc_empty(acc.stage), acc.phase ^ 1u, ab, kStatusWaitAccEmpty)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc.stage * p.block_t);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int s = ring.stage;
        if (!tc_wait(kInt8 ? ready(it) : full(s), kInt8 ? parity(it) : ring.phase, ab,
                     kStatusWaitFull)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t acc0 = kb > kb0 ? 1u : 0u;
          // codes past K are zeros, and mostly left out
          const int rem = p.K - kb * kBoxes * kTcBlockK;
          const uint64_t xdesc = xdesc0 + (uint64_t)((uint32_t)s * (x_step >> 4));
          const uint32_t half = x_bytes >> 4;  // 64 f16, or the second box of e4m3
          if (kInt8) {
            const uint32_t a0 = slots_base + (uint32_t)(wslots.stage * kTcSlotCols);
            const int next_slot = wslots.stage + 1 == p.w_slots ? 0 : wslots.stage + 1;
            const uint32_t a1 = slots_base + (uint32_t)(next_slot * kTcSlotCols);
            auto issue_box = [&](uint32_t a, uint64_t x, uint32_t acc) {
              mma_f16_pair_tmem_a(d, a, x, idesc, acc);
              mma_f16_pair_tmem_a(d, a + 8, x + 2, idesc, 1u);
              mma_f16_pair_tmem_a(d, a + 16, x + 4, idesc, 1u);
              mma_f16_pair_tmem_a(d, a + 24, x + 6, idesc, 1u);
              x += half;
              mma_f16_pair_tmem_a(d, a + 32, x, idesc, 1u);
              mma_f16_pair_tmem_a(d, a + 40, x + 2, idesc, 1u);
              mma_f16_pair_tmem_a(d, a + 48, x + 4, idesc, 1u);
              mma_f16_pair_tmem_a(d, a + 56, x + 6, idesc, 1u);
            };
            if (rem >= kBoxes * kTcBlockK) {
              issue_box(a0, xdesc, acc0);
              if (kBoxes == 2) issue_box(a1, xdesc + 2 * half, 1u);
            } else {
              for (int j = 0; 16 * j < rem; ++j)  // K = 16 each, four to a half
                mma_f16_pair_tmem_a(d, (j < 8 ? a0 : a1) + 8 * (j & 7),
                                    xdesc + (uint32_t)(j >> 2) * half + 2 * (j & 3), idesc,
                                    j > 0 ? 1u : acc0);
            }
            mma_commit_pair(done(it), pair_mask);
          } else {
            const uint64_t wdesc = wdesc0 + (uint64_t)((uint32_t)s * (kWStage >> 4));
            const uint64_t wdesc1 = wdesc + (kTcWBytes >> 4), xdesc1 = xdesc + half;
            if (rem >= 2 * kTcBlockK) {
              mma_f8f6f4_pair(d, wdesc, xdesc, idesc, acc0);
              mma_f8f6f4_pair(d, wdesc + 2, xdesc + 2, idesc, 1u);
              mma_f8f6f4_pair(d, wdesc + 4, xdesc + 4, idesc, 1u);
              mma_f8f6f4_pair(d, wdesc + 6, xdesc + 6, idesc, 1u);
              mma_f8f6f4_pair(d, wdesc1, xdesc1, idesc, 1u);
              mma_f8f6f4_pair(d, wdesc1 + 2, xdesc1 + 2, idesc, 1u);
              mma_f8f6f4_pair(d, wdesc1 + 4, xdesc1 + 4, idesc, 1u);
              mma_f8f6f4_pair(d, wdesc1 + 6, xdesc1 + 6, idesc, 1u);
            } else {
              for (int j = 0; 32 * j < rem; ++j)
                mma_f8f6f4_pair(d, (j < 4 ? wdesc : wdesc1) + 2 * (j & 3),
                                (j < 4 ? xdesc : xdesc1) + 2 * (j & 3), idesc, j > 0 ? 1u : acc0);
            }
            mma_commit_pair(empty(s), pair_mask);
          }
          if (kb + 1 == kb1) mma_commit_pair(acc_full(acc.stage), pair_mask);
        }
        __syncwarp();
        ring.next(ring_size);
        if (kInt8) {
          wslots.stage += kBoxes;
          if (wslots.stage >= p.w_slots) wslots.stage -= p.w_slots;
          ++it;
        }
      }
      acc.next(2);
    }
    // every MMA of the pair is complete before TMEM is released
    if (elect_one()) mma_commit_pair(drain_bar, (uint16_t)(1u << cluster_rank));
    __syncwarp();
    wait_drain(drain_bar, 0, p.timeout_ns, p.status, kStatusWaitDrain);
  }
  __syncwarp();
  if (*abort_flag) sleep_ns_bounded(kTcAbortSettleNs);
  tc_fence_before();
  if (p.splits > 1) {
    __syncthreads();
    cluster_sync();  // every slice's partial sums are in place
    if (first_tile < num_tiles) tc_join(p, tc_tile(p, first_tile), smem_u32(sW), split, rank);
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may still signal or read its memory
  tc_fence_after();
  if (warp == kTcMmaWarp) tmem_dealloc_pair(tmem_base, kTcTmemCols);
}

// x's int8 codes as f16. A thread turns 8 codes into 16 bytes, so that a warp's stores fill whole
// sectors, and has kExpand such loads on their way: bound by its 3 bytes of traffic a code. The codes
// between K and the pitch's 16 are not read later: the f16 matrix's map ends at K.
constexpr int kExpand = 4;
__global__ void __launch_bounds__(256) linear_expand_kernel(const LinearParams p) {
  pdl_launch_dependents();  // the product's kernel sets itself up meanwhile
  pdl_wait_primary();
  const int per_row = (p.K + 15) / 16 * 2;
  const int row_blocks = (per_row + 256 * kExpand - 1) / (256 * kExpand);
  const long long blocks = (long long)p.M * row_blocks;
  for (long long i = blockIdx.x; i < blocks; i += gridDim.x) {
    const long long m = i / row_blocks;
    const int c0 = (int)(i - m * row_blocks) * 256 * kExpand + (int)threadIdx.x;
    const uint2* from = reinterpret_cast<const uint2*>(p.x + m * p.x_pitch);
    uint4* to = reinterpret_cast<uint4*>(p.xh + m * p.xh_pitch);
    uint2 c[kExpand];
#pragma unroll
    for (int j = 0; j < kExpand; ++j)
      c[j] = c0 + 256 * j < per_row ? __ldg(from + c0 + 256 * j) : make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < kExpand; ++j) {
      if (c0 + 256 * j >= per_row) break;
      uint32_t h[4];
      int8_to_f16(c[j].x, h);
      int8_to_f16(c[j].y, h + 2);
      to[c0 + 256 * j] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

// Boxes of 128 codes of a K block: two, where TMEM has room for two K blocks of w (int8).
static int tc_boxes(bool int8, int t) { return int8 && t > 128 ? 1 : 2; }

void linear_tc_decide(LinearParams& p, int code_type, const TcLimits& lim) {
  const bool int8 = code_type == Q8_INT8;
  p.n_tiles = (p.N + kTcChannels - 1) / kTcChannels;
  // Tokens of a tile and slices of K: the choice whose waves of tiles are estimated to take the
  // fewest cycles. Measured on whole products, at 1.9 GHz: a K block of a tile of t tokens takes 4.7t
  // cycles (int8, 128 codes), 780 + 2.1t and at least 9.4t (int8, 256 codes), or 380 + 2.3t and at
  // least 5.6t (e4m3, 256 codes); the last epilogue about 8 a token; joining slices about 20 a token
  // and 3500 for the cluster's barriers.
  double best = 1e300;
  for (int t = 32; t <= tc_most_tokens(code_type) && t < p.M + 32; t += 32) {
    if (lim.block_t && t != lim.block_t) continue;
    const long long m_tiles = (p.M + t - 1) / t, tiles = m_tiles * p.n_tiles;
    const int boxes = tc_boxes(int8, t);
    const double kb = boxes == 1 ? 4.7 * t
                      : int8     ? std::max(780.0 + 2.1 * t, 9.4 * t)
                                 : std::max(380.0 + 2.3 * t, 5.6 * t);
    const int k_blocks = (p.K + boxes * kTcBlockK - 1) / (boxes * kTcBlockK);
    for (int splits = 1; splits <= kTcMaxSplits; ++splits) {
      if (lim.splits ? splits != lim.splits : splits > 1 && k_blocks < 2 * splits) continue;
      if (splits > k_blocks || (splits > 1 && tiles > lim.clusters[splits - 1])) continue;
      const long long held = std::max(1, lim.clusters[splits - 1]);
      const long long waves = (tiles + held - 1) / held;
      const double cost = (double)waves * ((k_blocks + splits - 1) / splits) * kb +
                          (splits > 1 ? 20.0 * t + 3500.0 : 8.0 * t);
      if (cost < best) {
        best = cost;
        p.block_t = t;
        p.m_tiles = (int)m_tiles;
        p.k_blocks = k_blocks;
        p.boxes = boxes;
        p.splits = splits;
      }
    }
  }
  if (!p.block_t) return;  // the limits leave none
  const int x_bytes = (int)tc_x_bytes(p.block_t);
  p.w_slots = p.x_slots = 0;
  if (int8) {
    p.w_slots = std::min(8, (kTcTmemCols - 2 * p.block_t) / kTcSlotCols);
    // w gets as many stages for each converter group as leave x five K blocks, x the rest
    const int x_step = p.boxes * 2 * x_bytes;
    const int groups = p.boxes == 1 ? kTcGroups<1> : kTcGroups<2>;
    p.stages = (kTcSmemBudget - 5 * x_step) / kTcWBytes / groups * groups;
    p.stages = std::max(groups, std::min(kTcMaxStages, p.stages));
    p.x_slots = std::min(kTcDepth, (kTcSmemBudget - p.stages * kTcWBytes) / x_step);
  } else {
    p.stages = std::min(kTcMaxStages, kTcSmemBudget / (2 * (kTcWBytes + x_bytes)));
  }
}

size_t linear_tc_smem_bytes(const LinearParams& p, int code_type) {
  const size_t x = tc_x_bytes(p.block_t);
  const size_t tiles = code_type == Q8_INT8 ? p.stages * kTcWBytes + p.x_slots * p.boxes * 2 * x
                                            : p.stages * 2 * (kTcWBytes + x);
  return 1024 + tc_head_bytes(p.block_t) + tiles;
}

constexpr int kTcMostSmem = 227 * 1024;  // all that a CTA may have
// tiles of more than 192 tokens have stages of 60 and 64 KB, and so leave room for more scales
static_assert(1024 + 18 * 1024 + kTcSmemBudget <= kTcMostSmem &&
              kTcBarBytes + kTcStaging + 2 * 192 * 4 <= 18 * 1024);

cudaError_t linear_tc_setup() {
  cudaError_t e = cudaSuccess;
  const void* kernels[] = {(const void*)linear_q8_tc_kernel<true, 1>,
                           (const void*)linear_q8_tc_kernel<true, 2>,
                           (const void*)linear_q8_tc_kernel<false, 2>};
  for (const void* k : kernels)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMostSmem);
  return e;
}

// Clusters of 2, 4, 6 and 8 CTAs that the current device holds at once.
cudaError_t linear_tc_max_clusters(int (&clusters)[kTcMaxSplits]) {
  for (int i = 0; i < kTcMaxSplits; ++i) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2 * (i + 1);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * (i + 1), 1, 1);
    cfg.blockDim = dim3(kTcThreads<true>, 1, 1);
    cfg.dynamicSmemBytes = kTcMostSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaOccupancyMaxActiveClusters(&clusters[i], linear_q8_tc_kernel<true, 1>, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename Kernel, typename... Args>
static cudaError_t launch_pdl(Kernel kernel, int grid, int block, int cluster, size_t smem,
                              cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_linear_expand(const LinearParams& p, cudaStream_t stream) {
  const long long per_row = (p.K + 15) / 16 * 2;
  const long long blocks = p.M * ((per_row + 256 * kExpand - 1) / (256 * kExpand));
  const int grid = (int)std::min<long long>(blocks, 152 * 8);  // eight blocks an SM of this device
  return launch_pdl(linear_expand_kernel, grid, 256, 1, 0, stream, p);
}

cudaError_t launch_linear_tc(const LinearParams& p, int code_type, const CUtensorMap& wmap,
                             const CUtensorMap& xmap, const CUtensorMap& ymap, const TcLimits& lim,
                             cudaStream_t stream) {
  const long long tiles = (long long)p.m_tiles * p.n_tiles;
  const int cluster = 2 * p.splits;
  const int grid = cluster * (int)std::min<long long>(tiles, std::max(1, lim.clusters[p.splits - 1]));
  const size_t smem = linear_tc_smem_bytes(p, code_type);
  auto launch = [&](auto kernel, int threads) {
    return launch_pdl(kernel, grid, threads, cluster, smem, stream, wmap, xmap, ymap, p);
  };
  if (code_type == Q8_E4M3) return launch(linear_q8_tc_kernel<false, 2>, kTcThreads<false>);
  return p.boxes == 1 ? launch(linear_q8_tc_kernel<true, 1>, kTcThreads<true>)
                      : launch(linear_q8_tc_kernel<true, 2>, kTcThreads<true>);
}

}  // namespace c3d
