// q8_linear_tc.cu -- products of 8-bit codes on the tensor cores (tcgen05, CTA pairs):
// y[m][n] = scale_x[m] * scale_w[n] * sum_k x[m][k] * w[n][k] + bias[n].
//
// The channels are the rows of the MMA (M = 256 over the pair, 128 a CTA) and the tokens its columns
// (N = block_t, 32 to 256), so that a batch of any size fills whole rows: the accumulator has a
// channel in each TMEM lane and a token in each column, and a warp's stores of one token cover 32
// consecutive channels of y.
//
// e4m3: both operands go from global memory to shared memory by TMA and into kind::f8f6f4.
//
// int8: sm_103a has no fast integer pipe, but an int8 code is exact in f16 (an 11-bit significand),
// a product of two is an integer of at most 2^14, and the fp32 accumulator holds their sums exactly
// up to 2^24. So the product runs as kind::f16, at the f16 rate, on codes turned into f16:
//   - x, which every channel tile reads again, is expanded to f16 once by a small kernel before
//     (3 bytes of traffic a code);
//   - w stays 8 bits wide all the way to shared memory. Converter warps read 64 codes of a row each
//     thread, turn them into f16 (a byte under the exponent of 1024, minus 1152 with the sign bit
//     flipped: a permute and a subtraction for each two codes) and write them to TMEM, from where
//     the MMA takes its A operand. Shared memory then carries the codes once in and once out, and no
//     f16 copy of w: 96 bytes a cycle at 256 tokens in place of 192, of the 128 that it moves. One
//     such step is a chain of about 800 cycles (wait, load, convert, store, publish), so four
//     groups of four warps take it by turns: two halves of a stage, every other stage.
//
// Few tiles: a tile is split along K over the pairs of one cluster (4 or 8 CTAs). Each CTA leaves its
// partial sums in its own shared memory and adds up its share of the tokens from all of them over
// distributed shared memory, in the order of the slices: nothing passes through global memory, and
// a result does not depend on which slice is ready first.
//
// Roles of a CTA: warps 0-3 epilogue, then 16 converters (int8), TMA and MMA (the leader CTA's).
// Every wait is bounded; one that runs out records a status bit and both CTAs wind down.
#include <algorithm>

#include "conv_common.cuh"
#include "q8_common.cuh"

namespace c3d {

template <bool kInt8>
constexpr int kTcTmaWarpOf = kInt8 ? 20 : 4;
template <bool kInt8>
constexpr int kTcThreads = (kTcTmaWarpOf<kInt8> + 2) * 32;
constexpr int kTcWBytes = kTcWBoxRows * kTcBlockK;  // w's codes of one stage: 16 KB a CTA
constexpr int kTcMaxStages = 8;
constexpr int kTcSmemBudget = 200 * 1024;
constexpr int kTcTmemCols = 512;
constexpr int kTcSlotK = 64;                        // codes of w a TMEM slot holds as f16
constexpr int kTcSlotCols = kTcSlotK / 2;           // in 32 columns
constexpr int kTcMaxSlots = 8;
constexpr uint64_t kTcAbortSettleNs = 2ull * 1000 * 1000;  // let copies in flight land on abort

constexpr int kTcBoxBytes = kTcYBoxBytes;           // one staging buffer of the epilogue
constexpr int kTcBars = 3 * kTcMaxStages + 2 * kTcMaxSlots + 5;

// x's bytes of one stage of one CTA (half of the tile's tokens).
__host__ __device__ inline uint32_t tc_x_bytes(int block_t, bool int8) {
  return (uint32_t)(block_t / 2) * kTcBlockK * (int8 ? 2 : 1);
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
  const int share = p.block_t / p.splits;
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
    float4 a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s < p.splits) a[s] = ld_cluster_f4(map_to_cta(at, 2u * s + rank));
#pragma unroll
    for (int s = 1; s < 4; ++s)
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

// The epilogue of one tile in one CTA, for its four epilogue warps: thread = channel. 8 KB of the
// tile at a time (32 tokens of a 16-bit y, 16 of an fp32 one) are staged in shared memory as
// [token][128 channels], in two buffers by turns (`boxes` counts them), and leave by a TMA store
// that y's extents bound, or by stores of whole token rows: for a y off the 16-byte grid, and for
// the last channels of a y whose rows end inside 16 bytes (a TMA store was seen to write the
// whole of the 16 bytes that hold a row's last element). Stored
// straight from the accumulator's lanes, 64 bytes a warp, the 67 MB of y of an e4m3 product of 4096 x
// 8192 x 4096 took 26 of its 105 us. `release` is called once the accumulator has been read.
template <typename Y, typename Release>
__device__ __forceinline__ void tc_epilogue(const LinearParams& p, const CUtensorMap* ymap,
                                            uint32_t trow, const float* scale, ScaleBias sc,
                                            int tokens, long long m0, int n0, uint8_t* staging,
                                            uint32_t& boxes, Release release) {
  constexpr int kRows = kTcBoxBytes / (128 * (int)sizeof(Y));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool by_tma = p.y_tma && (n0 + 128 <= p.N || p.N * (int)sizeof(Y) % 16 == 0);
  for (int c = 0; c < tokens; c += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(trow + c, r);
    tmem_ld_wait();
    if (c + 32 >= tokens) release();
#pragma unroll
    for (int h = 0; h < 32; h += kRows) {
      if (c + h >= tokens) break;
      uint8_t* buf = staging + (boxes & 1u) * kTcBoxBytes;
      if (threadIdx.x == 0) bulk_wait_group_read<1>();  // the store from this buffer, two boxes ago
      named_barrier_sync(1, 128);
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        reinterpret_cast<Y*>(buf)[j * 128 + threadIdx.x] =
            q8_from_float<Y>(sc(__uint_as_float(r[h + j]), scale[c + h + j]));
      if (by_tma) fence_proxy_async_smem();
      named_barrier_sync(1, 128);
      if (threadIdx.x == 0) {
        if (by_tma && n0 < p.N) tma_store_2d(ymap, smem_u32(buf), n0, (int)m0 + c + h);
        bulk_commit_group();  // one a box, empty or not: the wait above counts them
      }
      if (!by_tma) {
        const int rows = min(kRows, tokens - c - h);
        for (int j = warp; j < rows; j += 4) {
          Y* dst = static_cast<Y*>(p.y) + (m0 + c + h + j) * p.y_pitch + n0;
#pragma unroll
          for (int i = lane; i < 128; i += 32)
            if (n0 + i < p.N) dst[i] = reinterpret_cast<const Y*>(buf)[j * 128 + i];
        }
      }
      ++boxes;
    }
  }
}

template <bool kInt8>
__global__ void __launch_bounds__(kTcThreads<kInt8>, 1)
    linear_q8_tc_kernel(const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap,
                        const __grid_constant__ CUtensorMap ymap, const LinearParams p) {
  constexpr int kTcTmaWarp = kTcTmaWarpOf<kInt8>, kTcMmaWarp = kTcTmaWarp + 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
  const int S = p.stages;
  const uint32_t x_bytes = tc_x_bytes(p.block_t, kInt8);
  uint8_t* sW = smem;
  uint8_t* sX = smem + (size_t)S * kTcWBytes;
  uint8_t* sBox = sX + (size_t)S * x_bytes;  // the epilogue's two staging buffers
  float* sScale = reinterpret_cast<float*>(sBox + 2 * kTcBoxBytes);  // [4 warps][kTcMaxTokens]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sScale + 4 * kTcMaxTokens);
  // bars: full[S] (the leader's; e4m3: both operands, int8: x), empty[S], w_full[S] (int8),
  // slot_full[8] (the leader's), slot_empty[8], acc_full[2], acc_empty[2] (the leader's), drain
  const uint32_t bars_u32 = smem_u32(bars);
  auto full = [&](int s) { return bars_u32 + 8u * s; };
  auto empty = [&](int s) { return bars_u32 + 8u * (kTcMaxStages + s); };
  auto w_full = [&](int s) { return bars_u32 + 8u * (2 * kTcMaxStages + s); };
  auto slot_full = [&](int s) { return bars_u32 + 8u * (3 * kTcMaxStages + s); };
  auto slot_empty = [&](int s) { return bars_u32 + 8u * (3 * kTcMaxStages + kTcMaxSlots + s); };
  auto acc_full = [&](int b) { return bars_u32 + 8u * (3 * kTcMaxStages + 2 * kTcMaxSlots + b); };
  auto acc_empty = [&](int b) { return bars_u32 + 8u * (3 * kTcMaxStages + 2 * kTcMaxSlots + 2 + b); };
  const uint32_t drain_bar = bars_u32 + 8u * (kTcBars - 1);
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
      mbar_init(empty(s), 1);
      mbar_init(w_full(s), 1);
    }
    for (int s = 0; s < kTcMaxSlots; ++s) {
      mbar_init(slot_full(s), 2 * 4);  // a converter warp's arrival each, of both CTAs
      mbar_init(slot_empty(s), 1);
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
  const uint32_t slots_base = tmem_base + (uint32_t)(p.acc_bufs * p.acc_stride);
  pdl_wait_primary();
  pdl_launch_dependents();
  const AbortState ab{abort_flag, p.status, p.timeout_ns};

  if (warp < 4) {
    // ------------------------------------------------------------------------------ epilogue
    float* scale = sScale + warp * kTcMaxTokens;
    int buf = 0;
    uint32_t phase = 0, boxes = 0;
    for (int u = first_tile; u < num_tiles; u += tile_step) {
      const TcTile un = tc_tile(p, u);
      const long long n = (long long)un.n_tile * kTcChannels + rank * 128 + threadIdx.x;
      const long long m0 = (long long)un.m_tile * p.block_t;
      const int tokens = (int)min((long long)p.block_t, p.M - m0);
      __syncwarp();
      for (int t = lane; t < p.block_t; t += 32) scale[t] = t < tokens ? p.scale_x[m0 + t] : 0.0f;
      ScaleBias sc{0.0f, 0.0f};
      if (n < p.N) {
        sc.w = __ldg(p.scale_w + n);
        if (p.bias) sc.bias = q8_load_value(p.bias, p.bias_type, n);
      }
      __syncwarp();
      // the four warps go on or stop together: they share the staging buffers
      const bool ok = wait_bounded_warp(acc_full(buf), phase, ab, kStatusWaitAccFull);
      if (!named_barrier_and(1, 128, ok)) break;
      tc_fence_after();
      const uint32_t trow = tmem_base + (uint32_t)(buf * p.acc_stride) + ((uint32_t)(warp * 32) << 16);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_tmem(leader_bars + (acc_empty(buf) - bars_u32));
      };
      const int n0 = un.n_tile * kTcChannels + (int)rank * 128;
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
      if (++buf == p.acc_bufs) {
        buf = 0;
        phase ^= 1u;
      }
    }
    if (threadIdx.x == 0) bulk_wait_group_all();  // the stores have read their buffers
  } else if (warp < kTcTmaWarp) {
    // ---------------------------------------------------------------------------- converters
    if (kInt8) {
      const int quad = warp & 3, half = ((warp - 4) >> 2) & 1, turn = (warp - 4) >> 3;
      const int row = quad * 32 + lane;
      const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
      const uint32_t slot_shift = p.a_slots == 8 ? 3 : 2;
      Ring ring;
      uint32_t it = 0;     // K blocks of all tiles so far; this warp takes those of its turn
      int pending = -1;    // the slot whose store is under way
      auto publish = [&]() {
        if (pending < 0) return;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_tmem(leader_bars + (slot_full(pending) - bars_u32));
        pending = -1;
      };
      bool aborted = false;
      for (int u = first_tile; u < num_tiles && !aborted; u += tile_step) {
        for (int kb = kb0; kb < kb1; ++kb, ++it, ring.next(S)) {
          if ((it & 1u) != (uint32_t)turn) continue;
          const uint32_t seq = 2 * it + half;  // halves of stages go through the slots in order
          const int slot = (int)(seq & (uint32_t)(p.a_slots - 1));
          const uint32_t slot_phase = (seq >> slot_shift) & 1u;
          // the store before is published behind this stage's loads, which give it the time to
          // finish, unless those would have to wait
          if (!__all_sync(0xFFFFFFFFu, mbar_test(w_full(ring.stage), ring.phase))) publish();
          if (!wait_bounded_warp(w_full(ring.stage), ring.phase, ab, kStatusWaitFull)) {
            aborted = true;
            break;
          }
          const uint8_t* src = sW + (size_t)ring.stage * kTcWBytes + row * kTcBlockK;
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)  // 16-byte chunk i of this half, where the swizzle put it
            c[i] = *reinterpret_cast<const uint4*>(src + (((4 * half + i) ^ (row & 7)) << 4));
          publish();
          uint32_t h[32];
#pragma unroll
          for (int i = 0; i < 4; ++i) int8_to_f16(c[i], h + 8 * i);
          if (!wait_bounded_warp(slot_empty(slot), slot_phase ^ 1u, ab, kStatusWaitEmpty)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          tmem_st_32x32b_x32(slots_base + lane_base + (uint32_t)(slot * kTcSlotCols), h);
          pending = slot;
        }
      }
      publish();
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
      for (int kb = kb0; kb < kb1; ++kb) {
        const int s = ring.stage;
        if (!wait_bounded_warp(empty(s), ring.phase ^ 1u, ab, kStatusWaitEmpty)) {
          aborted = true;
          break;
        }
        if (!skip && elect_one()) {
          const uint32_t bar = leader_bars + (full(s) - bars_u32);
          const uint32_t w_dst = smem_u32(sW) + (uint32_t)s * kTcWBytes;
          const uint32_t x_dst = smem_u32(sX) + (uint32_t)s * x_bytes;
          const int k0 = kb * kTcBlockK;
          if (kInt8) {
            mbar_arrive_expect_tx(w_full(s), kTcWBytes);
            tma_load_2d(w_dst, &wmap, w_full(s), k0, n0);
            if (leader) mbar_arrive_expect_tx(full(s), 2 * x_bytes);
            tma_load_2d_pair(x_dst, &xmap, bar, k0, m0);
            tma_load_2d_pair(x_dst + x_bytes / 2, &xmap, bar, k0 + kTcBlockK / 2, m0);
          } else {
            if (leader) mbar_arrive_expect_tx(full(s), 2 * (kTcWBytes + x_bytes));
            tma_load_2d_pair(w_dst, &wmap, bar, k0, n0);
            tma_load_2d_pair(x_dst, &xmap, bar, k0, m0);
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
    Ring ring, slots;
    int buf = 0;
    uint32_t phase = 0;
    bool aborted = false;
    for (int u = first_tile; u < num_tiles && !aborted; u += tile_step) {
      const TcTile un = tc_tile(p, u);
      if (!wait_bounded_warp(acc_empty(buf), phase ^ 1u, ab, kStatusWaitAccEmpty)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(buf * p.acc_stride);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int s = ring.stage;
        if (!wait_bounded_warp(full(s), ring.phase, ab, kStatusWaitFull)) {
          aborted = true;
          break;
        }
        const uint32_t acc0 = kb > kb0 ? 1u : 0u;
        const int rem = p.K - kb * kTcBlockK;  // codes past K are zeros, and mostly left out
        const uint64_t xdesc = xdesc0 + (uint64_t)((uint32_t)s * (x_bytes >> 4));
        if (kInt8) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait_bounded_warp(slot_full(slots.stage), slots.phase, ab,
                                         kStatusWaitFull)) {
              aborted = true;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              const uint32_t a = slots_base + (uint32_t)(slots.stage * kTcSlotCols);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (kTcSlotK * half + 16 * j < rem)
                  mma_f16_pair_tmem_a(d, a + 8 * j, xdesc + half * (x_bytes >> 5) + 2 * j, idesc,
                                      half + j > 0 ? 1u : acc0);
              mma_commit_pair(slot_empty(slots.stage), pair_mask);
              if (half == 1) {
                mma_commit_pair(empty(s), pair_mask);
                if (kb + 1 == kb1) mma_commit_pair(acc_full(buf), pair_mask);
              }
            }
            __syncwarp();
            slots.next(p.a_slots);
          }
          if (aborted) break;
        } else {
          tc_fence_after();
          if (elect_one()) {
            const uint64_t wdesc = wdesc0 + (uint64_t)((uint32_t)s * (kTcWBytes >> 4));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (32 * j < rem)
                mma_f8f6f4_pair(d, wdesc + 2 * j, xdesc + 2 * j, idesc, j > 0 ? 1u : acc0);
            mma_commit_pair(empty(s), pair_mask);
            if (kb + 1 == kb1) mma_commit_pair(acc_full(buf), pair_mask);
          }
          __syncwarp();
        }
        ring.next(S);
      }
      if (++buf == p.acc_bufs) {
        buf = 0;
        phase ^= 1u;
      }
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

// x's int8 codes as f16, 16 a thread and step.
__global__ void __launch_bounds__(256) linear_expand_kernel(const LinearParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int per_row = (p.K + 15) / 16;  // the codes past K, inside the pitch, are not read later
  const long long total = (long long)p.M * per_row;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long m = i / per_row;
    const int c = (int)(i - m * per_row);
    uint32_t h[8];
    int8_to_f16(__ldg(reinterpret_cast<const uint4*>(p.x + m * p.x_pitch) + c), h);
    uint4* dst = reinterpret_cast<uint4*>(p.xh + m * p.xh_pitch) + 2 * c;
    dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
    dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

void linear_tc_decide(LinearParams& p, int code_type, const TcLimits& lim) {
  const bool int8 = code_type == Q8_INT8;
  p.n_tiles = (p.N + kTcChannels - 1) / kTcChannels;
  p.k_blocks = (p.K + kTcBlockK - 1) / kTcBlockK;
  // Tokens of a tile and slices of K: the choice whose waves of tiles are estimated to take the
  // fewest cycles. A K block of a 256 x t tile takes 4t cycles of f16 MMAs (2t of e4m3's), and never
  // less than w's 16 KB a CTA take to arrive: the memory's 6.8 TB/s (3570 bytes a cycle) shared by
  // the CTAs at work, up to 40 bytes a cycle each. An epilogue that no second accumulator hides
  // costs about 8 cycles a token, so does a kernel's last one; joining slices about 20 a token and
  // 2500 for the cluster's barriers.
  double best = 1e300;
  for (int t = 32; t <= kTcMaxTokens && t < p.M + 32; t += 32) {
    if (lim.block_t && t != lim.block_t) continue;
    const long long m_tiles = (p.M + t - 1) / t, tiles = m_tiles * p.n_tiles;
    for (int i = 0; i < 3; ++i) {
      const int splits = 1 << i;
      if (lim.splits ? splits != lim.splits : splits > 1 && p.k_blocks < 2 * splits) continue;
      if (splits > p.k_blocks || (splits > 1 && tiles > lim.clusters[i])) continue;
      const long long held = std::max(1, lim.clusters[i]);
      const long long waves = (tiles + held - 1) / held;
      const double ctas = 2.0 * splits * (double)std::min(tiles, held);
      const double arrive = kTcWBytes / std::min(40.0, 3570.0 / ctas);
      const double kb = std::max((int8 ? 4.0 : 2.0) * t, arrive);
      const bool two = !int8 || t <= 192;
      const double unit =
          (double)((p.k_blocks + splits - 1) / splits) * kb + (two ? 0.0 : 8.0 * t);
      const double cost = (double)waves * unit + (splits > 1 ? 20.0 * t + 2500.0 : 8.0 * t);
      if (cost < best) {
        best = cost;
        p.block_t = t;
        p.m_tiles = (int)m_tiles;
        p.splits = splits;
      }
    }
  }
  if (!int8) {
    p.acc_bufs = 2;
    p.acc_stride = kTcMaxTokens;
    p.a_slots = 1;
  } else {
    p.acc_bufs = p.block_t <= 192 ? 2 : 1;
    p.acc_stride = p.block_t <= 128 ? 128 : (p.block_t <= 192 ? 192 : 256);
    p.a_slots = (kTcTmemCols - p.acc_bufs * p.acc_stride) / kTcSlotCols;  // 8 or 4
  }
  const int stage = kTcWBytes + (int)tc_x_bytes(p.block_t, int8);
  p.stages = std::min(kTcMaxStages, kTcSmemBudget / stage);
}

size_t linear_tc_smem_bytes(const LinearParams& p, int code_type) {
  return 1024 + (size_t)p.stages * (kTcWBytes + tc_x_bytes(p.block_t, code_type == Q8_INT8)) +
         2 * kTcBoxBytes + 4 * kTcMaxTokens * sizeof(float) + kTcBars * 8 + 16;
}

constexpr int kTcMostSmem =
    1024 + kTcSmemBudget + 2 * kTcBoxBytes + 4 * kTcMaxTokens * 4 + kTcBars * 8 + 16;

cudaError_t linear_tc_setup() {
  cudaError_t e = cudaFuncSetAttribute(linear_q8_tc_kernel<true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMostSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(linear_q8_tc_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMostSmem);
  return e;
}

// Clusters of 2, 4 and 8 CTAs that the current device holds at once.
cudaError_t linear_tc_max_clusters(int (&clusters)[3]) {
  for (int i = 0; i < 3; ++i) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2u << i;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2u << i, 1, 1);
    cfg.blockDim = dim3(kTcThreads<true>, 1, 1);
    cfg.dynamicSmemBytes = kTcMostSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaOccupancyMaxActiveClusters(&clusters[i], linear_q8_tc_kernel<true>, &cfg);
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
  const long long total = (long long)p.M * ((p.K + 15) / 16);
  const int grid = (int)std::min<long long>((total + 255) / 256, 152 * 8);
  return launch_pdl(linear_expand_kernel, grid, 256, 1, 0, stream, p);
}

cudaError_t launch_linear_tc(const LinearParams& p, int code_type, const CUtensorMap& wmap,
                             const CUtensorMap& xmap, const CUtensorMap& ymap, const TcLimits& lim,
                             cudaStream_t stream) {
  const long long tiles = (long long)p.m_tiles * p.n_tiles;
  const int cluster = 2 * p.splits;
  const int grid = cluster * (int)std::min<long long>(tiles, std::max(1, lim.clusters[p.splits / 2]));
  const size_t smem = linear_tc_smem_bytes(p, code_type);
  if (code_type == Q8_INT8)
    return launch_pdl(linear_q8_tc_kernel<true>, grid, kTcThreads<true>, cluster, smem, stream, wmap, xmap,
                      ymap, p);
  return launch_pdl(linear_q8_tc_kernel<false>, grid, kTcThreads<false>, cluster, smem, stream, wmap, xmap,
                    ymap, p);
}

}  // namespace c3d
