// q8_attn_cache.cu -- attention of each sequence's newest tokens over a paged cache of codes.
//
// Each cached row is read once for every 8 or 16 rows of q (the heads that share it, newest tokens), and nearly always there are no
// more, so the memory is the bound (a key of 4-bit codes and 128 channels is 144 bytes with its value and scales), as long as
// turning codes into operands stays short: at 6.8 TB/s an SM meets 47 such codes a cycle.
//
// Products. m16n8k16 with the keys as rows and up to 8 rows of q (heads of one group, newest tokens) as columns
// (16 with two instructions): S^T = K q^T, then O^T = V^T P^T with V's channels as rows, so that a group of 8 heads
// fills the instruction. What the instruction sums over may come in any order if both operands agree:
//   - a lane's operands of K are the codes that lie next to each other in its part of a key's row, with q
//     arranged to match once a sequence; those of V pairs of keys of neighbouring channels;
//   - the two keys x heads of S^T that a lane holds become its operand of the second product by one transposition
//     of an 8 x 8 block (movmatrix), the softmax in between running in registers.
// Codes as f16, all exact. A 4-bit code masked in place under the exponent of 1024 (from the next four bits: of 64) is
// 1024 + code (64 + code): one LOP3 and one subtraction for two codes. What is subtracted leaves code - 8, and
// lowest + 8 * scale takes the place of the lowest value: sums of codes of both signs stay small and keep their bits (the
// instruction cuts its sum a bit or two below fp32's last). Without the subtraction, as subnormal numbers, the products
// would be cut at 2^-14 of a code: the instruction does not normalise them. An int8 code's byte under the exponent of
// 1024, minus 1152; e4m3 by its conversion.
//
// Softmax. A warp takes 16 or 32 keys at a time and keeps one reference M for each row of q. The weights that meet codes have
// v's scale in them, w = 2^(x + log2 scale_v - M); the sum of the weights alone, of w / scale_v, and that of the lowest values
// of 4-bit rows, of w * (lowest + 8 * scale_v) / scale_v, are fp32. For bf16 outputs w is cut to f16's bits, for all
// three alike: the cut, by d of w with 0 <= d < 2^-10, weighs a key's code, lowest value and share alike, and what all keys' d
// have in common cancels, so that an output errs by at most 2^-11 of sum p |v - o|, a fourth of its rounding. (Below 2^-14 f16
// has fewer bits: the code's part of such a weight errs by 2^-31 of the largest w, where that of the lowest value, which
// may be large beside a small scale, does not.) An f16 output shows that much (3.3e-4 instead of 2.1e-4 of the norm, 131072
// keys of int8), so there the rest of w is a second part and product: 64 sequences of up to 8192 keys
// take 102.8 us instead of 101.4 (int8), 124 instead of 119 (e4m3), 89.6 instead of 83.5 (4 bits).
// M moves only when a w would pass 2^15 (a vote; maxima over the warp are taken then only), so w keeps its bits
// relative to the largest one whatever v's scales are.
//
// Flat rows. A row of equal values (zeros, or any constant in 4 bits) has codes of 0 and the scale 1, whatever the size of the rows
// beside it. With that scale in its w it would push the others' w out of f16's bits (a key of zeros with 99% of the weight beside
// 32768 with scales of 0.006: 10% off), and lowest + 8 would cut the lowest value off. Any scale stands for codes of 0,
// so where a scale is 1 and the codes are 0 the warp puts another one in its place in the copy: 0 for k, for v 2^-64 or an eighth
// of the lowest value. A vote a step (of all keys, so that a row's results do not depend on its neighbours), and what it calls,
// not inlined, take 131072 int8 keys from 54.9 to 56.0 us (inlined: 57.2), 64 x ..8192 of 4 bits from 81.7 to 82.5, 8 x 131072 of
// them from 255 to 263.
//
// Copies. Every warp has a ring of its own, filled by bulk copies of 16 rows of codes and their scales (pages
// are multiples of 16 tokens: a copy never leaves its page), so no barrier but its own holds it up.
//
// Split. All groups of 64 or 128 keys of all sequences and key heads are cut into equal runs, one a block, on the device, from
// the lengths there (a captured graph keeps its grid for every length). A block's warps join in shared memory;
// where a sequence's head is shared by several blocks each leaves sums in the plan's workspace and a second kernel, that is
// waiting already, joins them in the blocks' order: results do not depend on which is ready first.
//
// 64 sequences of up to 8192 keys, 8 heads of 128, 32 of q, 4-bit codes: 82 us, 3.8 TB/s, by instructions (0.6 a cycle at 4
// warps a scheduler, 128 registers a thread); one of 131072 int8 keys 56.0 us, 4.9 TB/s. 5 or 8 newest tokens of those sequences,
// 20 or 32 rows of q a key head, read and convert the cache twice: 260 and 264 us.
#include <algorithm>
#include <type_traits>

#include "conv_common.cuh"
#include "q8_attn_internal.h"
#include "q8_common.cuh"

namespace c3d {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16;                    // keys of an instruction
constexpr int kHeadKeys = 256;               // what a head costs beside its keys, in keys
constexpr int kLeastShare = 128;             // of a block, where there is too little for all
constexpr float kLowest = -3.4028235e38f;    // M before the first key
constexpr float kLeastScale = 0x1p-80f;      // of v: a smaller one counts as this
constexpr float kFlatScale = 0x1p-64f;       // of a flat row of v (or more): w keeps it as long as other scales are below 2^57
// The largest w is 2^kHigh when M is set and 2^(kHigh + kGrowth), which f16 holds, before it is set again: so far up that those
// next to 0 keep their bits.
constexpr float kHigh = 7.0f, kGrowth = 8.0f;

template <int CODE>
constexpr int kScaleBytes = CODE == Q8_INT4 ? 8 : 4;
template <int CODE, int D>
constexpr int kRowBytes = CODE == Q8_INT4 ? D / 2 : D;
// Tiles of a step. Two of 4-bit codes take their turns at the waits, votes and copies together, where registers allow.
template <int CODE, int D, int NB>
constexpr int kStepTiles = CODE == Q8_INT4 && NB == 1 && D <= 128 ? 2 : 1;
template <int CODE, int D, int NB>
constexpr int kStepKeys = kTile * kStepTiles<CODE, D, NB>;
template <int CODE, int D, int NB>
constexpr int kGroup = kStepKeys<CODE, D, NB> * kWarps;  // keys of the smallest share
template <int CODE, int D>
constexpr int kTileBytes = 2 * kTile * (kRowBytes<CODE, D> + kScaleBytes<CODE>);
// Stages of a warp's ring: what kBlocksPerSm blocks have room for.
template <int CODE, int D, int NB>
constexpr int kStages = CODE == Q8_INT4 && D < 256 ? 4 / kStepTiles<CODE, D, NB> : D == 256 && CODE != Q8_INT4 ? 2 : 3;
// Channels of a row of the sums in shared memory: 4 more, so that the lanes of a store meet all banks.
template <int D>
constexpr int kSumPitch = D + 4;
template <int CODE, int D, int NB>
constexpr int kRingBytes = kWarps * kStages<CODE, D, NB> * kStepTiles<CODE, D, NB> * kTileBytes<CODE, D>;
template <int D, int NB>
constexpr int kBlocksPerSm = D * NB <= 128 ? 4 : D * NB == 256 ? 3 : 2;

// What a block leaves of a share: for each row the reference, the sum of weights and the channels' sums.
__host__ __device__ constexpr size_t part_floats(int rows, int dim) { return (size_t)rows * (dim + 2); }
// A sequence's head (with some rows of q) that blocks first to last share. There is one of these for each head, left by
// the block that begins it, or, where there are more heads than blocks, for each block (which leaves one head unfinished
// at most).
struct SharedHead {
  int first, last;  // last -1: none
  int seq, head, row0;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x without the bits that f16 has no room for.
__device__ __forceinline__ float f16_bits(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u); }
__device__ __forceinline__ float reciprocal_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += a * b, or d = a * b for a first product.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        bool first = false) {
  if (first)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

// Of the eight 4-bit codes of a word the ones from bits 0 and 16 (kOdd: 4 and 20) on, minus 8, as a pair of f16. The
// masking is one LOP3: written as an AND and an OR of constants it became two.
template <bool kOdd>
__device__ __forceinline__ uint32_t int4_signed(uint32_t w) {
  uint32_t u;
  if constexpr (kOdd)
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w), "n"(0x00F000F0), "r"(0x54005400));
  else
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w), "n"(0x000F000F), "r"(0x64006400));
  const float over = kOdd ? 72.0f : 1032.0f;
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __floats2half2_rn(over, over));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// WORDS consecutive words of shared memory.
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

// The channel behind code n of word w of lane t4's part of a key's row.
template <int CODE, int D>
__device__ __forceinline__ int key_channel(int t4, int w, int n) {
  if constexpr (CODE == Q8_INT4)
    return (w / 4) * 128 + t4 * (D < 128 ? D / 4 : 32) + (w % 4) * 8 + n;
  else
    return (w / 4) * 64 + t4 * 16 + (w % 4) * 4 + n;
}

// Lane t4's part of a key's row.
template <int CODE, int D>
__device__ __forceinline__ void load_key(const uint8_t* row, int t4, uint32_t* w) {
  constexpr int kWords = kRowBytes<CODE, D> / 16;
  if constexpr (kWords < 4) {
    load_words<kWords>(row + t4 * kWords * 4, w);
  } else {
#pragma unroll
    for (int j = 0; j < kWords / 4; ++j) load_words<4>(row + j * 64 + t4 * 16, w + 4 * j);
  }
}

// Whether all codes of a row are 0, asked by a whole warp, of a row by each four lanes.
template <int CODE, int D>
__device__ __forceinline__ bool no_codes(const uint8_t* row, int t4) {
  constexpr int kWords = kRowBytes<CODE, D> / 16;
  uint32_t w[kWords], any = 0;
  load_key<CODE, D>(row, t4, w);
#pragma unroll
  for (int i = 0; i < kWords; ++i) any |= w[i];
  any |= __shfl_xor_sync(0xFFFFFFFFu, any, 1);
  any |= __shfl_xor_sync(0xFFFFFFFFu, any, 2);
  return any == 0;
}

// Gives the flat rows of a step, whose scale is 1, the scales that they count with here. Those of v in 4 bits get codes of 8
// too, which meet their weight as 0, and the lowest value that 8 scales take back to theirs.
template <int CODE, int D, int TILES>
__device__ __noinline__ void find_flat_rows(uint8_t* stage, int g, int t4) {
  constexpr uint32_t kCodes = kTile * kRowBytes<CODE, D>, kScales = kTile * kScaleBytes<CODE>;
  constexpr int kWords = kRowBytes<CODE, D> / 16;
#pragma unroll 1
  for (int i = 0; i < 2 * TILES; ++i) {
    uint8_t* tile = stage + i / 2 * kTileBytes<CODE, D>;
    const int key = g + i % 2 * 8;
    float* k_scale = reinterpret_cast<float*>(tile + 2 * kCodes + key * kScaleBytes<CODE>);
    float* v_scale = k_scale + kScales / 4;
    uint8_t* v_row = tile + kCodes + key * kRowBytes<CODE, D>;
    const bool flat_v = no_codes<CODE, D>(v_row, t4) && *v_scale == 1.0f;
    if constexpr (CODE == Q8_INT4) {
      const bool flat_k = no_codes<CODE, D>(tile + key * kRowBytes<CODE, D>, t4) && *k_scale == 1.0f;
      __syncwarp();
      if (flat_k && t4 == 0) *k_scale = 0.0f;
      if (flat_v) {
        // (the order in which load_key takes words is of no account here)
#pragma unroll
        for (int w = 0; w < kWords; ++w) reinterpret_cast<uint32_t*>(v_row)[4 * w + t4] = 0x88888888u;
        if (t4 == 0) {
          const float lowest = v_scale[1], scale = fmaxf(fabsf(lowest) * 0.125f, kFlatScale);
          *reinterpret_cast<float2*>(v_scale) = make_float2(scale, fmaf(-8.0f, scale, lowest));
        }
      }
    } else {
      __syncwarp();
      if (flat_v && t4 == 0) *v_scale = kFlatScale;
    }
  }
  fence_proxy_async_smem();  // before the stage's next copies
  __syncwarp();
}

struct Found {
  int seq;
  long long before;  // groups of the sequences before it
};

// Quotients of sizes that nearly always fit 32 bits (64-bit ones take some hundred cycles).
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
// All units in `blocks` runs, the first `extra` of them one longer: where a block's begins, and which block has a unit.
struct Runs {
  long long each;
  int extra;
  __device__ __forceinline__ Runs(long long total, int blocks)
      : each(divide(total, blocks)), extra((int)(total - each * blocks)) {}
  __device__ __forceinline__ long long begin(int block) const { return block * each + min(block, extra); }
  __device__ __forceinline__ int block_of(long long unit) const {
    const long long longer = extra * (each + 1);
    return (int)(unit < longer ? divide(unit, each + 1) : extra + divide(unit - longer, each));
  }
};

// Groups that a sequence counts for each head: those of its keys and, before them, what a head costs whatever its length,
// which is about as much as kHeadKeys keys (otherwise the block that gets the shortest sequences is the last one to end).
// A bad length counts as no keys.
template <int GROUP>
constexpr int kHeadGroups = kHeadKeys / GROUP;
template <int GROUP>
constexpr int kLeastGroups = kLeastShare / GROUP;
template <int GROUP>
__device__ __forceinline__ int groups_of(const CacheAttnParams& p, int b) {
  const int n = p.lengths[b];
  const bool bad = n < 0 || n > (long long)p.table_width * p.cache.page_size;
  return kHeadGroups<GROUP> + (bad || n <= 0 ? 0 : (int)(((unsigned)n + GROUP - 1) / GROUP));
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <typename T, int CODE, int D, int NB>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<D, NB>)
    cache_attn_kernel(const CacheAttnParams p, float* parts, SharedHead* shared_heads) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[kWarps * kStages<CODE, D, NB>];
  __shared__ float stat[2][kWarps][NB * 8];
  __shared__ __align__(8) float sums[NB * 8 * kSumPitch<D>];
  __shared__ long long scan[kWarps];
  __shared__ Found found;
  __shared__ int abort_flag, bad_input[2];  // the flag of this round and of the next

  constexpr int kRows = NB * 8, kS = kStages<CODE, D, NB>, kBlocks = D / 16, kTiles = kStepTiles<CODE, D, NB>;
  constexpr int kStep = kStepKeys<CODE, D, NB>, kOneTile = kTileBytes<CODE, D>, kStageBytes = kTiles * kOneTile;
  constexpr int kKeyWords = kRowBytes<CODE, D> / 16, kValueWords = kRowBytes<CODE, D> / 32;
  constexpr int kShare = kGroup<CODE, D, NB>;
  constexpr bool kTwoParts = std::is_same_v<T, __half>;  // of a weight: an f16 output shows what one leaves out
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t4 = lane % 4;
  const Cache& c = p.cache;
  const int group = p.q_heads / c.kv_heads, rows_all = p.tokens * group;
  const int row_blocks = (rows_all + kRows - 1) / kRows;
  const long long heads = (long long)c.kv_heads * row_blocks;

  uint8_t* my_ring = ring + warp * kS * kStageBytes;
  const uint32_t ring_at = smem_u32(my_ring), bar_at = smem_u32(bars) + warp * kS * 8;
  if (threadIdx.x == 0) abort_flag = 0, bad_input[0] = 0;
  if (lane < kS) mbar_init(bar_at + 8 * lane, 1);
  fence_mbar_init();
  __syncthreads();  // the flags and barriers are set before any warp uses them; beside the wait for the kernel before

  pdl_wait_primary();
  // ---- this block's share
  long long total = 0, at, until, before = 0;
  int blocks, seq = 0;
  auto cut_runs = [&](long long groups_of_all) {
    total = groups_of_all * heads;
    // Heads that have less than four shares stay whole, for there is then nothing to join (one sequence of 8 heads: 128
    // keys 9.7 us in 24 blocks, 8.3 in 8; 512 keys 9.7 in 48).
    const long long enough = divide(total, kLeastGroups<kShare>), whole = p.seqs * heads;
    blocks = (int)min((long long)gridDim.x, enough < 4 * whole ? whole : enough);
    const Runs runs(total, blocks);
    at = runs.begin(blockIdx.x);
    until = runs.begin(blockIdx.x + 1);
  };
  if (p.seqs <= 32) {  // each warp by itself: without barriers and a second look (2 us of a short call)
    const int mine = lane < p.seqs ? groups_of<kShare>(p, lane) : 0;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    cut_runs(__shfl_sync(0xFFFFFFFFu, sum, 31));
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, sum > divide(at, heads));
    seq = hit ? __ffs(hit) - 1 : 0;
    before = __shfl_sync(0xFFFFFFFFu, sum - mine, seq);
  } else {
    for (int b = threadIdx.x; b < p.seqs; b += kThreads) total += groups_of<kShare>(p, b);
    total = warp_sum(total);
    if (lane == 0) scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += scan[w];
    __syncthreads();
    cut_runs(total);
    const long long want = divide(at, heads);
    if ((int)blockIdx.x < blocks) {
      for (int b0 = 0; b0 < p.seqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int mine = b < p.seqs ? groups_of<kShare>(p, b) : 0;
        long long sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += v;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        long long end = before;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) sum += scan[w];
          end += scan[w];
        }
        if (before + sum > want && before + sum - mine <= want) found = Found{b, before + sum - mine};
        __syncthreads();
        if (end > want) break;
        before = end;
      }
      seq = found.seq;
      before = found.before;
    }
  }
  pdl_launch_dependents();
  const bool by_head = p.seqs * heads <= (long long)gridDim.x;
  if (threadIdx.x == 0 && !by_head) shared_heads[blockIdx.x].last = -1;
  if ((int)blockIdx.x >= blocks) return;

  const AbortState ab{&abort_flag, p.status, p.timeout_ns};
  const float scale_log2 = p.scale * 1.44269504088896f;
  uint32_t issued = 0, used = 0;  // this warp's copies so far
  // A tile is four copies: the codes of k and of v and their scales, by the lanes 0 to 3 (4 to 7: the second tile's).
  constexpr uint32_t kCodes = kTile * kRowBytes<CODE, D>, kScales = kTile * kScaleBytes<CODE>;
  const uint32_t copy_bytes = t4 < 2 ? kCodes : kScales;
  const uint32_t copy_dst = ring_at + g * kOneTile + (t4 < 2 ? t4 * kCodes : 2 * kCodes + (t4 - 2) * kScales);
  const uint8_t* copy_src = t4 == 0   ? c.k_codes
                            : t4 == 1 ? c.v_codes
                                      : reinterpret_cast<const uint8_t*>(t4 == 2 ? c.k_scale : c.v_scale);

  // ---- the heads of sequences that it covers, or parts of them: of the one that it is at
  long long head_index;
  int groups, first_group, take, head, row0, keys, tiles, first, count;
  bool bad;
  long long places;  // where 32 of this warp's tiles lie, a lane each, in tiles of the whole cache; -1 behind the end
  int ahead;         // steps whose copies are issued
  // This lane's channels of q's rows, 16 bytes at a time.
  constexpr int kCodesOf = CODE == Q8_INT4 ? 8 : 4, kPer = 8 / kCodesOf;  // codes of a word, words of 16 bytes
  const unsigned page_tiles = (unsigned)c.page_size / kTile;
  auto places_from = [&](int i) {
    const int tile = (first + (i + lane / kTiles) * kWarps) * kTiles + lane % kTiles;
    if (i + lane / kTiles >= count || tile >= tiles) return -1LL;
    const unsigned entry = (unsigned)tile / page_tiles;
    unsigned page = (unsigned)p.table[seq * p.table_pitch + entry];
    if (page >= c.slots / (unsigned)c.page_size) {
      bad = true;
      page = 0;  // some page of the cache; what is read there is dropped
    }
    return ((long long)page * c.kv_heads + head) * page_tiles + ((unsigned)tile - entry * page_tiles);
  };
  auto issue = [&](int i) {
    const long long place = __shfl_sync(0xFFFFFFFFu, places, i * kTiles % 32 + g % kTiles);
    const uint32_t stage = issued % kS, bar = bar_at + 8 * stage;
    const bool mine = lane < 4 * kTiles && place >= 0;
    const bool all = kTiles == 1 || (__ballot_sync(0xFFFFFFFFu, mine) >> 4) != 0;
    if (lane == 0) mbar_arrive_expect_tx(bar, all ? kStageBytes : kOneTile);
    __syncwarp();
    const bool skip = (p.debug_flags & 1) && seq == 0 && head == 0 && row0 == 0 && first + i == 0;
    if (mine && !skip) bulk_load(copy_dst + stage * kStageBytes, copy_src + place * copy_bytes, copy_bytes, bar);
    ++issued;
  };
  auto start = [&] {
    groups = groups_of<kShare>(p, seq);
    head_index = divide(at - before * heads, groups);
    first_group = (int)((at - before * heads) - head_index * groups);
    take = (int)min((long long)groups - first_group, until - at);
    head = row_blocks == 1 ? (int)head_index : (int)head_index / row_blocks;
    row0 = ((int)head_index - head * row_blocks) * kRows;
    const int length = p.lengths[seq];
    bad = length < 0 || length > (long long)p.table_width * c.page_size;
    keys = bad ? 0 : length;
    tiles = (int)(((unsigned)keys + kTile - 1) / kTile);
    const int steps = (tiles + kTiles - 1) / kTiles;
    const int from = max(0, first_group - kHeadGroups<kShare>), to = max(0, first_group + take - kHeadGroups<kShare>);
    first = from * kWarps + warp;  // of this warp's steps, which are kWarps apart
    const int end = min(steps, to * kWarps);
    count = first < end ? (end - first + kWarps - 1) / kWarps : 0;
    places = places_from(0);
    ahead = min(count, kS);
    for (int i = 0; i < ahead; ++i) issue(i);
  };
  start();
  for (int round = 0;; round ^= 1) {
    // ---- q's operands: row g of the columns, in the order of the codes
    uint4 q_raw[NB][kKeyWords / kPer];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int r = row0 + 8 * nb + g, t = r / group;
      const T* q = static_cast<const T*>(p.q.p) + ((long long)seq * p.tokens + t) * p.q.pitch +
                   (long long)(head * group + r - t * group) * p.q.head_pitch;
#pragma unroll
      for (int w = 0; w < kKeyWords / kPer; ++w)
        q_raw[nb][w] = r < rows_all ? *reinterpret_cast<const uint4*>(q + key_channel<CODE, D>(t4, w * kPer, 0))
                                    : make_uint4(0, 0, 0, 0);
    }
    uint32_t q_frag[NB][kBlocks][2];
    float factor[NB][2], q_sum[NB][2];  // of the columns 2 t4 and the next
    int limit[NB][2];                   // keys that they see
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float amax = 0.0f;
#pragma unroll
      for (int w = 0; w < kKeyWords / kPer; ++w)
#pragma unroll
        for (int n = 0; n < 8; ++n) amax = fmaxf(amax, fabsf(q8_to_float(reinterpret_cast<const T*>(&q_raw[nb][w])[n])));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // the largest between 2^8 and 2^9, by a power of two (in two parts, each of which fp32 holds)
      const int up = amax > 0.0f && amax < 3.4e38f ? 135 - (int)(__float_as_uint(amax) >> 23) : 0;
      const float up0 = __uint_as_float((127 + up / 2) << 23), up1 = __uint_as_float((127 + up - up / 2) << 23);
      const float down0 = __uint_as_float((127 - up / 2) << 23), down1 = __uint_as_float((127 - up + up / 2) << 23);
      auto value = [&](int w, int n) {
        return q8_to_float(reinterpret_cast<const T*>(&q_raw[nb][w / kPer])[w % kPer * kCodesOf + n]) * up0 * up1;
      };
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kKeyWords; ++w) {
        if constexpr (CODE == Q8_INT4) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // as int4_signed leaves them: the codes 2i and 2i + 4, then 2i + 1 and 2i + 5
            const __half2 even = __floats2half2_rn(value(w, 2 * i), value(w, 2 * i + 4));
            const __half2 odd = __floats2half2_rn(value(w, 2 * i + 1), value(w, 2 * i + 5));
            sum += __low2float(even) + __high2float(even) + __low2float(odd) + __high2float(odd);
            q_frag[nb][2 * w + i][0] = *reinterpret_cast<const uint32_t*>(&even);
            q_frag[nb][2 * w + i][1] = *reinterpret_cast<const uint32_t*>(&odd);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 v = __floats2half2_rn(value(w, 2 * i), value(w, 2 * i + 1));
            q_frag[nb][w][i] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
      }
      const float back = scale_log2 * down0 * down1;
      float s = 0.0f;
      if constexpr (CODE == Q8_INT4) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
        s = back * sum;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        factor[nb][j] = __shfl_sync(0xFFFFFFFFu, back, (2 * t4 + j) * 4);
        q_sum[nb][j] = __shfl_sync(0xFFFFFFFFu, s, (2 * t4 + j) * 4);
        const int rj = row0 + 8 * nb + 2 * t4 + j;
        limit[nb][j] = rj < rows_all ? keys - p.tokens + 1 + rj / group : 0;
      }
    }

    float o[NB][kBlocks][4] = {};
    float top[NB][2], most[NB][2], weight[NB][2], low_sum[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) top[nb][j] = most[nb][j] = kLowest, weight[nb][j] = low_sum[nb][j] = 0.0f;

    // One step: the keys from key0 on, in a stage. kMasked: some row does not see all of them.
    auto step = [&](auto is_masked, uint8_t* stage, int key0) {
      constexpr bool kMasked = decltype(is_masked)::value;
      const float* a_scale = reinterpret_cast<const float*>(stage + lane % kStep / kTile * kOneTile + 2 * kCodes +
                                                            lane % kTile * kScaleBytes<CODE>);
      bool one = a_scale[kScales / 4] == 1.0f;
      if constexpr (CODE == Q8_INT4) one |= a_scale[0] == 1.0f;
      float s[kTiles][NB][4];  // of the keys g and g + 8 of each tile
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        uint32_t a[kKeyWords], b[kKeyWords];
        load_key<CODE, D>(stage + u * kOneTile + g * kRowBytes<CODE, D>, t4, a);
        load_key<CODE, D>(stage + u * kOneTile + (g + 8) * kRowBytes<CODE, D>, t4, b);
        float s2[NB][4];  // every other product: two chains
#pragma unroll
        for (int w = 0; w < kKeyWords; ++w) {
          if constexpr (CODE == Q8_INT4) {
            const uint32_t ah = a[w] >> 8, bh = b[w] >> 8;
            const uint32_t m0[4] = {int4_signed<false>(a[w]), int4_signed<false>(b[w]), int4_signed<true>(a[w]),
                                    int4_signed<true>(b[w])};
            const uint32_t m1[4] = {int4_signed<false>(ah), int4_signed<false>(bh), int4_signed<true>(ah),
                                    int4_signed<true>(bh)};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma_f16(s[u][nb], m0, q_frag[nb][2 * w][0], q_frag[nb][2 * w][1], w == 0);
              mma_f16(s2[nb], m1, q_frag[nb][2 * w + 1][0], q_frag[nb][2 * w + 1][1], w == 0);
            }
          } else {
            uint32_t ha[2], hb[2];
            if constexpr (CODE == Q8_INT8) {
              int8_to_f16(a[w], ha);
              int8_to_f16(b[w], hb);
            } else {
              ha[0] = e4m3_pair(a[w] & 0xFFFFu), ha[1] = e4m3_pair(a[w] >> 16);
              hb[0] = e4m3_pair(b[w] & 0xFFFFu), hb[1] = e4m3_pair(b[w] >> 16);
            }
            const uint32_t m[4] = {ha[0], hb[0], ha[1], hb[1]};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_f16(w % 2 ? s2[nb] : s[u][nb], m, q_frag[nb][w][0], q_frag[nb][w][1], w < 2);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nb][e] += s2[nb][e];
      }
      if (__any_sync(0xFFFFFFFFu, one)) find_flat_rows<CODE, D, kTiles>(stage, g, t4);
      float v_mid[kTiles][2], v_inv[kTiles][2];  // of the keys g and g + 8
      bool grows = false;
#pragma unroll
      for (int u = 0; u < kTiles; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = kTile * u + g + 8 * j;
          const float* k_scale = reinterpret_cast<const float*>(stage + u * kOneTile + 2 * kCodes);
          const float* v_scale = k_scale + kScales / 4;
          float ks, vs, vl = 0.0f;
          [[maybe_unused]] float k_mid = 0.0f;
          if constexpr (CODE == Q8_INT4) {
            const float2 a = reinterpret_cast<const float2*>(k_scale)[g + 8 * j];
            const float2 b = reinterpret_cast<const float2*>(v_scale)[g + 8 * j];
            ks = a.x, k_mid = fmaf(8.0f, a.x, a.y), vs = b.x, vl = fmaf(8.0f, b.x, b.y);
          } else {
            ks = k_scale[g + 8 * j], vs = v_scale[g + 8 * j];
          }
          vs = vs < kLeastScale ? kLeastScale : vs;  // a NaN stays
          if (kMasked && key0 + key >= keys) vs = 1.0f, vl = 0.0f;  // whatever lies there
          const float v_log = log2_fast(vs);
          v_inv[u][j] = reciprocal_fast(vs);
          v_mid[u][j] = vl * v_inv[u][j];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = fmaf(s[u][nb][2 * j + i], ks * factor[nb][i], v_log);
              if constexpr (CODE == Q8_INT4) x = fmaf(k_mid, q_sum[nb][i], x);
              if (kMasked && key0 + key >= limit[nb][i]) x = -INFINITY;
              s[u][nb][2 * j + i] = x;
              grows |= x > most[nb][i];
            }
        }
      if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float m = fmaxf(s[0][nb][j], s[0][nb][2 + j]);
            if constexpr (kTiles == 2) m = fmaxf(m, fmaxf(s[kTiles - 1][nb][j], s[kTiles - 1][nb][2 + j]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, w));
            const bool up = m > most[nb][j];  // only then: a row's results do not depend on its neighbours
            const float keep = up ? exp2_fast(top[nb][j] - (m - kHigh)) : 1.0f;
            // (rounded down: beside a score of 2^26 a step is 8, and w would pass f16's range)
            if (up) top[nb][j] = m - kHigh, most[nb][j] = __fadd_rd(top[nb][j], kHigh + kGrowth);
            weight[nb][j] *= keep;
            low_sum[nb][j] *= keep;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) o[nb][b][j] *= keep, o[nb][b][2 + j] *= keep;
          }
      }
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        uint32_t p_frag[NB][2];
        [[maybe_unused]] uint32_t p_rest[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x0 = s[u][nb][2 * j], x1 = s[u][nb][2 * j + 1];
            float w0 = exp2_fast(x0 - top[nb][0]), w1 = exp2_fast(x1 - top[nb][1]);
            const float cut0 = f16_bits(w0), cut1 = f16_bits(w1);
            const __half2 h = __floats2half2_rn(cut0, cut1);
            p_frag[nb][j] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h));
            if constexpr (kTwoParts) {
              const __half2 rest = __floats2half2_rn(w0 - cut0, w1 - cut1);
              p_rest[nb][j] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&rest));
            } else {
              w0 = cut0, w1 = cut1;
            }
            // a key that a row does not see may be marked NaN
            const bool see0 = !kMasked || x0 != -INFINITY, see1 = !kMasked || x1 != -INFINITY;
            if (see0) weight[nb][0] = fmaf(w0, v_inv[u][j], weight[nb][0]);
            if (see1) weight[nb][1] = fmaf(w1, v_inv[u][j], weight[nb][1]);
            if constexpr (CODE == Q8_INT4) {
              if (see0) low_sum[nb][0] = fmaf(w0, v_mid[u][j], low_sum[nb][0]);
              if (see1) low_sum[nb][1] = fmaf(w1, v_mid[u][j], low_sum[nb][1]);
            }
          }
        // values of the keys 2 t4, the next, and both 8 further on
        const uint8_t* v_codes = stage + u * kOneTile + kCodes;
        uint32_t v[4][kValueWords];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = 2 * t4 + (j & 1) + 8 * (j >> 1);
          load_words<kValueWords>(v_codes + key * kRowBytes<CODE, D> + g * kValueWords * 4, v[j]);
          if (CODE == Q8_E4M3 && kMasked && key0 + kTile * u + key >= keys) {
#pragma unroll
            for (int w = 0; w < kValueWords; ++w) v[j][w] = 0;  // it may be a NaN
          }
        }
#pragma unroll
        for (int w = 0; w < kValueWords; ++w) {
          if constexpr (CODE == Q8_INT4) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // the codes 0 to 3 and 4 to 7
              const uint32_t pick = half ? 0x7632u : 0x5410u;
              uint32_t lo = __byte_perm(v[0][w], v[1][w], pick), hi = __byte_perm(v[2][w], v[3][w], pick);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t m[4] = {int4_signed<false>(lo), int4_signed<true>(lo), int4_signed<false>(hi),
                                       int4_signed<true>(hi)};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  mma_f16(o[nb][4 * w + 2 * half + i], m, p_frag[nb][0], p_frag[nb][1]);
                  if constexpr (kTwoParts) mma_f16(o[nb][4 * w + 2 * half + i], m, p_rest[nb][0], p_rest[nb][1]);
                }
                lo >>= 8, hi >>= 8;
              }
            }
          } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // the codes 0 and 1, 2 and 3
              const uint32_t pick = half ? 0x7362u : 0x5140u;
              const uint32_t lo = __byte_perm(v[0][w], v[1][w], pick), hi = __byte_perm(v[2][w], v[3][w], pick);
              uint32_t hl[2], hh[2];
              if constexpr (CODE == Q8_INT8) {
                int8_to_f16(lo, hl);
                int8_to_f16(hi, hh);
              } else {
                hl[0] = e4m3_pair(lo & 0xFFFFu), hl[1] = e4m3_pair(lo >> 16);
                hh[0] = e4m3_pair(hi & 0xFFFFu), hh[1] = e4m3_pair(hi >> 16);
              }
              const uint32_t m[4] = {hl[0], hl[1], hh[0], hh[1]};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma_f16(o[nb][2 * w + half], m, p_frag[nb][0], p_frag[nb][1]);
                if constexpr (kTwoParts) mma_f16(o[nb][2 * w + half], m, p_rest[nb][0], p_rest[nb][1]);
              }
            }
          }
        }
      }
    };

    bool waited = true;
    for (int i = 0; i < count; ++i) {
      const uint32_t stage = used % kS;
      waited = tc_wait(bar_at + 8 * stage, (used / kS) & 1, ab, kAttnTimeout);
      if (!waited) break;
      const int key0 = (first + i * kWarps) * kStep;
      if (keys - p.tokens + 1 - key0 >= kStep)
        step(std::false_type{}, my_ring + stage * kStageBytes, key0);
      else
        step(std::true_type{}, my_ring + stage * kStageBytes, key0);
      ++used;
      __syncwarp();  // the stage is free
      if (ahead < count) {
        if (ahead * kTiles % 32 == 0) places = places_from(ahead);
        issue(ahead++);
      }
    }
    if (bad || !waited) bad_input[round] = 1;

    // ---- the next one's copies are under way while this one's sums are joined
    const bool whole = take == groups;
    const int part_side = first_group > 0 ? 0 : 1, done_seq = seq, done_head = head, done_row0 = row0;
    const bool begins = first_group == 0;
    const long long done_index = head_index, last_unit = before * heads + (head_index + 1) * groups - 1;
    at += take;
    const bool more = at < until;
    if (more && waited) {
      if (at == (before + groups) * heads) before += groups, ++seq;
      start();
    }

    // ---- the warps' sums, joined
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          weight[nb][j] += __shfl_xor_sync(0xFFFFFFFFu, weight[nb][j], w);
          low_sum[nb][j] += __shfl_xor_sync(0xFFFFFFFFu, low_sum[nb][j], w);
        }
        if (g == 0) stat[0][warp][8 * nb + 2 * t4 + j] = top[nb][j];
      }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {  // one after another: there is room for one warp's beside the rings
      if (w == warp) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = 8 * nb + 2 * t4 + j;
            float m = stat[0][0][r];
#pragma unroll
            for (int v = 1; v < kWarps; ++v) m = fmaxf(m, stat[0][v][r]);
            const float keep = top[nb][j] == m ? 1.0f : exp2_fast(top[nb][j] - m);
            if (g == 0) stat[1][warp][r] = weight[nb][j] * keep;
            const float add = low_sum[nb][j] * keep;
            float* row = sums + r * kSumPitch<D> + 2 * g;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
              float2 v = make_float2(fmaf(o[nb][b][j], keep, add), fmaf(o[nb][b][2 + j], keep, add));
              float2* to = reinterpret_cast<float2*>(row + 16 * b);
              if (w > 0) v.x += to->x, v.y += to->y;
              *to = v;
            }
          }
      }
      __syncthreads();
    }
    float* part = parts + (2 * (long long)blockIdx.x + part_side) * part_floats(kRows, D);
    const float nan = __int_as_float(0x7FFFFFFF);
    if (threadIdx.x == 0) {
      bad_input[round ^ 1] = 0;
      if (bad_input[round] && !abort_flag) atomicOr(p.status, kAttnBadInput);
      if (begins && (by_head || !whole))
        // its last block is the one that holds the head's last group
        shared_heads[by_head ? done_seq * heads + done_index : blockIdx.x] =
            SharedHead{(int)blockIdx.x, whole ? -1 : Runs(total, blocks).block_of(last_unit), done_seq, done_head, done_row0};
    }
    for (int i = threadIdx.x; i < kRows * (D / 2); i += kThreads) {
      const int r = i / (D / 2), pair = i % (D / 2);
      const int lane_of = 2 * pair / (D / 8), block_of = pair % (D / 16);
      const float2 sum = *reinterpret_cast<const float2*>(sums + r * kSumPitch<D> + 16 * block_of + 2 * lane_of);
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l += stat[1][w][r];
      if (bad_input[round]) l = nan;
      const int rr = done_row0 + r;
      if (!whole) {
        *reinterpret_cast<float2*>(part + 2 * kRows + r * D + 2 * pair) = sum;
        if (pair == 0) {
          float m = stat[0][0][r];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) m = fmaxf(m, stat[0][w][r]);
          part[r] = m;
          part[kRows + r] = l;
        }
      } else if (rr < rows_all) {
        const int t = rr / group, h = rr - t * group;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.o.p) +
                                                    ((long long)done_seq * p.tokens + t) * p.o.pitch +
                                                    (long long)(done_head * group + h) * p.o.head_pitch + 2 * pair);
        *out = q8_pack2<T>(make_float2(sum.x * inv, sum.y * inv));
      }
    }
    const bool stop = __syncthreads_or(!waited) || !more;
    if (stop) {
      // On abort: heads that would have begun here are marked whole, so that nothing is joined for them by what an earlier
      // run left; and another warp may have copies of the next one under way.
      if (threadIdx.x == 0 && by_head && more) {
        if (waited && first_group == 0) shared_heads[seq * heads + head_index].last = -1;  // the one started above
        long long unit = before * heads + (head_index + 1) * groups;
        if (!waited) unit = last_unit + 1;  // not started: what `seq` and `groups` still stand for is done
        while (unit < until) {
          if (unit >= (before + groups) * heads) before += groups, groups = groups_of<kShare>(p, ++seq);
          shared_heads[seq * heads + divide(unit - before * heads, groups)].last = -1;
          unit += groups;
        }
      }
      for (; used < issued; ++used) {
        int own = 0;
        tc_wait(bar_at + 8 * (used % kS), (used / kS) & 1, AbortState{&own, p.status, 1000000ull}, kAttnTimeout);
      }
      break;
    }
  }
}

// Joins the sums of heads that several blocks share: gridDim.y blocks for each of them, between whose rows the warps
// are divided. A warp joins its parts as the main kernel does keys, so that they are looked at once.
constexpr int kJoinWarps = 8;
template <typename T, int D, int NB>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(const CacheAttnParams p, const float* parts,
                                                                     const SharedHead* shared_heads) {
  constexpr int kRows = NB * 8, kVec = D / 32, kAtOnce = 4;
  __shared__ float sums[kJoinWarps][D];
  __shared__ float2 stats[kJoinWarps];  // the reference and the sum of the weights
  pdl_wait_primary();
  const SharedHead s = shared_heads[blockIdx.x];
  if (s.last < 0) return;  // whole in its block, or given up
  const int group = p.q_heads / p.cache.kv_heads;
  const int rows = kRows / gridDim.y, at_once = min(rows, kJoinWarps), share = kJoinWarps / at_once;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, mine = warp % share;
  const int n = s.last - s.first + 1;
  for (int r0 = blockIdx.y * rows; r0 < (int)(blockIdx.y + 1) * rows; r0 += at_once) {
    const int r = r0 + warp / share;
    float m = kLowest, l = 0.0f, sum[kVec] = {};
    for (int i0 = mine; i0 < n; i0 += share * kAtOnce) {
      float pm[kAtOnce], pl[kAtOnce], v[kAtOnce][kVec];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int i = i0 + a * share;
        pm[a] = kLowest;
        if (i < n) {
          const float* part = parts + (2 * ((long long)s.first + i) + (i == 0)) * part_floats(kRows, D);
          pm[a] = part[r];
          pl[a] = part[kRows + r];
#pragma unroll
          for (int e = 0; e < kVec; ++e) v[a][e] = part[2 * kRows + r * D + 32 * e + lane];
        }
      }
      float now = m;
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) now = fmaxf(now, pm[a]);
      const float before = now == m ? 1.0f : exp2_fast(m - now);
      m = now;
      l *= before;
#pragma unroll
      for (int e = 0; e < kVec; ++e) sum[e] *= before;
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        if (i0 + a * share >= n) continue;
        const float keep = pm[a] == m ? 1.0f : exp2_fast(pm[a] - m);
        l = fmaf(pl[a], keep, l);
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[e] = fmaf(v[a][e], keep, sum[e]);
      }
    }
    if (share > 1) {
      if (lane == 0) stats[warp] = make_float2(m, l);
#pragma unroll
      for (int e = 0; e < kVec; ++e) sums[warp][32 * e + lane] = sum[e];
      __syncthreads();
      if (mine == 0) {
        float now = m;
        for (int w = 1; w < share; ++w) now = fmaxf(now, stats[warp + w].x);
        const float before = m == now ? 1.0f : exp2_fast(m - now);
        l *= before;
#pragma unroll
        for (int e = 0; e < kVec; ++e) sum[e] *= before;
        for (int w = 1; w < share; ++w) {
          const float2 st = stats[warp + w];
          const float keep = st.x == now ? 1.0f : exp2_fast(st.x - now);
          l = fmaf(st.y, keep, l);
#pragma unroll
          for (int e = 0; e < kVec; ++e) sum[e] = fmaf(sums[warp + w][32 * e + lane], keep, sum[e]);
        }
      }
      __syncthreads();
    }
    const int rr = s.row0 + r;
    if (mine == 0 && rr < p.tokens * group) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int t = rr / group, h = rr - t * group;
      T* out = static_cast<T*>(p.o.p) + ((long long)s.seq * p.tokens + t) * p.o.pitch +
               (long long)(s.head * group + h) * p.o.head_pitch;
#pragma unroll
      for (int e = 0; e < kVec; ++e) out[32 * e + lane] = q8_from_float<T>(sum[e] * inv);
    }
  }
}

// Rows of q that the instructions' columns hold, in eights: 16 where 8 do not hold all of a key head's.
static int cache_attn_eights(int tokens, int q_heads, int kv_heads) {
  return tokens * (q_heads / kv_heads) <= 8 ? 1 : 2;
}

static int cache_attn_blocks(int sms, int dim, int nb) {
  return sms * (dim * nb <= 128 ? 4 : dim * nb == 256 ? 3 : 2);
}

size_t cache_attn_workspace(int sms, int tokens, int q_heads, int kv_heads, int dim) {
  // a run of fewer tokens may use the form with fewer rows, and more blocks
  size_t most = 0;
  for (int nb = 1; nb <= cache_attn_eights(tokens, q_heads, kv_heads); ++nb)
    most = std::max(most, cache_attn_blocks(sms, dim, nb) *
                              (2 * part_floats(8 * nb, dim) * sizeof(float) + sizeof(SharedHead)));
  return most;
}

// One form of the kernels: with p null only what it needs of the device is set up.
template <typename T, int CODE, int D, int NB>
static cudaError_t cache_attn_form(const CacheAttnParams* p, void* workspace, int sms, cudaStream_t stream) {
  constexpr int kSmem = kRingBytes<CODE, D, NB>;
  auto kernel = cache_attn_kernel<T, CODE, D, NB>;
  if (!p) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  const int blocks = cache_attn_blocks(sms, D, NB);
  float* parts = static_cast<float*>(workspace);
  SharedHead* shared_heads = reinterpret_cast<SharedHead*>(parts + 2 * blocks * part_floats(8 * NB, D));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  config.gridDim = dim3(blocks);
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = kSmem;
  const cudaError_t e = cudaLaunchKernelEx(&config, kernel, *p, parts, shared_heads);
  if (e != cudaSuccess) return e;
  config.dynamicSmemBytes = 0;
  const int row_blocks = (p->tokens * (p->q_heads / p->cache.kv_heads) + 8 * NB - 1) / (8 * NB);
  const long long heads = (long long)p->seqs * p->cache.kv_heads * row_blocks;
  // few heads have many parts: blocks for each of their rows of their own
  config.gridDim = heads <= sms ? dim3((unsigned)heads, NB * 8) : dim3((unsigned)std::min<long long>(heads, blocks), 1);
  config.blockDim = dim3(kJoinWarps * 32);
  return cudaLaunchKernelEx(&config, cache_join_kernel<T, D, NB>, *p, (const float*)parts,
                            (const SharedHead*)shared_heads);
}

template <typename T, int CODE>
static cudaError_t cache_attn_of(int dim, int eights, const CacheAttnParams* p, void* workspace, int sms,
                                 cudaStream_t stream) {
  auto form = dim == 64    ? (eights == 2 ? cache_attn_form<T, CODE, 64, 2> : cache_attn_form<T, CODE, 64, 1>)
              : dim == 128 ? (eights == 2 ? cache_attn_form<T, CODE, 128, 2> : cache_attn_form<T, CODE, 128, 1>)
                           : (eights == 2 ? cache_attn_form<T, CODE, 256, 2> : cache_attn_form<T, CODE, 256, 1>);
  return form(p, workspace, sms, stream);
}

template <typename T>
static cudaError_t cache_attn_in(int code_type, int dim, int eights, const CacheAttnParams* p, void* workspace,
                                 int sms, cudaStream_t stream) {
  switch (code_type) {
    case Q8_INT8: return cache_attn_of<T, Q8_INT8>(dim, eights, p, workspace, sms, stream);
    case Q8_E4M3: return cache_attn_of<T, Q8_E4M3>(dim, eights, p, workspace, sms, stream);
    default: return cache_attn_of<T, Q8_INT4>(dim, eights, p, workspace, sms, stream);
  }
}

cudaError_t cache_attn_setup(int code_type, int dim) {
  for (int eights = 1; eights <= 2; ++eights) {
    cudaError_t e = cache_attn_in<__nv_bfloat16>(code_type, dim, eights, nullptr, nullptr, 0, nullptr);
    if (e == cudaSuccess) e = cache_attn_in<__half>(code_type, dim, eights, nullptr, nullptr, 0, nullptr);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_cache_attn(const CacheAttnParams& p, int value_type, void* workspace, int sms, cudaStream_t stream) {
  const int eights = cache_attn_eights(p.tokens, p.q_heads, p.cache.kv_heads);
  auto in = value_type == Q8_BF16 ? cache_attn_in<__nv_bfloat16> : cache_attn_in<__half>;
  return in(p.cache.code_type, p.cache.head_dim, eights, &p, workspace, sms, stream);
}

}  // namespace c3d
