// q8_attn_prompt.cu -- attention over whole prompts on the tensor cores, packed sequences, grouped heads.
//
// A block takes one unit after another: 256 rows of q of one head, two tiles A and B of 128. It walks over the keys 128 at
// a time:
//   S = Q K^T (tcgen05, both operands in shared memory), P = 2^(S scale - m) in registers, O += P V (P from TMEM, V from
//   shared memory), the running maximum m and sum l of a row held by the one thread that owns the row.
// TMEM is full: two S of 128 columns, two O of up to 128; P, half as wide as S, takes S's place. While one tile's
// softmax runs the tensor cores work on the other: PV_A(j), QK_A(j+1), PV_B(j), QK_B(j+1). The commit after QK_A(j+1)
// says that PV_A(j) is done too; products of one thread run in the order of their issue, so QK may overwrite the P that
// PV before it reads.
//
// m lags behind: O and l are scaled only when a row's maximum has grown by more than 2^8 over m (P is 2^7 there and stays
// below 2^15, so that f16 holds the largest and the small ones keep their bits), which is rare after the first keys; the
// row's thread then rescales O in TMEM.
//
// What a row does not see. A masked score is -inf, its weight 0; but 0 times a value that is not finite is NaN, so the tiles
// that some row sees only in part (the last ones of a block) pass two more warps, which zero such values in shared
// memory. Rows that do see them add them when they are done, read from memory again (their weight is positive, so the
// sum is the value).
//
// Roles: warps 0 to 7 softmax and epilogue (a row a thread), 8 the products, 9 the units and copies, 10 the gate (below), 11
// the check of values. They pass from unit to unit on their own: the next unit's copies and first scores run beside this
// one's last softmax and epilogue (a block for each unit: 4.3 us of 8 were its start and end for 500 keys of 64 channels).
// Every wait is bounded; one that runs out records a status bit and the block winds down.
//
// 8192 tokens, 32 heads of 128, causal: 385 us, 1.43 PFLOP/s, the tensor pipe active 63% of the time. The softmax bounds it:
// ~1300 cycles a tile in one warpgroup, two of which take turns, where the tile's products take ~550.
#include <algorithm>

#include "conv_common.cuh"
#include "q8_attn_internal.h"
#include "q8_common.cuh"
#include "q8_host.h"

namespace c3d {

constexpr int kRows = 128;                   // of a tile of q
constexpr int kKeys = 128;                   // of a tile of k and v
constexpr int kUnitRows = 2 * kRows;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kGateWarp = 10;  // and the check
constexpr int kPromptThreads = 12 * 32;
constexpr uint32_t kHalfBytes = 128 * 128;   // 64 channels of a tile: 128 rows of 128 bytes
constexpr int kPromptSlots = 5;              // tiles of k and v under way
constexpr float kNone = -INFINITY;           // m before the first key
constexpr float kFar = 65536.0f;             // of m in powers of two: from there on its multiple is off by 2^-8
constexpr float kGrowth = 8.0f;              // of a maximum, as a power of two, before O follows
constexpr float kHigh = 7.0f;                // P of the maximum, as a power of two: f16 has bits for small ones then
constexpr uint64_t kSettleNs = 2ull * 1000 * 1000;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256, kColTile = 128;

template <int HALVES>
constexpr uint32_t kTileBytes = HALVES * kHalfBytes;
template <int HALVES>
constexpr size_t kPromptSmem = 1024 + (2 + kPromptSlots) * (size_t)kTileBytes<HALVES> + 256;

// Barriers. The copies of tiles of v that are checked have their own, as the warp that checks does not follow the slots'
// phases; it then arrives for the slot in the copy's place. (The rows of a unit end within 255 keys of each other: 3 tiles.)
// Units alternate between two places, and with them those barriers: a role is at most one unit ahead of another.
// A slot is free again once the products that read it are complete, and its other readers must have seen its phase by then:
// the gate has for all copies whose products wait for it, which are all but a unit's first of k. For that one it arrives at
// kBarSeen, where the copies wait before they fill the slot again, or begin another unit. (A wait for the very copy, three
// barriers in turn and a record of the last slots, took 392 instead of 386 us for 8192 tokens and as long for short prompts.)
constexpr int kMostChecked = 3;
enum { kBarUnit, kBarUnitFree = kBarUnit + 2, kBarQ = kBarUnitFree + 2, kBarQFree, kBarBlock, kBarDrain, kBarRaw,
       kBarS = kBarRaw + 2 * kMostChecked, kBarP = kBarS + 2, kBarO = kBarP + 2, kBarFull = kBarO + 2,
       kBarEmpty = kBarFull + kPromptSlots, kBarSeen = kBarEmpty + kPromptSlots, kBarCount };

// 256 rows of one head of a sequence.
struct PromptUnit {
  int q0, queries;     // the sequence's rows of q
  int k0, keys;        // and of k
  int row0, head;      // the unit's first row in the sequence; head < 0: no more units
  int tiles[2];        // tiles of keys that each tile of rows sees
  int checked_from;    // tiles from here on are not seen whole by every row
  int poison;          // a value that is not finite was zeroed in one of those
};

// A warpgroup's registers a thread, raised or lowered. The block is launched with 168 for each of its 384 threads; 256 x 208
// and 128 x 80 are less than that in all, so the raise never waits for more than the others' drop.
constexpr int kSoftmaxRegisters = 208, kOtherRegisters = 80;
static_assert(256 * kSoftmaxRegisters + 128 * kOtherRegisters <= 384 * 168);
template <int N>
__device__ __forceinline__ void set_max_registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Takes over a block of this grid that has not started: asks for one, with the answer (16 bytes) in shared memory and its
// completion on the barrier, then whether there was one and which. Not to be asked again after there was none.
__device__ __forceinline__ void ask_for_block(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool answered_block(uint32_t answer, uint32_t& block) {
  uint32_t some;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(some), "=r"(block)
      : "r"(answer)
      : "memory");
  return some != 0;
}
// D (+)= A * B with A in TMEM (row i in lane i, two consecutive elements of K in each column), one CTA.
__device__ __forceinline__ void mma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of V as the B operand: channels (the product's N) contiguous, keys (its K) 128 bytes apart, 128-byte
// swizzle. Groups of 8 keys follow each other by 1024 bytes (stride offset), blocks of 64 channels by kHalfBytes
// (leading offset).
__device__ __forceinline__ uint64_t make_v_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kHalfBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(kLayoutSw128) << 61;
  return d;
}

template <typename T>
constexpr uint32_t kExponent2 = std::is_same_v<T, __half> ? 0x7C007C00u : 0x7F807F80u;  // of a pair
template <typename T>
constexpr uint32_t kCarry2 = std::is_same_v<T, __half> ? 0x04000400u : 0x00800080u;     // to the sign if all set

template <typename T, int HALVES>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const PromptParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[kBarCount];
  __shared__ PromptUnit units[2];
  __shared__ __align__(16) uint4 answer;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * i; };

  if (threadIdx.x == 0) {
    abort_word = 0;
    for (int i = 0; i < kBarCount; ++i)
      mbar_init(bar(i), i == kBarP || i == kBarP + 1                 ? 5                  // four of softmax, the gate
                        : i == kBarUnitFree || i == kBarUnitFree + 1 ? kSoftmaxWarps + 3  // all roles but the copies
                                                                     : 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int* abort_flag = &abort_word;
  const AbortState ab{abort_flag, p.status, p.timeout_ns};
  auto q_at = [&](int t) { return base + t * kTileBytes<HALVES>; };
  auto slot_at = [&](uint32_t i) { return base + (2 + i % kPromptSlots) * kTileBytes<HALVES>; };
  auto full = [&](uint32_t i) { return bar(kBarFull + i % kPromptSlots); };
  auto empty = [&](uint32_t i) { return bar(kBarEmpty + i % kPromptSlots); };
  auto lap = [&](uint32_t i) { return (i / kPromptSlots) & 1u; };
  // Keys that row r of a unit's sequence sees.
  auto limit_of = [&](const PromptUnit& u, int r) { return p.causal ? min(u.keys, max(0, r + 1 + u.keys - u.queries)) : u.keys; };
  // The block's n-th unit; false when there is none, or on abort.
  auto next_unit = [&](int n, PromptUnit& u) {
    if (!tc_wait(bar(kBarUnit + n % 2), (n / 2) & 1, ab, kAttnTimeout)) return false;
    u = units[n % 2];
    return u.head >= 0;
  };
  auto free_unit = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarUnitFree + n % 2));
  };

  if (warp < kSoftmaxWarps) {
    set_max_registers_up<kSoftmaxRegisters>();
    // ------------------------------------------------------------------------------ softmax
    const int t = warp / 4, row_in = t * kRows + (warp % 4) * 32;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;  // this warp's lanes of TMEM, << 16
    const uint32_t s_at = tmem + kColS + t * kColTile + lanes, o_at = tmem + kColO + t * kColTile + lanes;
    uint32_t scores = 0, outputs = 0;  // of this tile so far
    bool ok = true;
    for (int n = 0; ok; ++n) {
      int count, limit, whole;  // tiles; keys that this row sees, and that all rows of the warp see
      {
        PromptUnit u;
        if (!next_unit(n, u)) break;
        const int first = u.row0 + row_in;
        count = u.tiles[t];
        limit = first + lane < u.queries ? limit_of(u, first + lane) : 0;
        whole = first + 31 < u.queries ? limit_of(u, first) : 0;
      }
      float m = kNone;
      float2 l = make_float2(0.0f, 0.0f);
      for (int j = 0; j < count; ++j, ++scores) {
        ok = tc_wait(bar(kBarS + t), scores & 1, ab, kAttnTimeout);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
        auto load = [&] {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(s_at + 32 * i, s[i]);
          tmem_ld_wait();
          if (whole - j * kKeys < kKeys) {
            const int seen = limit - j * kKeys;
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (c >= seen) s[c / 32][c % 32] = 0xFF800000u;
          }
        };
        load();
        auto f = [&](int c) -> float { return __uint_as_float(s[c / 32][c % 32]); };
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(f(32 * i), f(32 * i + 1));
#pragma unroll
        for (int c = 2; c < 32; c += 2)
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = max3(top[i], f(32 * i + c), f(32 * i + c + 1));
        const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]);
        const bool grows = most > m && (m == kNone || (most - m) * p.scale > kGrowth);
        if (__any_sync(0xFFFFFFFFu, grows)) {
          // of the rows that grow: the others' results do not depend on their neighbours
          const float now = grows ? most : m, keep = !grows ? 1.0f : m == kNone ? 0.0f : exp2_fast((m - now) * p.scale);
          if (j > 0) {  // the tile's product before these scores is complete
#pragma unroll
            for (int i = 0; i < 2 * HALVES; ++i) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_at + 32 * i, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * keep);
              tmem_st_32x32b_x32(o_at + 32 * i, o);
            }
            load();  // there are no registers to hold them meanwhile
          }
          l.x *= keep;
          l.y *= keep;
          m = now;
        }
        float neg = m == kNone ? 0.0f : fmaf(-m, p.scale, kHigh);
        const bool far = m != kNone && !(fabsf(neg) < kFar);
        if (__any_sync(0xFFFFFFFFu, far)) {  // m is taken off first: what the multiple is off by would be P's exponent
          const float off = far ? m : 0.0f;
          neg = far ? kHigh : neg;
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c / 32][c % 32] = __float_as_uint(f(c) - off);
        }
        const float2 scale2 = make_float2(p.scale, p.scale), neg2 = make_float2(neg, neg);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            float2 x = make_float2(f(64 * half + 2 * c), f(64 * half + 2 * c + 1));
            x = q8_fma2(x, scale2, neg2);
            x.x = exp2_fast(x.x);
            x.y = exp2_fast(x.y);
            l = q8_add2(l, x);
            w[c] = q8_pack2<T>(x);
          }
          tmem_st_32x32b_x32(s_at + 32 * half, w);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + t));
      }
      // ---- the row's output
      if (ok && count > 0) {
        ok = tc_wait(bar(kBarO + t), outputs++ & 1, ab, kAttnTimeout);
        tc_fence_after();
      }
      if (!ok) break;
      const PromptUnit u = units[n % 2];  // read again: the loop above has no registers for it
      const int row = u.row0 + row_in + lane;
      const bool poison = u.poison != 0;
      const float sum = l.x + l.y, inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      T* out = static_cast<T*>(p.o.p) + (long long)(u.q0 + row) * p.o.pitch + u.head * p.o.head_pitch;
      const T* v = static_cast<const T*>(p.v.p) + (long long)u.k0 * p.v.pitch +
                   (u.head / (p.q_heads / p.kv_heads)) * p.v.head_pitch;
#pragma unroll
      for (int i = 0; i < 2 * HALVES; ++i) {
        uint32_t o[32];
        if (count > 0) {  // the same for the whole warp
          tmem_ld_32x32b_x32(o_at + 32 * i, o);
          tmem_ld_wait();
        }
        float x[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = sum == 0.0f ? 0.0f : __uint_as_float(o[c]) * inv;
        if (poison)
          for (int k = u.checked_from * kKeys; k < limit; ++k)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * i + c < p.head_dim) {
                const float add = q8_to_float(v[k * p.v.pitch + 32 * i + c]);
                if (!(fabsf(add) <= 3.4028234e38f)) x[c] += add;
              }
        if (row < u.queries) {
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            if (32 * i + c < p.head_dim) {
              uint4 w;
              w.x = q8_pack2<T>(make_float2(x[c], x[c + 1]));
              w.y = q8_pack2<T>(make_float2(x[c + 2], x[c + 3]));
              w.z = q8_pack2<T>(make_float2(x[c + 4], x[c + 5]));
              w.w = q8_pack2<T>(make_float2(x[c + 6], x[c + 7]));
              *reinterpret_cast<uint4*>(out + 32 * i + c) = w;
            }
        }
      }
      tc_fence_before();  // O is read before the next unit's first P arrives
      free_unit(n);
    }
  } else if (set_max_registers_down<kOtherRegisters>(); warp == kMmaWarp) {
    // ------------------------------------------------------------------------------ products
    constexpr bool kBf16 = !std::is_same_v<T, __half>;
    const uint32_t type = kBf16 ? make_idesc_bf16_f32(kRows, kKeys) : make_idesc_f16_f32(kRows, kKeys);
    const uint32_t qk_idesc = type | (p.negate ? 1u << 13 : 0u);  // -Q for a negative scale
    const uint32_t pv_idesc = (kBf16 ? make_idesc_bf16_f32(kRows, 64 * HALVES) : make_idesc_f16_f32(kRows, 64 * HALVES)) |
                              (1u << 16);  // B lies with its N contiguous
    const int qk_steps = (p.head_dim + 15) / 16;
    // The tensor cores take few instructions ahead, so whatever this warp does between two products leaves them idle (a wait
    // takes it some 150 cycles, eight products 512): it waits once a round, for P, whose barrier the gate warp holds until
    // V and the next K are there too, and commits what somebody waits for.
    // Descriptors of the first tiles; others lie a multiple of 16 bytes further on.
    constexpr uint32_t kTile16 = kTileBytes<HALVES> >> 4;
    const uint64_t q_desc = make_sw128_kmajor_desc(q_at(0)), k_desc = make_sw128_kmajor_desc(slot_at(0));
    const uint64_t v_desc = make_v_desc(slot_at(0));
    auto qk = [&](int t, uint32_t slot, bool last_use, bool last_of_unit) {
      if (elect_one()) {
        const uint64_t a = q_desc + t * kTile16, b = k_desc + slot * kTile16;
#pragma unroll
        for (int s = 0; s < 4 * HALVES; ++s)
          if (s < qk_steps) {
            const uint32_t at = (s / 4) * (kHalfBytes >> 4) + (s % 4) * 2;
            mma_bf16(tmem + kColS + t * kColTile, a + at, b + at, qk_idesc, s > 0);
          }
        mma_commit(bar(kBarS + t));  // the product of P and V before it is then complete too
        if (last_use) mma_commit(bar(kBarEmpty + slot));
        if (last_of_unit) mma_commit(bar(kBarQFree));
      }
      __syncwarp();
    };
    uint32_t copies = 0, with_tiles = 0;      // before this unit: copies of k and v, units that had any
    uint32_t rounds[2] = {0, 0};              // of P so far
    PromptUnit u;
    bool ok = true;
    for (int n = 0; ok && next_unit(n, u); ++n) {
      const int all = max(u.tiles[0], u.tiles[1]);
      if (all > 0) {
        ok = tc_wait(bar(kBarQ), with_tiles++ & 1, ab, kAttnTimeout) && tc_wait(full(copies), lap(copies), ab, kAttnTimeout);
        tc_fence_after();
      }
      // Tile t's last use of the tile j of keys.
      auto last_use = [&](int t, int j) { return t == 1 || u.tiles[1] <= j; };
      for (int t = 0; t < 2; ++t)
        if (ok && u.tiles[t] > 0) qk(t, copies % kPromptSlots, last_use(t, 0), all == 1 && last_use(t, 0));
      for (int j = 0; ok && j < all; ++j) {
        const uint32_t v_slot = (copies + 2 * j + 1) % kPromptSlots, k_slot = (copies + 2 * j + 2) % kPromptSlots;
        for (int t = 0; t < 2; ++t) {
          if (j >= u.tiles[t]) continue;
          ok = tc_wait(bar(kBarP + t), rounds[t]++ & 1, ab, kAttnTimeout);
          if (!ok) break;
          tc_fence_after();
          const bool more = j + 1 < u.tiles[t];
          if (elect_one()) {
            const uint64_t b = v_desc + v_slot * kTile16;
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              mma_f16_tmem_a(tmem + kColO + t * kColTile, tmem + kColS + t * kColTile + 8 * s, b + s * (2048 >> 4),
                             pv_idesc, j > 0 || s > 0);
            if (!more) mma_commit(bar(kBarO + t));
            if (last_use(t, j)) mma_commit(bar(kBarEmpty + v_slot));
          }
          __syncwarp();
          if (more) qk(t, k_slot, last_use(t, j + 1), j + 2 == all && last_use(t, j + 1));
        }
      }
      copies += 2 * all;
      if (ok) free_unit(n);
    }
    // every product is complete before TMEM is released
    if (elect_one()) mma_commit(bar(kBarDrain));
    __syncwarp();
    wait_drain(bar(kBarDrain), 0, p.timeout_ns, p.status, kAttnTimeout);
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------------------------------------ units and copies
    // Units of all sequences are counted from the last one, which has the most keys, heads first; there is a block for each
    // (or more). A block that has issued its unit's copies takes over another that has not started.
    auto begin_of = [&](const int* starts, int b, int rows) { return min(max(starts[b], 0), rows); };
    auto end_of = [&](const int* starts, int b, int rows, int begin) { return min(max(starts[b + 1], begin), rows); };
    const int* key_starts = p.key_starts ? p.key_starts : p.starts;
    long long behind = 0, wanted = 0;  // units of the sequences from `from` on; the last one asked for
    int from = p.seqs;
    auto find = [&](long long want, PromptUnit& u) {
      if (want < wanted) behind = 0, from = p.seqs;
      wanted = want;
      while (from > 0) {
        const int b = from - 1 - lane;
        int q0 = 0, queries = 0;
        if (b >= 0) {
          q0 = begin_of(p.starts, b, p.q_rows);
          queries = end_of(p.starts, b, p.q_rows, q0) - q0;
        }
        const int mine = (queries + kUnitRows - 1) / kUnitRows;
        long long sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, behind + sum > want);
        if (hit) {
          const int at = __ffs(hit) - 1;
          const long long upto = __shfl_sync(0xFFFFFFFFu, sum, at);
          const int b_at = from - 1 - at;
          u.q0 = __shfl_sync(0xFFFFFFFFu, q0, at);
          u.queries = __shfl_sync(0xFFFFFFFFu, queries, at);
          u.row0 = (int)(behind + upto - 1 - want) * kUnitRows;
          u.k0 = begin_of(key_starts, b_at, p.k_rows);
          u.keys = end_of(key_starts, b_at, p.k_rows, u.k0) - u.k0;
          return true;
        }
        behind += __shfl_sync(0xFFFFFFFFu, sum, 31);
        from -= 32;
      }
      return false;
    };
    uint32_t copies = 0, with_tiles = 0;
    uint32_t seen = 0;  // units whose first copy of k the gate is known to have seen
    uint32_t block = blockIdx.x, asked = 0;
    bool first = true;  // this block's own
    for (int n = 0;; ++n) {
      // The next block that has a unit (those behind the last unit have none: they are taken over here one after another,
      // where it is known that there are no more).
      PromptUnit u;
      u.poison = 0;
      u.head = -1;
      bool answered = true;
      for (bool some = true; some; first = false) {
        if (!first) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(kBarBlock), 16);
            ask_for_block(smem_u32(&answer), bar(kBarBlock));
          }
          __syncwarp();
          answered = tc_wait(bar(kBarBlock), asked++ & 1, ab, kAttnTimeout);
          some = answered && answered_block(smem_u32(&answer), block);
          fence_proxy_async_smem();  // the next answer comes to the same place
          __syncwarp();
        }
        if (some && find(block / p.q_heads, u)) {
          u.head = (int)(block % p.q_heads);
          first = false;
          break;
        }
      }
      if (!answered) break;
      if (u.head >= 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int first = u.row0 + t * kRows, last = min(first + kRows, u.queries) - 1;
          u.tiles[t] = first < u.queries ? (limit_of(u, last) + kKeys - 1) / kKeys : 0;
        }
        u.checked_from = limit_of(u, u.row0) / kKeys;
      }
      if (n >= 2 && !tc_wait(bar(kBarUnitFree + n % 2), (n / 2 - 1) & 1, ab, kAttnTimeout)) break;
      if (lane == 0) {
        units[n % 2] = u;
        mbar_arrive(bar(kBarUnit + n % 2));
      }
      __syncwarp();
      if (u.head < 0) break;
      const int all = max(u.tiles[0], u.tiles[1]), kv_head = u.head / (p.q_heads / p.kv_heads);
      if (all == 0) continue;
      if (with_tiles > 0 && !tc_wait(bar(kBarQFree), (with_tiles - 1) & 1, ab, kAttnTimeout)) break;
      if (seen < with_tiles && !tc_wait(bar(kBarSeen), seen++ & 1, ab, kAttnTimeout)) break;
      ++with_tiles;
      if (elect_one()) {
        const int q_tiles = u.tiles[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(bar(kBarQ), q_tiles * kTileBytes<HALVES>);
        for (int t = 0; t < q_tiles; ++t)
          for (int h = 0; h < HALVES; ++h)
            tma_load_3d(q_at(t) + h * kHalfBytes, &qmap, bar(kBarQ), 64 * h, u.head, u.q0 + u.row0 + t * kRows);
      }
      __syncwarp();
      bool ok = true;
      for (int i = 0; ok && i < 2 * all; ++i) {  // k of tile i / 2, then v
        const uint32_t c = copies + i;
        if (c >= kPromptSlots) ok = tc_wait(empty(c), lap(c) ^ 1u, ab, kAttnTimeout);
        if (ok && i == kPromptSlots) ok = tc_wait(bar(kBarSeen), seen++ & 1, ab, kAttnTimeout);
        if (ok && elect_one()) {
          const uint32_t to =
              i % 2 && i / 2 >= u.checked_from ? bar(kBarRaw + kMostChecked * (n % 2) + i / 2 - u.checked_from) : full(c);
          mbar_arrive_expect_tx(to, kTileBytes<HALVES>);
          const bool skip = (p.debug_flags & 1) && blockIdx.x == 0 && c == 0;
          for (int h = skip ? HALVES : 0; h < HALVES; ++h)
            tma_load_3d(slot_at(c) + h * kHalfBytes, i % 2 ? &vmap : &kmap, to, 64 * h, kv_head, u.k0 + (i / 2) * kKeys);
        }
        __syncwarp();
      }
      if (!ok) break;
      copies += 2 * all;
    }
  } else if (warp == kGateWarp) {
    // ------------------------------------------------------------------------------ the gate
    // Arrives for round j of P once the copies are there that its products read, and the round before is over.
    uint32_t copies = 0, rounds[2] = {0, 0};
    PromptUnit u;
    bool ok = true;
    for (int n = 0; ok && next_unit(n, u); ++n) {
      const int all = max(u.tiles[0], u.tiles[1]);
      if (all > 0) {  // no phase of a slot is passed over
        ok = tc_wait(full(copies), lap(copies), ab, kAttnTimeout);
        if (ok && lane == 0) mbar_arrive(bar(kBarSeen));
      }
      for (int j = 0; ok && j < all; ++j) {
        const uint32_t v = copies + 2 * j + 1;
        ok = tc_wait(full(v), lap(v), ab, kAttnTimeout) &&
             (j + 1 >= all || tc_wait(full(v + 1), lap(v + 1), ab, kAttnTimeout));
        for (int t = 0; ok && t < 2; ++t) {
          if (j >= u.tiles[t]) continue;
          ok = rounds[t] == 0 || tc_wait(bar(kBarP + t), (rounds[t] - 1) & 1, ab, kAttnTimeout);
          ++rounds[t];
          if (ok && lane == 0) mbar_arrive(bar(kBarP + t));
        }
      }
      copies += 2 * all;
      if (ok) free_unit(n);
    }
  } else {
    // ------------------------------------------------------------------------------ values that are not finite
    uint32_t copies = 0, checked[2][kMostChecked] = {};
    PromptUnit u;
    bool ok = true;
    for (int n = 0; ok && next_unit(n, u); ++n) {
      const int all = max(u.tiles[0], u.tiles[1]);
#pragma unroll
      for (int c = 0; c < kMostChecked; ++c) {
        const int j = u.checked_from + c;
        if (!ok || j >= all) break;
        ok = tc_wait(bar(kBarRaw + kMostChecked * (n % 2) + c), (n % 2 ? checked[1][c]++ : checked[0][c]++) & 1, ab, kAttnTimeout);
        if (!ok) break;
        const uint32_t copy = copies + 2 * j + 1;
        uint8_t* tile = raw + (slot_at(copy) - smem_u32(raw));
        // 16 bytes at a time: whether any is not finite, before which
        uint32_t any = 0;
#pragma unroll 8
        for (uint32_t i = lane; i < kTileBytes<HALVES> / 16; i += 32) {
          const uint4 w = *reinterpret_cast<const uint4*>(tile + 16 * i);
          any |= (w.x & kExponent2<T>) + kCarry2<T>;
          any |= (w.y & kExponent2<T>) + kCarry2<T>;
          any |= (w.z & kExponent2<T>) + kCarry2<T>;
          any |= (w.w & kExponent2<T>) + kCarry2<T>;
        }
        if (__any_sync(0xFFFFFFFFu, any & 0x80008000u)) {
          for (uint32_t i = lane; i < kTileBytes<HALVES> / 4; i += 32) {
            uint32_t* word = reinterpret_cast<uint32_t*>(tile) + i;
            const uint32_t bad = ((*word & kExponent2<T>) + kCarry2<T>) & 0x80008000u;
            if (!bad) continue;
            const int key = j * kKeys + (int)(i * 4 % kHalfBytes) / 128;
            *word &= (bad & 0x8000u ? 0u : 0xFFFFu) | (bad & 0x80000000u ? 0u : 0xFFFF0000u);
            if (key < u.keys) *reinterpret_cast<volatile int*>(&units[n % 2].poison) = 1;
          }
          __threadfence_block();
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full(copy));
      }
      copies += 2 * all;
      if (ok) free_unit(n);
    }
  }
  __syncwarp();
  if (*abort_flag) sleep_ns_bounded(kSettleNs);  // copies in flight land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Heads of 16-bit values in boxes of 64 channels by 128 rows of one head; what lies outside reads zero.
static bool encode_heads(CUtensorMap* map, const Heads& m, bool bf16, int rows, int heads, int dim) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const long long unit = (dim + 7) / 8 * 8;  // a pitch that no second row uses
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)(2 * (heads > 1 ? m.head_pitch : unit)),
                                 (cuuint64_t)(2 * (rows > 1 ? m.pitch : unit * heads))};
  const cuuint32_t box[3] = {64, 1, 128}, steps[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, m.p, dims, strides,
             box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int HALVES>
static cudaError_t prompt_form(const PromptParams* p, cudaStream_t stream) {
  auto kernel = prompt_attn_kernel<T, HALVES>;
  if (!p) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPromptSmem<HALVES>);
  constexpr bool kBf16 = !std::is_same_v<T, __half>;
  CUtensorMap qmap{}, kmap{}, vmap{};
  if (!encode_heads(&qmap, p->q, kBf16, p->q_rows, p->q_heads, p->head_dim)) return cudaErrorInvalidValue;
  if (p->k_rows == 0) {
    kmap = vmap = qmap;  // not used
  } else if (!encode_heads(&kmap, p->k, kBf16, p->k_rows, p->kv_heads, p->head_dim) ||
             !encode_heads(&vmap, p->v, kBf16, p->k_rows, p->kv_heads, p->head_dim)) {
    return cudaErrorInvalidValue;
  }
  const long long units = p->q_rows / kUnitRows + std::min<long long>(p->seqs, p->q_rows);  // at most
  kernel<<<(unsigned)(units * p->q_heads), kPromptThreads, kPromptSmem<HALVES>, stream>>>(qmap, kmap, vmap, *p);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t prompt_of(int dim, const PromptParams* p, cudaStream_t stream) {
  return dim <= 64 ? prompt_form<T, 1>(p, stream) : prompt_form<T, 2>(p, stream);
}

cudaError_t prompt_attn_setup() {
  for (int dim : {64, 128}) {
    cudaError_t e = prompt_of<__nv_bfloat16>(dim, nullptr, nullptr);
    if (e == cudaSuccess) e = prompt_of<__half>(dim, nullptr, nullptr);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_prompt_attn(const PromptParams& p, int value_type, cudaStream_t stream) {
  return value_type == Q8_BF16 ? prompt_of<__nv_bfloat16>(p.head_dim, &p, stream) : prompt_of<__half>(p.head_dim, &p, stream);
}

}  // namespace c3d
