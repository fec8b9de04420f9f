// q8_attn_api.cu -- the C ABI declared in include/q8_attention.h: validation, plans and launches.
#include <cmath>
#include <new>

#include "q8_attn_internal.h"
#include "q8_host.h"

using namespace c3d;

constexpr size_t kStatusBytes = 256;  // a workspace's head

namespace {

// What both plans hold: device memory that begins with a status word, zero between runs.
struct Plan {
  int device = -1;
  uint8_t* workspace = nullptr;
  size_t bytes = 0;
  unsigned long long timeout_ns = 0;
  int debug_flags = 0;
};

constexpr unsigned long long kTimeoutNs = 2000ull * 1000 * 1000;

void plan_options(Plan& plan, const attn_options* opts) {
  plan.timeout_ns = opts && opts->wait_timeout_ms > 0 ? opts->wait_timeout_ms * 1000000ull : kTimeoutNs;
  plan.debug_flags = opts ? opts->debug_flags : 0;
}

conv3d_status plan_memory(Plan& plan, int device, size_t bytes) {
  plan.device = device;
  plan.bytes = bytes;
  if (cudaMalloc(&plan.workspace, bytes) != cudaSuccess) {
    cudaGetLastError();
    plan.workspace = nullptr;
    return CONV3D_ENOMEM;
  }
  // in place for runs on every stream
  if (cudaMemset(plan.workspace, 0, bytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    cudaFree(plan.workspace);
    plan.workspace = nullptr;
    return CONV3D_ECUDA;
  }
  return CONV3D_OK;
}

conv3d_status plan_check(const Plan& plan) {
  DeviceRestore restore;
  int word = 0;
  if (cudaSetDevice(plan.device) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&word, plan.workspace, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  if (word == 0) return CONV3D_OK;
  // cleared before a run on any stream can report again
  if (cudaMemset(plan.workspace, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  return CONV3D_EDEVICE;
}

void plan_free(const Plan& plan) {
  DeviceRestore restore;
  if (cudaSetDevice(plan.device) == cudaSuccess) {
    cudaDeviceSynchronize();
    cudaFree(plan.workspace);
  }
  cudaGetLastError();
}

conv3d_status current_device_is(int device) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  return cur == device ? CONV3D_OK : CONV3D_EINVAL;
}

// A matrix of heads whose rows lie on 16 bytes and do not overlap: either its heads lie inside a token's
// pitch or its tokens inside a head's.
bool heads_ok(const void* p, long long tokens, int heads, int dim, long long pitch,
              long long head_pitch, int elem) {
  if (!p || !aligned(p, 16)) return false;
  if (tokens > 1 && (pitch < dim || pitch * elem % 16 != 0)) return false;
  if (heads > 1 && (head_pitch < dim || head_pitch * elem % 16 != 0)) return false;
  if (tokens <= 1 || heads <= 1) return true;
  typedef __int128 wide;  // a product of two 64-bit sizes
  return (wide)pitch >= (wide)(heads - 1) * head_pitch + dim ||
         (wide)head_pitch >= (wide)(tokens - 1) * pitch + dim;
}

// A pitch counts only where there is a second row.
Heads heads_of(const void* p, long long tokens, int heads, long long pitch, long long head_pitch) {
  return Heads{const_cast<void*>(p), tokens > 1 ? pitch : 0, heads > 1 ? head_pitch : 0};
}

conv3d_status check_cache(const q8_cache* c) {
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !aligned(c->k_codes, 16) ||
      !aligned(c->v_codes, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return CONV3D_EINVAL;
  if (c->pages < 1 || c->page_size < 1 || c->page_size % 16 != 0 || c->kv_heads < 1 ||
      c->head_dim < 1 || (!code_type_ok(c->code_type) && c->code_type != Q8_INT4))
    return CONV3D_EINVAL;
  if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->kv_heads >= (1 << 15) ||
      c->pages >= (1LL << 31) || c->pages * c->page_size >= (1LL << 31))
    return CONV3D_EUNSUPPORTED;
  return CONV3D_OK;
}

Cache cache_of(const q8_cache* c) {
  return Cache{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scale,
               c->v_scale, (unsigned)(c->pages * c->page_size), c->page_size, c->kv_heads,
               c->head_dim, c->code_type};
}

}  // namespace

struct attn_q8_plan_s : Plan {
  long long max_seqs = 0;
  int max_tokens = 0, q_heads = 0, kv_heads = 0, head_dim = 0, code_type = 0, sms = 0;
};
struct attn_prompt_plan_s : Plan {};

extern "C" conv3d_status heads_q8_run(const heads_q8_args* a) {
  if (!a) return CONV3D_EINVAL;
  const bool has_q = a->q != nullptr, has_k = a->k != nullptr;
  if ((!has_q && !has_k) || has_q != (a->q_out != nullptr) || a->tokens < 0 ||
      !value_type_ok(a->value_type) || a->head_dim < 1 || (has_q && a->q_heads < 1) ||
      (has_k && a->kv_heads < 1) || !(a->eps >= 0.0f) || std::isinf(a->eps))
    return CONV3D_EINVAL;
  const bool cached = a->cache != nullptr;
  if (cached != (a->v != nullptr) || cached != (a->slots != nullptr) || (cached && !has_k) ||
      (a->k_out && !has_k) || (has_k && !a->k_out && !cached) || (!has_q && a->q_weight) ||
      (!has_k && a->k_weight))
    return CONV3D_EINVAL;
  if (a->tokens >= (1LL << 31) || a->head_dim % 8 != 0 || a->head_dim > Q8_MAX_HEAD_DIM ||
      (has_q && a->q_heads >= (1 << 16)) || (has_k && a->kv_heads >= (1 << 16)))
    return CONV3D_EUNSUPPORTED;
  if ((a->q_weight || a->k_weight) && !value_type_ok(a->weight_type)) return CONV3D_EINVAL;
  if (a->turns && (a->rot_dim < 2 || a->rot_dim % 2 != 0 || a->rot_dim > a->head_dim || a->axes < 1 ||
                   a->axes > Q8_MAX_AXES || (a->axes > 1 && !a->axis) || !aligned(a->turns, 8)))
    return CONV3D_EINVAL;
  if (cached) {
    const conv3d_status st = check_cache(a->cache);
    if (st != CONV3D_OK) return st;
    if (a->cache->kv_heads != a->kv_heads || a->cache->head_dim != a->head_dim) return CONV3D_EINVAL;
  }
  if (a->tokens > 0) {
    const int vb = value_bytes(a->value_type), dim = a->head_dim;
    const int wb = a->q_weight || a->k_weight ? value_bytes(a->weight_type) : 1;
    if (a->turns && (!a->positions || !aligned(a->positions, 8) ||
                     (a->axes > 1 && a->positions_pitch != 0 && a->positions_pitch < a->tokens)))
      return CONV3D_EINVAL;
    if (!aligned(a->q_weight, wb) || !aligned(a->k_weight, wb) || !aligned(a->slots, 8))
      return CONV3D_EINVAL;
    if (has_q && (!heads_ok(a->q, a->tokens, a->q_heads, dim, a->q_pitch, a->q_head_pitch, vb) ||
                  !heads_ok(a->q_out, a->tokens, a->q_heads, dim, a->q_out_pitch, a->q_out_head_pitch, vb)))
      return CONV3D_EINVAL;
    if (has_k && !heads_ok(a->k, a->tokens, a->kv_heads, dim, a->k_pitch, a->k_head_pitch, vb))
      return CONV3D_EINVAL;
    if (a->k_out &&
        !heads_ok(a->k_out, a->tokens, a->kv_heads, dim, a->k_out_pitch, a->k_out_head_pitch, vb))
      return CONV3D_EINVAL;
    if (cached && !heads_ok(a->v, a->tokens, a->kv_heads, dim, a->v_pitch, a->v_head_pitch, vb))
      return CONV3D_EINVAL;
  }
  const conv3d_status st = check_device(a->device);
  if (st != CONV3D_OK || a->tokens == 0) return st;
  HeadsParams p{};
  const int q_heads = has_q ? a->q_heads : 0, kv_heads = has_k ? a->kv_heads : 0;
  p.q = heads_of(a->q, a->tokens, q_heads, a->q_pitch, a->q_head_pitch);
  p.q_out = heads_of(a->q_out, a->tokens, q_heads, a->q_out_pitch, a->q_out_head_pitch);
  p.k = heads_of(a->k, a->tokens, kv_heads, a->k_pitch, a->k_head_pitch);
  p.k_out = heads_of(a->k_out, a->tokens, kv_heads, a->k_out_pitch, a->k_out_head_pitch);
  p.v = heads_of(a->v, a->tokens, kv_heads, a->v_pitch, a->v_head_pitch);
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.turns = a->turns;
  p.axis = a->axes > 1 ? a->axis : nullptr;
  p.positions = a->positions;
  p.positions_pitch = a->axes > 1 ? a->positions_pitch : 0;
  p.slots = a->slots;
  if (cached) p.cache = cache_of(a->cache);
  p.tokens = (int)a->tokens;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.head_dim = a->head_dim;
  p.rot_dim = a->turns ? a->rot_dim : 0;
  p.axes = a->axes;
  p.weight_type = a->weight_type;
  p.eps = a->eps;
  return launched(launch_heads(p, a->value_type, cached ? a->cache->code_type : 0, a->adjacent != 0,
                               static_cast<cudaStream_t>(a->stream)));
}

extern "C" conv3d_status cache_q8_read_run(const cache_q8_read_args* a) {
  if (!a || !a->cache || a->tokens < 0 || !value_type_ok(a->value_type)) return CONV3D_EINVAL;
  conv3d_status st = check_cache(a->cache);
  if (st != CONV3D_OK) return st;
  if (a->tokens >= (1LL << 31) || a->tokens / 32 * 2 * a->cache->kv_heads >= (1LL << 30))
    return CONV3D_EUNSUPPORTED;
  const int vb = value_bytes(a->value_type), heads = a->cache->kv_heads, dim = a->cache->head_dim;
  if (a->tokens > 0 &&
      (!a->slots || !aligned(a->slots, 8) ||
       !heads_ok(a->k, a->tokens, heads, dim, a->k_pitch, a->k_head_pitch, vb) ||
       !heads_ok(a->v, a->tokens, heads, dim, a->v_pitch, a->v_head_pitch, vb)))
    return CONV3D_EINVAL;
  st = check_device(a->device);
  if (st != CONV3D_OK || a->tokens == 0) return st;
  ReadParams p{};
  p.cache = cache_of(a->cache);
  p.slots = a->slots;
  p.k = heads_of(a->k, a->tokens, heads, a->k_pitch, a->k_head_pitch);
  p.v = heads_of(a->v, a->tokens, heads, a->v_pitch, a->v_head_pitch);
  p.tokens = (int)a->tokens;
  return launched(launch_cache_read(p, a->value_type, static_cast<cudaStream_t>(a->stream)));
}

extern "C" conv3d_status attn_q8_plan(attn_q8_plan_t* plan, long long max_seqs, int max_tokens,
                                      int q_heads, int kv_heads, int head_dim, int code_type,
                                      int device) {
  return attn_q8_plan_ex(plan, max_seqs, max_tokens, q_heads, kv_heads, head_dim, code_type, device, nullptr);
}

extern "C" conv3d_status attn_q8_plan_ex(attn_q8_plan_t* plan, long long max_seqs, int max_tokens,
                                         int q_heads, int kv_heads, int head_dim, int code_type,
                                         int device, const attn_options* opts) {
  if (!plan) return CONV3D_EINVAL;
  *plan = nullptr;
  if (opts && opts->wait_timeout_ms < 0) return CONV3D_EINVAL;
  if (max_seqs < 1 || max_tokens < 1 || q_heads < 1 || kv_heads < 1 || head_dim < 1 ||
      q_heads % kv_heads != 0 || (!code_type_ok(code_type) && code_type != Q8_INT4))
    return CONV3D_EINVAL;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || max_seqs > 65536 || max_tokens > 64 ||
      q_heads >= 4096)
    return CONV3D_EUNSUPPORTED;
  conv3d_status st = check_device(device);
  if (st != CONV3D_OK) return st;
  attn_q8_plan_s* pl = new (std::nothrow) attn_q8_plan_s();
  if (!pl) return CONV3D_ENOMEM;
  pl->max_seqs = max_seqs;
  pl->max_tokens = max_tokens;
  pl->q_heads = q_heads;
  pl->kv_heads = kv_heads;
  pl->head_dim = head_dim;
  pl->code_type = code_type;
  plan_options(*pl, opts);
  if (cudaDeviceGetAttribute(&pl->sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
      cache_attn_setup(code_type, head_dim) != cudaSuccess) {
    cudaGetLastError();
    delete pl;
    return CONV3D_ECUDA;
  }
  st = plan_memory(*pl, device,
                   kStatusBytes + cache_attn_workspace(pl->sms, max_tokens, q_heads, kv_heads, head_dim));
  if (st != CONV3D_OK) {
    delete pl;
    return st;
  }
  *plan = pl;
  return CONV3D_OK;
}

extern "C" conv3d_status attn_q8_run(attn_q8_plan_t plan, const attn_q8_args* a) {
  if (!plan || !a || !a->cache) return CONV3D_EINVAL;
  const conv3d_status cache = check_cache(a->cache);
  if (cache != CONV3D_OK) return cache;
  if (a->seqs < 0 || a->seqs > plan->max_seqs || a->tokens < 1 || a->tokens > plan->max_tokens ||
      a->q_heads != plan->q_heads || a->cache->kv_heads != plan->kv_heads ||
      a->cache->head_dim != plan->head_dim || a->cache->code_type != plan->code_type ||
      (a->value_type != Q8_BF16 && a->value_type != Q8_F16) || !std::isfinite(a->scale))
    return CONV3D_EINVAL;
  const long long rows = a->seqs * a->tokens;
  if (a->seqs > 0) {
    if (!heads_ok(a->q, rows, a->q_heads, plan->head_dim, a->q_pitch, a->q_head_pitch, 2) ||
        !heads_ok(a->o, rows, a->q_heads, plan->head_dim, a->o_pitch, a->o_head_pitch, 2) || !a->table ||
        !aligned(a->table, 4) || !a->lengths || !aligned(a->lengths, 4) || a->table_width < 1 ||
        (a->seqs > 1 && a->table_pitch < a->table_width))
      return CONV3D_EINVAL;
    if (a->table_width >= (1LL << 31)) return CONV3D_EUNSUPPORTED;
  }
  const conv3d_status st = current_device_is(plan->device);
  if (st != CONV3D_OK || a->seqs == 0) return st;
  CacheAttnParams p{};
  p.cache = cache_of(a->cache);
  p.q = heads_of(a->q, rows, a->q_heads, a->q_pitch, a->q_head_pitch);
  p.o = heads_of(a->o, rows, a->q_heads, a->o_pitch, a->o_head_pitch);
  p.table = a->table;
  p.lengths = a->lengths;
  p.table_pitch = a->seqs > 1 ? a->table_pitch : 0;
  p.seqs = (int)a->seqs;
  p.tokens = a->tokens;
  p.q_heads = a->q_heads;
  p.table_width = (int)a->table_width;
  p.scale = a->scale;
  p.status = reinterpret_cast<int*>(plan->workspace);
  p.timeout_ns = plan->timeout_ns;
  p.debug_flags = plan->debug_flags;
  return launched(launch_cache_attn(p, a->value_type, plan->workspace + kStatusBytes, plan->sms,
                                    static_cast<cudaStream_t>(a->stream)));
}

extern "C" conv3d_status attn_q8_check(attn_q8_plan_t plan) {
  return plan ? plan_check(*plan) : CONV3D_EINVAL;
}
extern "C" size_t attn_q8_workspace_size(attn_q8_plan_t plan) { return plan ? plan->bytes : 0; }
extern "C" void attn_q8_destroy(attn_q8_plan_t plan) {
  if (!plan) return;
  plan_free(*plan);
  delete plan;
}

extern "C" conv3d_status attn_prompt_plan(attn_prompt_plan_t* plan, int device) {
  return attn_prompt_plan_ex(plan, device, nullptr);
}

extern "C" conv3d_status attn_prompt_plan_ex(attn_prompt_plan_t* plan, int device, const attn_options* opts) {
  if (!plan) return CONV3D_EINVAL;
  *plan = nullptr;
  if (opts && opts->wait_timeout_ms < 0) return CONV3D_EINVAL;
  conv3d_status st = check_device(device);
  if (st == CONV3D_OK) st = launched(prompt_attn_setup());
  if (st != CONV3D_OK) return st;
  attn_prompt_plan_s* pl = new (std::nothrow) attn_prompt_plan_s();
  if (!pl) return CONV3D_ENOMEM;
  plan_options(*pl, opts);
  st = plan_memory(*pl, device, kStatusBytes);
  if (st != CONV3D_OK) {
    delete pl;
    return st;
  }
  *plan = pl;
  return CONV3D_OK;
}

extern "C" conv3d_status attn_prompt_run(attn_prompt_plan_t plan, const attn_prompt_args* a) {
  if (!plan || !a) return CONV3D_EINVAL;
  if (a->q_rows < 0 || a->k_rows < 0 || a->seqs < 0 || a->q_heads < 1 || a->kv_heads < 1 ||
      a->head_dim < 1 || a->q_heads % a->kv_heads != 0 ||
      (a->value_type != Q8_BF16 && a->value_type != Q8_F16) || !std::isfinite(a->scale))
    return CONV3D_EINVAL;
  if (a->head_dim % 8 != 0 || a->head_dim > 128 || a->q_rows >= (1LL << 31) - 256 ||
      a->k_rows >= (1LL << 31) - 256 || a->seqs > 65536 || a->q_heads >= 65536 ||
      (a->q_rows / 256 + a->seqs) * a->q_heads >= (1LL << 31))
    return CONV3D_EUNSUPPORTED;
  if (a->seqs > 0 && a->q_rows > 0) {
    if (!heads_ok(a->q, a->q_rows, a->q_heads, a->head_dim, a->q_pitch, a->q_head_pitch, 2) ||
        !heads_ok(a->o, a->q_rows, a->q_heads, a->head_dim, a->o_pitch, a->o_head_pitch, 2) ||
        !a->starts || !aligned(a->starts, 4) || !aligned(a->key_starts, 4))
      return CONV3D_EINVAL;
    if (a->k_rows > 0 &&
        (!heads_ok(a->k, a->k_rows, a->kv_heads, a->head_dim, a->k_pitch, a->k_head_pitch, 2) ||
         !heads_ok(a->v, a->k_rows, a->kv_heads, a->head_dim, a->v_pitch, a->v_head_pitch, 2)))
      return CONV3D_EINVAL;
  }
  const conv3d_status st = current_device_is(plan->device);
  if (st != CONV3D_OK || a->seqs == 0 || a->q_rows == 0) return st;
  PromptParams p{};
  p.q = heads_of(a->q, a->q_rows, a->q_heads, a->q_pitch, a->q_head_pitch);
  p.k = heads_of(a->k, a->k_rows, a->kv_heads, a->k_pitch, a->k_head_pitch);
  p.v = heads_of(a->v, a->k_rows, a->kv_heads, a->v_pitch, a->v_head_pitch);
  p.o = heads_of(a->o, a->q_rows, a->q_heads, a->o_pitch, a->o_head_pitch);
  p.starts = a->starts;
  p.key_starts = a->key_starts;
  p.q_rows = (int)a->q_rows;
  p.k_rows = (int)a->k_rows;
  p.seqs = (int)a->seqs;
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.head_dim = a->head_dim;
  p.causal = a->causal;
  p.negate = a->scale < 0.0f;
  // a scale of 0 as 2^-149, which leaves every finite score below 2^-21 and -inf, a masked one, -inf; the largest ones finite
  p.scale = std::fmin(std::fmax(std::fabs(a->scale) * 1.44269504088896f, 0x1p-149f), 3.4028234e38f);
  p.status = reinterpret_cast<int*>(plan->workspace);
  p.timeout_ns = plan->timeout_ns;
  p.debug_flags = plan->debug_flags;
  return launched(launch_prompt_attn(p, a->value_type, static_cast<cudaStream_t>(a->stream)));
}

extern "C" conv3d_status attn_prompt_check(attn_prompt_plan_t plan) {
  return plan ? plan_check(*plan) : CONV3D_EINVAL;
}
extern "C" void attn_prompt_destroy(attn_prompt_plan_t plan) {
  if (!plan) return;
  plan_free(*plan);
  delete plan;
}
