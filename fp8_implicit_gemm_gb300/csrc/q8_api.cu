// q8_api.cu -- the C ABI declared in include/q8.h: validation, planning and launch.
#include <algorithm>
#include <cmath>
#include <new>

#include "q8_host.h"
#include "q8_internal.h"

using namespace c3d;

struct linear_q8_plan_s {
  int device = -1;
  int code_type = 0;
  long long max_rows = 0, N = 0, K = 0;
  TcLimits lim{};
  int kernel = 0;                  // as in the options
  unsigned long long timeout_ns = 0;
  int debug_flags = 0;
  uint8_t* workspace = nullptr;    // status word; x as f16 (int8)
  size_t workspace_bytes = 0;
};

constexpr size_t kStatusBytes = 256;  // the workspace's head


namespace {

// A matrix argument: its pointer, the alignment it needs and its pitch (which a single row has no
// use for).
bool matrix_ok(const void* p, int align, long long rows, long long pitch, long long cols) {
  return p && aligned(p, align) && (rows <= 1 || pitch >= cols);
}

// Sizes and the matrices that both row operators have.
conv3d_status check_rows(long long rows, long long cols, int value_type, int code_type) {
  if (rows < 0 || cols < 1 || !value_type_ok(value_type) || !code_type_ok(code_type))
    return CONV3D_EINVAL;
  if (cols > Q8_MAX_COLS || rows >= (1LL << 31)) return CONV3D_EUNSUPPORTED;
  return CONV3D_OK;
}

constexpr unsigned long long kLinearTimeoutNs = 2000ull * 1000ull * 1000ull;

// A matrix of codes (elem 1) or f16 (elem 2), loaded in boxes of 128 bytes by box_rows rows with the
// 128-byte swizzle; what lies outside reads zero.
bool encode_rows(CUtensorMap* map, const void* base, int elem, long long rows, long long cols,
                 long long pitch, int box_rows) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(pitch * elem)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y, stored in boxes of 32 channels by as many tokens as make 2 KB; what lies outside is dropped. The
// boxes of a 16-bit y are swizzled, for the matrix stores that fill them.
bool encode_y(CUtensorMap* map, void* y, int y_type, long long rows, long long cols,
              long long pitch) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const int elem = value_bytes(y_type);
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(pitch * elem)};
  const cuuint32_t box[2] = {32, (cuuint32_t)(kTcYBoxBytes / (32 * elem))};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType type = y_type == Q8_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : y_type == Q8_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, type, 2, y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             elem == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where the rows start. A pitch counts only between rows.
RowsGrid rows_grid(const RowsParams& p, int vb, int weight_bytes) {
  auto all_on = [&](int value_grid, int code_grid, int weight_grid) {
    auto on = [&](const void* m, long long pitch, int grid, int elem) {
      return !m || (aligned(m, grid) && (p.rows <= 1 || pitch * elem % grid == 0));
    };
    return on(p.a, p.a_pitch, value_grid, vb) && on(p.b, p.b_pitch, value_grid, vb) &&
           on(p.sum_out, p.sum_pitch, value_grid, vb) && on(p.q, p.q_pitch, code_grid, 1) &&
           aligned(p.weight, weight_grid);
  };
  if (all_on(16, 8, 16)) return RowsGrid::kChunk;
  if (p.cols % 2 == 0 && all_on(2 * vb, 2, 2 * weight_bytes)) return RowsGrid::kPair;
  return RowsGrid::kElement;
}

}  // namespace

extern "C" conv3d_status rmsnorm_q8_run(const rmsnorm_q8_args* a) {
  if (!a) return CONV3D_EINVAL;
  conv3d_status st = check_rows(a->rows, a->cols, a->value_type, a->code_type);
  if (st != CONV3D_OK) return st;
  if (!value_type_ok(a->weight_type) || !(a->eps >= 0.0f) || std::isinf(a->eps) ||
      (a->residual == nullptr) != (a->residual_out == nullptr))
    return CONV3D_EINVAL;
  const int vb = value_bytes(a->value_type);
  if (a->rows > 0) {
    if (!matrix_ok(a->x, vb, a->rows, a->x_pitch, a->cols) ||
        !matrix_ok(a->q, 1, a->rows, a->q_pitch, a->cols) ||
        !a->scale || !aligned(a->scale, 4) || !a->weight ||
        !aligned(a->weight, value_bytes(a->weight_type)))
      return CONV3D_EINVAL;
    if (a->residual && (!matrix_ok(a->residual, vb, a->rows, a->residual_pitch, a->cols) ||
                        !matrix_ok(a->residual_out, vb, a->rows, a->residual_out_pitch, a->cols)))
      return CONV3D_EINVAL;
  }
  st = check_device(a->device);
  if (st != CONV3D_OK || a->rows == 0) return st;
  RowsParams p{};
  p.a = a->x;
  p.b = a->residual;
  p.weight = a->weight;
  p.sum_out = a->residual_out;
  p.q = static_cast<uint8_t*>(a->q);
  p.scale = a->scale;
  p.a_pitch = a->x_pitch;
  p.b_pitch = a->residual_pitch;
  p.sum_pitch = a->residual_out_pitch;
  p.q_pitch = a->q_pitch;
  p.rows = a->rows;
  p.cols = (int)a->cols;
  p.code_type = a->code_type;
  p.weight_type = a->weight_type;
  p.eps = a->eps;
  const RowsGrid grid = rows_grid(p, vb, value_bytes(a->weight_type));
  return launched(
      launch_rows_q8(p, a->value_type, true, grid, static_cast<cudaStream_t>(a->stream)));
}

extern "C" conv3d_status silu_mul_q8_run(const silu_mul_q8_args* a) {
  if (!a) return CONV3D_EINVAL;
  conv3d_status st = check_rows(a->rows, a->cols, a->value_type, a->code_type);
  if (st != CONV3D_OK) return st;
  const int vb = value_bytes(a->value_type);
  if (a->rows > 0 &&
      (!matrix_ok(a->gate, vb, a->rows, a->gate_pitch, a->cols) ||
       !matrix_ok(a->up, vb, a->rows, a->up_pitch, a->cols) ||
       !matrix_ok(a->q, 1, a->rows, a->q_pitch, a->cols) ||
       !a->scale || !aligned(a->scale, 4)))
    return CONV3D_EINVAL;
  st = check_device(a->device);
  if (st != CONV3D_OK || a->rows == 0) return st;
  RowsParams p{};
  p.a = a->gate;
  p.b = a->up;
  p.q = static_cast<uint8_t*>(a->q);
  p.scale = a->scale;
  p.a_pitch = a->gate_pitch;
  p.b_pitch = a->up_pitch;
  p.q_pitch = a->q_pitch;
  p.rows = a->rows;
  p.cols = (int)a->cols;
  p.code_type = a->code_type;
  return launched(launch_rows_q8(p, a->value_type, false, rows_grid(p, vb, 1),
                                 static_cast<cudaStream_t>(a->stream)));
}

extern "C" conv3d_status linear_q8_plan(linear_q8_plan_t* plan, long long max_rows, long long N,
                                        long long K, int code_type, int device) {
  return linear_q8_plan_ex(plan, max_rows, N, K, code_type, device, nullptr);
}

extern "C" conv3d_status linear_q8_plan_ex(linear_q8_plan_t* plan, long long max_rows, long long N,
                                           long long K, int code_type, int device,
                                           const linear_q8_options* opts) {
  if (!plan) return CONV3D_EINVAL;
  *plan = nullptr;
  if (max_rows < 1 || N < 1 || K < 1 || !code_type_ok(code_type)) return CONV3D_EINVAL;
  linear_q8_options o{};
  if (opts) o = *opts;
  if (o.kernel < 0 || o.kernel > 2 || o.block_t < 0 || o.block_t > tc_most_tokens(code_type) ||
      o.block_t % 32 != 0 || o.splits < 0 || o.splits > kTcMaxSplits ||
      o.max_ctas < 0 || o.wait_timeout_ms < 0)
    return CONV3D_EINVAL;
  if (max_rows >= (1LL << 30) || N >= (1LL << 30) || K >= (1LL << 30)) return CONV3D_EUNSUPPORTED;
  if (o.kernel == 1 && max_rows > few_tokens(code_type)) return CONV3D_EUNSUPPORTED;
  const conv3d_status st = check_device(device);
  if (st != CONV3D_OK) return st;
  linear_q8_plan_s* pl = new (std::nothrow) linear_q8_plan_s();
  if (!pl) return CONV3D_ENOMEM;
  pl->device = device;
  pl->code_type = code_type;
  pl->max_rows = max_rows;
  pl->N = N;
  pl->K = K;
  pl->kernel = o.kernel;
  pl->timeout_ns = o.wait_timeout_ms > 0 ? o.wait_timeout_ms * 1000000ull : kLinearTimeoutNs;
  pl->debug_flags = o.debug_flags;
  // few tokens need no workspace; a product of fewer tokens than max_rows is not dearer to them
  if (o.kernel != 1 && (o.kernel == 2 || !prefer_few(max_rows, N, K, code_type))) {
    if (linear_tc_setup() != cudaSuccess || linear_tc_max_clusters(pl->lim.clusters) != cudaSuccess) {
      cudaGetLastError();
      delete pl;
      return CONV3D_ECUDA;
    }
    for (int i = 0; i < kTcMaxSplits; ++i)
      if (o.max_ctas > 0)
        pl->lim.clusters[i] = std::min(pl->lim.clusters[i], o.max_ctas / (2 * (i + 1)));
    pl->lim.block_t = o.block_t;
    pl->lim.splits = o.splits;
    pl->workspace_bytes = kStatusBytes;
    if (code_type == Q8_INT8)
      pl->workspace_bytes += (size_t)(max_rows * round_up(K, 16) * 2);
    if (cudaMalloc(&pl->workspace, pl->workspace_bytes) != cudaSuccess) {
      cudaGetLastError();
      delete pl;
      return CONV3D_ENOMEM;
    }
    // the status word is zero between runs; on every stream from here on
    if (cudaMemset(pl->workspace, 0, kStatusBytes) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
      cudaGetLastError();
      cudaFree(pl->workspace);
      delete pl;
      return CONV3D_ECUDA;
    }
  }
  *plan = pl;
  return CONV3D_OK;
}

extern "C" conv3d_status linear_q8_run(linear_q8_plan_t plan, const linear_q8_args* a) {
  if (!plan || !a) return CONV3D_EINVAL;
  if (a->rows < 0 || a->rows > plan->max_rows || a->N != plan->N || a->K != plan->K ||
      a->code_type != plan->code_type || !value_type_ok(a->y_type))
    return CONV3D_EINVAL;
  if (a->bias && (!value_type_ok(a->bias_type) || !aligned(a->bias, value_bytes(a->bias_type))))
    return CONV3D_EINVAL;
  if (a->rows > 0) {
    if (!matrix_ok(a->x, 16, a->rows, a->x_pitch, plan->K) ||
        !matrix_ok(a->w, 16, plan->N, a->w_pitch, plan->K) ||
        !matrix_ok(a->y, value_bytes(a->y_type), a->rows, a->y_pitch, plan->N) || !a->scale_x ||
        !aligned(a->scale_x, 4) || !a->scale_w || !aligned(a->scale_w, 4))
      return CONV3D_EINVAL;
    if ((a->rows > 1 && a->x_pitch % 16 != 0) || (plan->N > 1 && a->w_pitch % 16 != 0))
      return CONV3D_EINVAL;
  }
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  if (cur != plan->device) return CONV3D_EINVAL;
  if (a->rows == 0) return CONV3D_OK;
  LinearParams p{};
  p.x = static_cast<const uint8_t*>(a->x);
  p.scale_x = a->scale_x;
  p.w = static_cast<const uint8_t*>(a->w);
  p.scale_w = a->scale_w;
  p.bias = a->bias;
  p.y = a->y;
  p.x_pitch = a->rows > 1 ? a->x_pitch : round_up(plan->K, 16);
  p.w_pitch = plan->N > 1 ? a->w_pitch : round_up(plan->K, 16);
  p.y_pitch = a->y_pitch;
  p.M = (int)a->rows;
  p.N = (int)plan->N;
  p.K = (int)plan->K;
  p.y_type = a->y_type;
  p.bias_type = a->bias_type;
  const int yb = value_bytes(a->y_type);
  p.y_vec = aligned(a->y, 4 * yb) && (p.M <= 1 || p.y_pitch % 4 == 0);
  cudaStream_t stream = static_cast<cudaStream_t>(a->stream);
  if (plan->kernel == 1 || !plan->workspace ||
      (plan->kernel == 0 && prefer_few(p.M, p.N, p.K, plan->code_type)))
    return launched(launch_linear_few(p, plan->code_type, stream));
  linear_tc_decide(p, plan->code_type, plan->lim);
  if (!p.block_t) return CONV3D_EUNSUPPORTED;  // the options leave no tiling for this many tokens
  p.status = reinterpret_cast<int*>(plan->workspace);
  p.xh = reinterpret_cast<uint16_t*>(plan->workspace + kStatusBytes);
  p.xh_pitch = round_up(plan->K, 16);
  p.timeout_ns = plan->timeout_ns;
  p.debug_flags = plan->debug_flags;
  const long long y_pitch = p.M > 1 ? p.y_pitch : round_up(p.N, 8);
  p.y_tma = aligned(p.y, 16) && y_pitch * value_bytes(p.y_type) % 16 == 0;
  const bool int8 = plan->code_type == Q8_INT8;
  CUtensorMap wmap{}, xmap{}, ymap{};
  if (!encode_rows(&wmap, p.w, 1, p.N, p.K, p.w_pitch, kTcWBoxRows) ||
      !(int8 ? encode_rows(&xmap, p.xh, 2, p.M, p.K, p.xh_pitch, p.block_t / 2)
                     : encode_rows(&xmap, p.x, 1, p.M, p.K, p.x_pitch, p.block_t / 2)) ||
      (p.y_tma && !encode_y(&ymap, p.y, p.y_type, p.M, p.N, y_pitch)))
    return CONV3D_ECUDA;
  if (int8) {
    const conv3d_status st = launched(launch_linear_expand(p, stream));
    if (st != CONV3D_OK) return st;
  }
  return launched(launch_linear_tc(p, plan->code_type, wmap, xmap, ymap, plan->lim, stream));
}

extern "C" conv3d_status linear_q8_check(linear_q8_plan_t plan) {
  if (!plan) return CONV3D_EINVAL;
  DeviceRestore restore;
  if (cudaSetDevice(plan->device) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
    return CONV3D_ECUDA;
  if (!plan->workspace) return CONV3D_OK;
  int word = 0;
  if (cudaMemcpy(&word, plan->workspace, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return CONV3D_ECUDA;
  if (word == 0) return CONV3D_OK;
  // cleared before a run on any stream can report again
  if (cudaMemset(plan->workspace, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
    return CONV3D_ECUDA;
  return CONV3D_EDEVICE;
}

extern "C" size_t linear_q8_workspace_size(linear_q8_plan_t plan) {
  return plan ? plan->workspace_bytes : 0;
}

extern "C" void linear_q8_destroy(linear_q8_plan_t plan) {
  if (!plan) return;
  {
    DeviceRestore restore;
    if (cudaSetDevice(plan->device) == cudaSuccess) {
      cudaDeviceSynchronize();  // without a workspace too: the runs read the caller's memory
      cudaFree(plan->workspace);
    }
    cudaGetLastError();
  }
  delete plan;
}
