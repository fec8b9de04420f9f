// q8_api.cu -- the C ABI declared in include/q8.h: validation, planning and launch.
#include <cmath>
#include <new>

#include "q8_internal.h"

using namespace c3d;

struct linear_q8_plan_s {
  int device = -1;
  int code_type = 0;
  long long max_rows = 0, N = 0, K = 0;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
};

namespace {

bool value_type_ok(int t) { return t == Q8_F32 || t == Q8_BF16 || t == Q8_F16; }
bool code_type_ok(int t) { return t == Q8_INT8 || t == Q8_E4M3; }
int value_bytes(int t) { return t == Q8_F32 ? 4 : 2; }
long long round_up(long long a, long long b) { return (a + b - 1) / b * b; }
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Whether `device` is the current device and an sm_103.
conv3d_status check_device(int device) {
  int cur = -1, major = 0, minor = 0;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  if (cur != device) return CONV3D_EINVAL;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, cur) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, cur) != cudaSuccess) {
    cudaGetLastError();
    return CONV3D_ECUDA;
  }
  return major == 10 && minor == 3 ? CONV3D_OK : CONV3D_EUNSUPPORTED;
}

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
    if (!matrix_ok(a->x, vb, a->rows, a->x_pitch, a->cols) || !matrix_ok(a->q, 1, a->rows, a->q_pitch, a->cols) ||
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
  p.eps = a->eps;
  return launch_rmsnorm_q8(p, a->value_type, a->weight_type, a->code_type,
                           static_cast<cudaStream_t>(a->stream)) == cudaSuccess
             ? CONV3D_OK
             : CONV3D_ECUDA;
}

extern "C" conv3d_status silu_mul_q8_run(const silu_mul_q8_args* a) {
  if (!a) return CONV3D_EINVAL;
  conv3d_status st = check_rows(a->rows, a->cols, a->value_type, a->code_type);
  if (st != CONV3D_OK) return st;
  const int vb = value_bytes(a->value_type);
  if (a->rows > 0 &&
      (!matrix_ok(a->gate, vb, a->rows, a->gate_pitch, a->cols) ||
       !matrix_ok(a->up, vb, a->rows, a->up_pitch, a->cols) || !matrix_ok(a->q, 1, a->rows, a->q_pitch, a->cols) ||
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
  return launch_silu_mul_q8(p, a->value_type, a->code_type,
                            static_cast<cudaStream_t>(a->stream)) == cudaSuccess
             ? CONV3D_OK
             : CONV3D_ECUDA;
}

extern "C" conv3d_status linear_q8_plan(linear_q8_plan_t* plan, long long max_rows, long long N,
                                        long long K, int code_type, int device) {
  if (!plan) return CONV3D_EINVAL;
  *plan = nullptr;
  if (max_rows < 1 || N < 1 || K < 1 || !code_type_ok(code_type)) return CONV3D_EINVAL;
  if (max_rows >= (1LL << 30) || N >= (1LL << 30) || K >= (1LL << 30)) return CONV3D_EUNSUPPORTED;
  const conv3d_status st = check_device(device);
  if (st != CONV3D_OK) return st;
  linear_q8_plan_s* pl = new (std::nothrow) linear_q8_plan_s();
  if (!pl) return CONV3D_ENOMEM;
  pl->device = device;
  pl->code_type = code_type;
  pl->max_rows = max_rows;
  pl->N = N;
  pl->K = K;
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
    if (!matrix_ok(a->x, 16, a->rows, a->x_pitch, plan->K) || !matrix_ok(a->w, 16, plan->N, a->w_pitch, plan->K) ||
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
  return launch_linear_q8(p, plan->code_type, static_cast<cudaStream_t>(a->stream)) == cudaSuccess
             ? CONV3D_OK
             : CONV3D_ECUDA;
}

extern "C" conv3d_status linear_q8_check(linear_q8_plan_t plan) {
  if (!plan) return CONV3D_EINVAL;
  return cudaDeviceSynchronize() == cudaSuccess ? CONV3D_OK : CONV3D_ECUDA;
}

extern "C" size_t linear_q8_workspace_size(linear_q8_plan_t plan) {
  return plan ? plan->workspace_bytes : 0;
}

extern "C" void linear_q8_destroy(linear_q8_plan_t plan) {
  delete plan;
}
