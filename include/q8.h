/*
 * q8.h -- C ABI of the quantised transformer path for one NVIDIA GB300 (sm_103a): products of 8-bit
 * codes with a scale for each token and each output channel, and the two operators that write such
 * codes, the root-mean-square norm (with the residual's addition) and the gated activation. Exported
 * by the same library as conv3d_fp8.h and with the same conventions:
 *   - Every entry point returns a conv3d_status; conv3d_fp8_strerror names it. Argument errors are
 *     reported before anything is launched.
 *   - Device pointers are plain CUDA addresses on the plan's or the arguments' device, which must be
 *     the current one; the caller owns them. `stream` is a cudaStream_t as void* (NULL: the legacy
 *     default stream). Everything a call reads is to be ready, and stay unchanged, in stream order.
 *   - Nothing here synchronises except linear_q8_plan, linear_q8_check and linear_q8_destroy; a run
 *     allocates nothing and can be captured in a CUDA graph.
 *
 * Codes. A row of values v is held as codes q and one fp32 scale s, v ~ q * s:
 *   s = amax / T with amax = max |v| over the row and T = 127 (int8) or 448 (e4m3); 1 if amax == 0;
 *   q = v / s rounded to the nearest code, ties to even (int8 codes lie in [-127, 127]).
 * A row whose values include a NaN or an infinity has the scale NaN and codes 0, so whatever is made
 * of that row is NaN and no other row is touched; so has a row of the norm whose sum of squares, or a
 * product h * weight, overflows fp32.
 *
 * Rows. Every matrix is row-major with a pitch (the distance between rows) in ELEMENTS; the
 * elements of a row are contiguous. Elements between a row's end and the next row's start are
 * neither written nor used; a matrix of one row has no use for its pitch.
 */
#ifndef Q8_H
#define Q8_H

#include <stddef.h>

#include "conv3d_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { Q8_F32 = 1, Q8_BF16 = 2, Q8_F16 = 3 } q8_value_type;
typedef enum { Q8_INT8 = 1, Q8_E4M3 = 2 } q8_code_type;

/* The widest row of rmsnorm_q8_run and silu_mul_q8_run. */
#define Q8_MAX_COLS 32768

/*
 * Root-mean-square norm with the residual's addition and an 8-bit output, for each row:
 *   h = x + residual (in fp32; h = x without a residual), residual_out = h rounded to value_type,
 *   y = h / sqrt(sum(h^2) / cols + eps) * weight, q and scale = the codes of y.
 * y is taken from the unrounded h. residual_out may be x or residual itself (same pitch); apart
 * from that no output may overlap an input. With an eps below 2^-120 (0, mostly) the squares of small
 * values would underflow beside it: their sum is then taken of lifted values, by a second launch.
 * Errors: EINVAL (NULL x, weight, q or scale with rows > 0; a residual without residual_out or the
 * reverse; rows < 0, cols < 1, a pitch below cols, an unknown type, a pointer that is not aligned to
 * its element, eps negative or not finite, `device` not the current device), EUNSUPPORTED
 * (cols > Q8_MAX_COLS, rows of 2^31 or more, a device that is not sm_103), ECUDA. rows == 0 does
 * nothing.
 */
typedef struct {
    const void *x;              /* [rows][cols] value_type */
    const void *residual;       /* [rows][cols] value_type, or NULL */
    const void *weight;         /* [cols] weight_type */
    void *residual_out;         /* [rows][cols] value_type; NULL exactly when residual is */
    void *q;                    /* [rows][cols] codes */
    float *scale;               /* [rows] */
    long long x_pitch, residual_pitch, residual_out_pitch, q_pitch;
    long long rows, cols;
    void *stream;
    int value_type, weight_type, code_type, device;
    float eps;
    int reserved;               /* 0 */
} rmsnorm_q8_args;

conv3d_status rmsnorm_q8_run(const rmsnorm_q8_args *args);

/*
 * Gated activation with an 8-bit output, for each row: y = silu(gate) * up, silu(g) = g / (1 +
 * exp(-g)), in fp32; q and scale = the codes of y. y's relative error is below (|g| + 12) * 2^-23;
 * for gates below -87.3, whose exponential is a subnormal number, 2^-148 * exp(-g) more, and from
 * about -104 on silu is 0. gate and up may be the two halves of one matrix (the same pitch). No
 * output may overlap an input. Errors: as rmsnorm_q8_run.
 */
typedef struct {
    const void *gate;           /* [rows][cols] value_type */
    const void *up;             /* [rows][cols] value_type */
    void *q;                    /* [rows][cols] codes */
    float *scale;               /* [rows] */
    long long gate_pitch, up_pitch, q_pitch;
    long long rows, cols;
    void *stream;
    int value_type, code_type, device;
    int reserved;               /* 0 */
} silu_mul_q8_args;

conv3d_status silu_mul_q8_run(const silu_mul_q8_args *args);

/*
 * The product of 8-bit codes, with a scale for each token (row of x) and each channel (row of w):
 *   y[m][n] = scale_x[m] * scale_w[n] * sum_k x[m][k] * w[n][k] + bias[n]
 * x and w are both int8 or both e4m3. The sum is kept in 32 bits: int8 products are summed exactly
 * as long as every partial sum stays within 2^24 in magnitude (always, for K <= 1024); beyond that,
 * and for e4m3, each addition rounds by at most 2^-23 of the largest operand. (int8 codes of both
 * signs stay exact: K = 32768, sums to 4e6. Codes of one sign: random ones from 0 to 127 err by 3e-8 to
 * 6e-8 of the sum for K up to 16384 and 4e-6 for 32768, from 100 to 127 by 9e-7 for K = 8192, 3.4e-6 for
 * 16384 and 1.5e-5 for 32768, downwards.) The scaling and the bias are fp32, y is rounded once.
 */
typedef struct linear_q8_plan_s *linear_q8_plan_t; /* opaque, owned by the library */

/*
 * Plan products of up to max_rows tokens by an [N][K] weight on `device`. Allocates the workspace: a
 * status word and, for int8 codes, x as f16 (2 * max_rows * K bytes); nothing where max_rows and the
 * sizes leave all runs to the kernel for few tokens.
 * Errors: EINVAL (a size below 1, an unknown code type), EUNSUPPORTED (sizes of 2^30 or more, a
 * device that is not sm_103), ENOMEM, ECUDA. On error *plan is set to NULL.
 */
conv3d_status linear_q8_plan(linear_q8_plan_t *plan, long long max_rows, long long N, long long K,
                             int code_type, int device);

/* Optional planning knobs. Zero-initialise and set only what you need; none changes what is
 * computed beyond the order of a sum's additions. */
typedef struct {
    int kernel;          /* 0: the library chooses; 1: the kernel for few tokens (EUNSUPPORTED for
                            max_rows above 32 (int8) or 16 (e4m3)); 2: the tensor-core kernel for
                            any number */
    int block_t;         /* 0: the library chooses; else the tokens of a tensor-core tile, a multiple
                            of 32 up to 256 (int8: 192), and less than the run's rows + 32 */
    int splits;          /* 0: the library chooses; 1 to 4: slices of K (no more than K has blocks of
                            256 codes; with more than one, all tiles must be held by the device at
                            once) */
    int max_ctas;        /* 0: all the device holds; else an upper bound on the grid, which is one pair
                            of CTAs at least */
    int wait_timeout_ms; /* 0: 2000 ms; a bounded wait inside a kernel gives up after this long */
    int debug_flags;     /* test-only: bit 0 makes the loader skip its first copy, so the waits on it
                            must run out (exercises the error path without faulting anything) */
} linear_q8_options;

/* As linear_q8_plan, with planning knobs (opts may be NULL). Where the options leave no tiling for a
 * run's rows, that run returns EUNSUPPORTED. */
conv3d_status linear_q8_plan_ex(linear_q8_plan_t *plan, long long max_rows, long long N, long long K,
                                int code_type, int device, const linear_q8_options *opts);

/*
 * One product, asynchronously on `stream`. A plan's workspace is shared by its runs: at most one run
 * of a plan may be in flight at a time (one plan for each concurrent stream). Every element of y is
 * written exactly once and nothing outside it. A row or channel whose scale is NaN is NaN in y.
 * Rows of codes on 32-byte boundaries are read fastest. Errors: EINVAL (a NULL pointer with rows > 0,
 * rows < 0 or above max_rows, N, K or a code type other than the plan's, a pitch too small, x or w not
 * 16-byte aligned or with a pitch that is not a multiple of 16, an unknown type, a pointer that
 * is not aligned to its element, the wrong current device), ECUDA. Device errors are reported later,
 * by linear_q8_check. rows == 0 does nothing.
 */
typedef struct {
    const void *x;              /* [rows][K] codes */
    const float *scale_x;       /* [rows] */
    const void *w;              /* [N][K] codes */
    const float *scale_w;       /* [N] */
    const void *bias;           /* [N] bias_type, or NULL */
    void *y;                    /* [rows][N] y_type */
    long long x_pitch, w_pitch, y_pitch;
    long long rows, N, K;       /* N and K must equal the plan's */
    void *stream;
    int y_type, bias_type;      /* bias_type is ignored without a bias */
    int code_type;              /* must equal the plan's */
    int reserved;               /* 0 */
} linear_q8_args;

conv3d_status linear_q8_run(linear_q8_plan_t plan, const linear_q8_args *args);

/* Synchronise the device, then report and clear the plan's device status: OK, or EDEVICE if one of a
 * kernel's bounded waits ran out (its output is then incomplete). */
conv3d_status linear_q8_check(linear_q8_plan_t plan);

/* Device bytes the plan holds; 0 for NULL. */
size_t linear_q8_workspace_size(linear_q8_plan_t plan);

/* Wait for the device and free the plan (NULL is allowed). */
void linear_q8_destroy(linear_q8_plan_t plan);

#ifdef __cplusplus
}
#endif
#endif /* Q8_H */
