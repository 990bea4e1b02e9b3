/*
 * linear_norm: the operators of a transformer block beside the plain fp16 product, on one
 * MI355X (gfx950): a linear layer with its epilogue and its backward pass, and the
 * root-mean-square norm with the residual's addition and its backward pass.
 *
 *   linear_forward      v = a b (* scale_a[i] scale_b[j]) + bias[j]
 *                       pre = v (optional);  out = act(v) + residual
 *   linear_backward     dpre = dc act'(pre);  da = dpre b^T;  db = a^T dpre;
 *                       dbias[j] = sum_i dpre[i][j]
 *   rms_norm_forward    h = x + residual;  rstd[i] = 1 / sqrt(mean_j h[i][j]^2 + eps)
 *                       y = h rstd[i] weight[j], in x's type, or in e4m3 with a scale a row:
 *                       scale[i] = max_j |y[i][j]| / 448 (1 for a row of zeros), y / scale[i]
 *   rms_norm_backward   xh = h rstd[i];  g = dy weight[j]
 *                       dx = rstd[i] (g - xh mean_j(g xh)) + dh;  dweight[j] = sum_i dy xh
 *
 * Sums, statistics and gradients are held in fp32; every output is rounded once (to nearest,
 * ties to even), with one exception: dpre is rounded to the operands' type before it enters
 * the matrix products (their operands are 16 bits wide; beyond f16's range it is infinite).
 * dbias sums the unrounded values.
 *
 * Activations, their lower tails included, and the terms of their slopes are off by a few 2^-23 of
 * their own values around 0, and by up to 2^-15 where exp leaves fp32's range.
 * The norm's squares may leave fp32's range; rstd may not.
 *
 * 8-bit operands: with up to 16 rows (m) or k up to 512 the values are multiplied as f16,
 * exactly.  Beyond, they go through the 8-bit matrix instruction, which rounds inside: measured
 * over random operands, a sum is off by up to 2^-17 of the sum of its products' magnitudes at k
 * = 1000.
 *
 * Activations: none, relu, gelu (0.5 v (1 + erf(v / sqrt 2))), gelu_tanh (the tanh form of it),
 * silu (v / (1 + exp(-v))).  relu's slope at 0 is 0.
 *
 * Matrices are described by a device pointer and a row and a column stride in elements.  a and
 * b may be row- or column-major (one unit stride, any leading dimension, any alignment of
 * their type); 8-bit operands are k-contiguous (a row-major, b column-major) with 16-byte
 * aligned pointers and leading dimensions that are multiples of 16.  All other matrices are
 * row-major with any row stride of at least their row length.  Stride arguments of an axis of
 * extent 1 are ignored.
 *
 * Extents are below 2^31.  A product is refused with GEMM_F16F32_ERR_TOO_LARGE where the rows of
 * a stored panel (64 if k is not the unit-stride axis, else a tile's 64 to 256) times the leading
 * dimension reach 2^31 16-bit elements and it has more rows than the kernels for up to 16 take,
 * or where its tiles need 2^32 threads.
 *
 * Ownership and execution as in gemm_f16f32.h: every pointer is the caller's, nothing is
 * allocated, no state is kept, calls only enqueue kernels on `stream` (a hipStream_t) and may
 * be captured in a HIP graph.  Workspaces are sized by the *_workspace functions; they need no
 * initial contents, and are free for reuse by later work on the same stream.
 *
 * Errors: 0 or a negative GEMM_F16F32_ERR_* code (gemm_f16f32.h); arguments are checked on the
 * host before anything is launched.
 */
#ifndef LINEAR_NORM_H
#define LINEAR_NORM_H

#include <stdint.h>

#include "gemm_f16f32.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { LINEAR_NORM_F16 = 0, LINEAR_NORM_BF16 = 1, LINEAR_NORM_E4M3 = 2 };

enum {
    LINEAR_ACT_NONE = 0,
    LINEAR_ACT_RELU = 1,
    LINEAR_ACT_GELU = 2,
    LINEAR_ACT_GELU_TANH = 3,
    LINEAR_ACT_SILU = 4
};

/* All fields are 8 bytes wide, in this order, so that a caller without this header can pack
 * them as an array of 64-bit integers (pointers and stream handles as addresses). */
typedef struct linear_forward_args {
    int64_t m, n, k;
    int64_t type;             /* of a and b: LINEAR_NORM_F16, _BF16 or _E4M3 */
    int64_t out_type;         /* of bias, residual, out and pre: F16 or BF16; equal to `type`
                                 unless that is E4M3 */
    int64_t activation;       /* LINEAR_ACT_* */
    const void* a;            /* m x k */
    int64_t a_row, a_col;
    const void* b;            /* k x n */
    int64_t b_row, b_col;
    const float* scale_a;     /* E4M3 only: m row scales (NULL: 1) */
    const float* scale_b;     /* E4M3 only: n column scales (NULL: 1) */
    const void* bias;         /* n values, or NULL */
    const void* residual;     /* m x n, or NULL */
    int64_t residual_row;
    void* out;                /* m x n; may be the residual's own memory (same row stride) */
    int64_t out_row;
    void* pre;                /* m x n: the value before the activation, or NULL */
    int64_t pre_row;
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} linear_forward_args;

typedef struct linear_backward_args {
    int64_t m, n, k;
    int64_t type;             /* of every 16-bit matrix: F16 or BF16 */
    int64_t activation;
    const void* dc;           /* m x n */
    int64_t dc_row;
    const void* a;            /* m x k */
    int64_t a_row, a_col;
    const void* b;            /* k x n */
    int64_t b_row, b_col;
    const void* pre;          /* m x n; needed unless activation is LINEAR_ACT_NONE */
    int64_t pre_row;
    void* da;                 /* m x k, or NULL */
    int64_t da_row;
    void* db;                 /* k x n, row- or column-major, or NULL */
    int64_t db_row, db_col;
    void* dbias;              /* n, or NULL */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} linear_backward_args;

typedef struct rms_norm_forward_args {
    int64_t rows, dim;
    int64_t type;             /* of x, weight, residual and h: F16 or BF16 */
    int64_t out_type;         /* of y: equal to `type`, or E4M3 */
    const void* x;            /* rows x dim */
    int64_t x_row;
    const void* residual;     /* rows x dim, or NULL */
    int64_t residual_row;
    const void* weight;       /* dim */
    void* y;                  /* rows x dim */
    int64_t y_row;
    float* scale;             /* E4M3 only: rows */
    void* h;                  /* rows x dim; NULL only without a residual.  May be x's or the
                                 residual's own memory (same row stride) */
    int64_t h_row;
    float* rstd;              /* rows, or NULL */
    double eps;
    void* stream;
} rms_norm_forward_args;

typedef struct rms_norm_backward_args {
    int64_t rows, dim;
    int64_t type;
    const void* dy;           /* rows x dim */
    int64_t dy_row;
    const void* h;            /* rows x dim */
    int64_t h_row;
    const void* weight;       /* dim */
    const float* rstd;        /* rows */
    const void* dh;           /* rows x dim: the gradient that reaches h directly, or NULL */
    int64_t dh_row;
    void* dx;                 /* rows x dim; may be dy's or dh's own memory (same row stride) */
    int64_t dx_row;
    void* dweight;            /* dim, or NULL */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} rms_norm_backward_args;

int linear_forward(const linear_forward_args* args);
int linear_backward(const linear_backward_args* args);
int rms_norm_forward(const rms_norm_forward_args* args);
int rms_norm_backward(const rms_norm_backward_args* args);

/* Bytes of workspace that the call needs (0: none), or a negative error code.  The workspace
 * is 16-byte aligned; workspace, workspace_bytes and stream are not read. */
int64_t linear_forward_workspace(const linear_forward_args* args);
int64_t linear_backward_workspace(const linear_backward_args* args);
int64_t rms_norm_backward_workspace(const rms_norm_backward_args* args);

#ifdef __cplusplus
}
#endif

#endif
