/*
 * linear_norm: the operators of a transformer block beside the plain fp16 product, on one
 * MI355X (gfx950): a linear layer with its epilogue and its backward pass, the root-mean-square
 * norm and the layer norm with the residual's addition and their backward passes, and activations
 * in 8 bits: as operands of the layer, and as what is kept for its backward pass.
 *
 *   linear_forward      v = a b (* scale_a[i] scale_b[j]) + bias[j]
 *                       pre = v (optional);  out = act(v) + residual
 *   linear_backward     dpre = dc act'(pre);  da = dpre b^T;  db = a^T dpre;
 *                       dbias[j] = sum_i dpre[i][j]
 *   rms_norm_forward    h = x + residual;  rstd[i] = 1 / sqrt(mean_j h[i][j]^2 + eps)
 *                       y = h rstd[i] weight[j], in x's type, or in e4m3 with a scale a row:
 *                       scale[i] = max_j |y[i][j]| / 448 (1 for a row of zeros), y / scale[i];
 *                       or in int8 in the same way with 127 in the place of 448
 *   rms_norm_backward   xh = h rstd[i];  g = dy weight[j]
 *                       dx = rstd[i] (g - xh mean_j(g xh)) + dh;  dweight[j] = sum_i dy xh
 *   layer_norm_forward  h = x + residual;  mean[i] = mean_j h[i][j]
 *                       rstd[i] = 1 / sqrt(mean_j (h[i][j] - mean[i])^2 + eps)
 *                       y = (h - mean[i]) rstd[i] weight[j] + bias[j], in the types of the norm
 *   layer_norm_backward xh = (h - mean[i]) rstd[i];  g = dy weight[j]
 *                       dx = rstd[i] (g - mean_j(g) - xh mean_j(g xh)) + dh
 *                       dweight[j] = sum_i dy xh;  dbias[j] = sum_i dy
 *   quantize_rows       scale[i] as the norm's 8-bit results have it, values = x / scale[i]
 *   pack8               each row in blocks of 32 columns, with a power of two for each:
 *                       scale = 2^(f - 6), f = floor(log2(max |x|)) over the block, but not below
 *                       2^-24 (f16) or 2^-120 (bf16); values = x / scale, to the nearest integer
 *                       (ties to even), at most 127 in magnitude.  Integers times scales are values
 *                       of the 16-bit type.  A block that holds an infinity or a NaN has scale NaN,
 *                       and NaN for its slopes, relu's too
 *   unpack8             y = act(values scale)
 *   linear_forward_packed    linear_forward, with pre in 8 bits as pack8 would make it of the
 *                       unrounded values; with relu, whose slope goes by the sign, a positive value is
 *                       1 scale at least (pack8 takes one of up to half a scale to 0, slope 0)
 *   linear_backward_packed   linear_backward, with a, pre or both in 8 bits.  With a_activation, a
 *                       holds the values before that activation: the layer's input is act(a),
 *                       rounded to the 16-bit type, and da the gradient of that
 *
 * Sums, statistics and gradients are held in fp32; every output is rounded once (to nearest,
 * ties to even), with one exception: dpre is rounded to the operands' type before it enters
 * the matrix products (their operands are 16 bits wide; beyond f16's range it is infinite).
 * dbias sums the unrounded values.
 *
 * Activations, their lower tails included, and the terms of their slopes are off by a few 2^-23 of
 * their own values around 0, and by up to 2^-15 where exp leaves fp32's range.
 * The norms' squares may leave fp32's range; rstd may not, nor a layer norm's differences from the
 * mean.  int8 results cannot hold a NaN: a row with a NaN or an infinity has scale NaN.
 *
 * int8 operands are summed exactly in 32-bit integers, which bounds k by 131071, and the sum is
 * rounded to fp32 before it is scaled.
 *
 * e4m3 operands: with up to 16 rows (m) or k up to 512 the values are multiplied as f16, exactly.
 * Beyond, they may go through the 8-bit matrix instruction, which rounds inside: measured over random
 * operands, a sum is off by up to 2^-17 of the sum of its products' magnitudes at k = 1000.  (Where a
 * result of at most 16 columns, or a sliver of as many, is a pass over a, its values are multiplied
 * as f16 too; that goes by an estimate of the time, and is no part of this contract.)
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

enum { LINEAR_NORM_F16 = 0, LINEAR_NORM_BF16 = 1, LINEAR_NORM_E4M3 = 2, LINEAR_NORM_I8 = 8 };

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
    int64_t type;             /* of a and b: LINEAR_NORM_F16, _BF16, _E4M3 or _I8 */
    int64_t out_type;         /* of bias, residual, out and pre: F16 or BF16; equal to `type`
                                 unless that is E4M3 or I8 */
    int64_t activation;       /* LINEAR_ACT_* */
    const void* a;            /* m x k */
    int64_t a_row, a_col;
    const void* b;            /* k x n */
    int64_t b_row, b_col;
    const float* scale_a;     /* E4M3 and I8 only: m row scales (NULL: 1) */
    const float* scale_b;     /* E4M3 and I8 only: n column scales (NULL: 1) */
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
    int64_t out_type;         /* of y: equal to `type`, E4M3 or I8 */
    const void* x;            /* rows x dim */
    int64_t x_row;
    const void* residual;     /* rows x dim, or NULL */
    int64_t residual_row;
    const void* weight;       /* dim */
    void* y;                  /* rows x dim */
    int64_t y_row;
    float* scale;             /* E4M3 and I8 only: rows */
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

typedef struct layer_norm_forward_args {
    int64_t rows, dim;
    int64_t type;             /* of x, weight, bias, residual and h: F16 or BF16 */
    int64_t out_type;         /* of y: equal to `type`, E4M3 or I8 */
    const void* x;            /* rows x dim */
    int64_t x_row;
    const void* residual;     /* rows x dim, or NULL */
    int64_t residual_row;
    const void* weight;       /* dim */
    const void* bias;         /* dim, or NULL */
    void* y;                  /* rows x dim */
    int64_t y_row;
    float* scale;             /* E4M3 and I8 only: rows */
    void* h;                  /* rows x dim; NULL only without a residual.  May be x's or the
                                 residual's own memory (same row stride) */
    int64_t h_row;
    float* mean;              /* rows, or NULL */
    float* rstd;              /* rows, or NULL */
    double eps;
    void* stream;
} layer_norm_forward_args;

typedef struct layer_norm_backward_args {
    int64_t rows, dim;
    int64_t type;
    const void* dy;           /* rows x dim */
    int64_t dy_row;
    const void* h;            /* rows x dim */
    int64_t h_row;
    const void* weight;       /* dim */
    const float* mean;        /* rows */
    const float* rstd;        /* rows */
    const void* dh;           /* rows x dim: the gradient that reaches h directly, or NULL */
    int64_t dh_row;
    void* dx;                 /* rows x dim; may be dy's or dh's own memory (same row stride) */
    int64_t dx_row;
    void* dweight;            /* dim, or NULL */
    void* dbias;              /* dim, or NULL */
    void* workspace;
    int64_t workspace_bytes;
    void* stream;
} layer_norm_backward_args;

typedef struct quantize_rows_args {
    int64_t rows, dim;
    int64_t type;             /* of x: F16 or BF16 */
    int64_t out_type;         /* of values: E4M3 or I8 */
    const void* x;            /* rows x dim */
    int64_t x_row;
    void* values;             /* rows x dim */
    int64_t values_row;
    float* scale;             /* rows */
    void* stream;
} quantize_rows_args;

/* A rows x dim matrix in 8 bits: integers, and for each 32 neighbours of a row (the last block may
 * hold fewer) the byte b of their scale 2^(b - 127); 255 is NaN.  Both row-major, any row stride
 * of at least the row length, any alignment. */
typedef struct packed8_matrix {
    void* values;             /* rows x dim int8 */
    int64_t values_row;
    void* scale;              /* rows x ceil(dim / 32) bytes */
    int64_t scale_row;
} packed8_matrix;

typedef struct pack8_args {
    int64_t rows, dim;
    int64_t type;             /* of x: F16 or BF16 */
    const void* x;            /* rows x dim */
    int64_t x_row;
    packed8_matrix out;
    void* stream;
} pack8_args;

typedef struct unpack8_args {
    int64_t rows, dim;
    int64_t type;             /* of y: F16 or BF16 */
    int64_t activation;       /* LINEAR_ACT_* */
    packed8_matrix in;
    void* y;                  /* rows x dim */
    int64_t y_row;
    void* stream;
} unpack8_args;

/* What linear_backward_packed reads in 8 bits: a (m x k) in the place of linear_backward_args.a,
 * pre (m x n) in the place of its pre; the field there is then NULL.  Values of NULL: given there,
 * in 16 bits. */
typedef struct linear_kept {
    packed8_matrix a;
    int64_t a_activation;     /* LINEAR_ACT_*; NONE unless a is given here or empty (m or k 0) */
    packed8_matrix pre;
} linear_kept;

int linear_forward(const linear_forward_args* args);
int linear_backward(const linear_backward_args* args);
int rms_norm_forward(const rms_norm_forward_args* args);
int rms_norm_backward(const rms_norm_backward_args* args);
int layer_norm_forward(const layer_norm_forward_args* args);
int layer_norm_backward(const layer_norm_backward_args* args);
int quantize_rows(const quantize_rows_args* args);
int pack8(const pack8_args* args);
int unpack8(const unpack8_args* args);
/* args->pre is NULL; pre NULL: linear_forward */
int linear_forward_packed(const linear_forward_args* args, const packed8_matrix* pre);
/* kept NULL: linear_backward */
int linear_backward_packed(const linear_backward_args* args, const linear_kept* kept);

/* Bytes of workspace that the call needs (0: none), or a negative error code.  The workspace
 * is 16-byte aligned; workspace, workspace_bytes and stream are not read.  Of pointers it counts
 * which are NULL, and in layer_norm_backward whether dx is dy. */
int64_t linear_forward_workspace(const linear_forward_args* args);
int64_t linear_backward_workspace(const linear_backward_args* args);
int64_t rms_norm_backward_workspace(const rms_norm_backward_args* args);
int64_t layer_norm_backward_workspace(const layer_norm_backward_args* args);
int64_t linear_forward_packed_workspace(const linear_forward_args* args, const packed8_matrix* pre);
int64_t linear_backward_packed_workspace(const linear_backward_args* args, const linear_kept* kept);

#ifdef __cplusplus
}
#endif

#endif
