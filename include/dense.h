/*
 * dense.h -- the dense layer and layer norm, forward and backward, for AMD
 * Instinct MI355X (gfx950): the operators of a feed-forward block, beside the
 * INT8 convolution of conv_i8.h.
 *
 *   linear               z = (x w^T) * x_scale[m] * w_scale[n] + bias[n]
 *                        y = act(z) + residual
 *   linear_backward      g = dy * act'(z); dx = g w; dw = g^T x; dbias = sum over rows of g
 *   layer_norm           y = (x - mean) * rstd * weight + bias, rstd = 1 / sqrt(var + eps)
 *   layer_norm_backward  dx, dweight and dbias of it
 *
 * A matrix is a device pointer, its dims and its strides in ELEMENTS; strides
 * must be >= 0 and outputs must not overlap themselves.  The kernels keep no
 * state between calls.  All device work is enqueued on `stream` (a
 * hipStream_t, NULL: the default stream); no entry allocates, waits or clears
 * memory with a runtime call, so every entry can be recorded into a HIP graph.
 * Argument errors are found on the host before any device work.  Results do
 * not depend on the order in which workgroups run: no sum uses atomics.
 *
 * Sums, norms and products accumulate in 32 bits; each output is rounded once
 * (half to even) to its type.  NaN and infinities propagate as in the formulas.
 */
#ifndef DENSE_H
#define DENSE_H

#include "conv_i8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types; DENSE_NONE marks an operand that is absent. */
typedef enum {
    DENSE_NONE = 0,
    DENSE_INT8 = 1, /* CONV_I8_DT_INT8 */
    DENSE_BF16 = 3,
    DENSE_FP16 = 4,
    DENSE_FP32 = 5
} dense_dtype_t;

/* [rows, cols] of `dtype`; element (r, c) at ptr + r*row_stride + c*col_stride.
 * A stride along a dim of size 1 is ignored.  ptr must be aligned to the
 * element size; it may be NULL where rows or cols is 0. */
typedef struct {
    const void *ptr;
    int64_t rows, cols;
    int64_t row_stride, col_stride;
    int64_t dtype;
} dense_mat_t;

/* `n` contiguous elements of `dtype`. */
typedef struct {
    const void *ptr;
    int64_t n;
    int64_t dtype;
} dense_vec_t;

typedef enum {
    DENSE_ACT_NONE = 0,
    DENSE_ACT_RELU = 1,      /* max(z, 0); slope 0 at 0 */
    DENSE_ACT_GELU = 2,      /* z/2 (1 + erf(z / sqrt 2)) */
    DENSE_ACT_GELU_TANH = 3, /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    DENSE_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} dense_act_t;

/* May be added to the activation of dense_linear_backward. */
#define DENSE_WIDE_G 256

/*
 * Dense layer.  x [M, K] and w [N, K] share one type: BF16, FP16 or INT8.
 * INT8 operands are summed exactly in 32-bit integers (K <= 131071,
 * CONV_I8_ERR_RANGE otherwise), then scaled.  y [M, N], preact and residual
 * [M, N] share one type: FP32, or the inputs' own (BF16 or FP16 for INT8
 * inputs).  y, preact and residual have col_stride 1.  residual may be y
 * itself; no other output may overlap an operand.
 */
typedef struct {
    dense_mat_t x, w, y;
    dense_mat_t residual;  /* added after the activation; dtype DENSE_NONE: none */
    dense_mat_t preact;    /* receives z, for the backward pass; dtype DENSE_NONE: not kept */
    dense_vec_t bias;      /* N of BF16, FP16 or FP32; dtype DENSE_NONE: none */
    dense_vec_t x_scale;   /* M of FP32, INT8 inputs only; dtype DENSE_NONE: ones */
    dense_vec_t w_scale;   /* N of FP32, INT8 inputs only; dtype DENSE_NONE: ones */
    int64_t activation;    /* dense_act_t */
} dense_linear_t;

/* Bytes of device workspace, 256-byte aligned, that the call needs: copies of
 * operands the kernels cannot read in place (rows that are not 16-byte aligned
 * or not contiguous) and the partial sums of a split reduction.  Host-only. */
conv_i8_status_t dense_linear_workspace_size(const dense_linear_t *args, size_t *bytes);

/* CONV_I8_ERR_WORKSPACE if `bytes` is less than the size above or the
 * workspace is not 256-byte aligned. */
conv_i8_status_t dense_linear(const dense_linear_t *args, void *workspace, size_t bytes, void *stream);

/* One line that says how the call would run.  Host-only.
 *
 * For tests and measurements, the environment variable CONV_I8_DENSE_TILE names
 * the tile of every product of the dense layer and its gradients ("256x256",
 * "128x128", "64x64", "128x128d") and, after a slash, its split of the inner
 * dimension (1 to 64; the largest that leaves each part four stages, if that is
 * less).  The kernel for a few rows is then not used.  Any other value is
 * CONV_I8_ERR_PARAM. */
conv_i8_status_t dense_linear_plan(const dense_linear_t *args, char *buf, size_t len);

/*
 * Gradients of the dense layer.  All operands BF16, or all FP16.  dy [M, N]
 * and preact [M, N] (the z that dense_linear kept; not needed, and not read,
 * without an activation) give g, which is rounded to the operands' type for
 * the two products (dbias sums the unrounded g): in FP16, a g below 2^-14 has
 * steps of 2^-24, and one below 2^-25 counts as zero.  With DENSE_WIDE_G the
 * products take g as two values of that type, which together have 16 (BF16) or
 * 22 (FP16) bits and no such loss above 2^-36, at twice the products' work.  Any of dx [M, K], dw [N, K]
 * and dbias (N) may be absent; outputs have col_stride 1.  The gradient of
 * the residual is dy itself.
 */
typedef struct {
    dense_mat_t dy, x, w, preact;
    dense_mat_t dx, dw;
    dense_vec_t dbias;
    int64_t activation;
} dense_linear_backward_t;

conv_i8_status_t dense_linear_backward_workspace_size(const dense_linear_backward_t *args, size_t *bytes);
conv_i8_status_t dense_linear_backward(const dense_linear_backward_t *args, void *workspace, size_t bytes,
                                       void *stream);
conv_i8_status_t dense_linear_backward_plan(const dense_linear_backward_t *args, char *buf, size_t len);

/*
 * Layer norm over the columns of x [M, D] (BF16, FP16 or FP32, col_stride 1,
 * D >= 1).  weight and bias: D of x's type.  y [M, D] has x's type, or INT8:
 * then row m holds round(y / s) with s = max |y| / 127 in scale[m] (a row of
 * zeros has scale 0).  mean and rstd (M of FP32) may be absent.
 */
typedef struct {
    dense_mat_t x, y;
    dense_vec_t weight, bias;  /* dtype DENSE_NONE: ones, zeros */
    dense_vec_t mean, rstd;    /* M of FP32; dtype DENSE_NONE: not written */
    dense_vec_t scale;         /* M of FP32, for an INT8 y only */
    double eps;                /* >= 0 */
} dense_layer_norm_t;

conv_i8_status_t dense_layer_norm(const dense_layer_norm_t *args, void *stream);

/*
 * Gradients of layer norm from dy, x (of one type, as above) and the
 * statistics of the forward pass:
 *   xh = (x - mean) rstd; c = dy weight
 *   dx = rstd (c - mean(c) - xh mean(c xh)); dweight = sum over rows of dy xh; dbias = sum over rows of dy
 * dx [M, D], dweight and dbias (D) are of x's type; dweight and dbias may be
 * absent, both or neither.
 */
typedef struct {
    dense_mat_t dy, x, dx;
    dense_vec_t weight;         /* dtype DENSE_NONE: ones */
    dense_vec_t mean, rstd;     /* M of FP32 */
    dense_vec_t dweight, dbias; /* dtype DENSE_NONE: not computed */
} dense_layer_norm_backward_t;

conv_i8_status_t dense_layer_norm_backward_workspace_size(const dense_layer_norm_backward_t *args, size_t *bytes);
conv_i8_status_t dense_layer_norm_backward(const dense_layer_norm_backward_t *args, void *workspace, size_t bytes,
                                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_H */
