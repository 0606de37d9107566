/*
 * dense.h -- the operators of a feed-forward block and of its training, for AMD
 * Instinct MI355X (gfx950), beside the INT8 convolution of conv_i8.h: the dense
 * layer in 16, 32 and 8 bits, norms, the quantiser, the clipping of gradients.
 *
 *   linear               z = (x w^T) * x_scale[m] * w_scale[n] + bias[n]
 *                        y = act(z) + residual
 *   linear_backward      g = dy * act'(z); dx = g w; dw = g^T x; dbias = sum over rows of g
 *   layer_norm           y = (x - mean) * rstd * weight + bias, rstd = 1 / sqrt(var + eps)
 *   layer_norm_backward  dx, dweight and dbias of it
 *   quantize             x to 8-bit floating point with a scale for each block of 128
 *   dequantize           and back
 *   linear_fp8           the dense layer on such operands
 *   linear_fp8_backward  its gradients
 *   residual_norm        r = alpha x + gate n, n = norm(h) post_weight or h; y = norm(r) weight + bias
 *   residual_norm_backward its gradients
 *   clip_grads           many gradients scaled so that their norm together stays within a limit
 *
 * A matrix is a device pointer, its dims and its strides in ELEMENTS; strides
 * must be >= 0 and outputs must not overlap themselves.  The kernels keep no
 * state between calls.  All device work is enqueued on `stream` (a
 * hipStream_t, NULL: the default stream); no entry allocates, waits or clears
 * memory with a runtime call, so every entry can be recorded into a HIP graph.
 * Argument errors are found on the host before any device work.  Results do
 * not depend on the order in which workgroups run: no sum uses atomics.
 *
 * Sums, norms and products accumulate in 32 bits, the norm of many gradients in
 * 64 (what 8-bit products lose before that: see dense_linear_fp8); each output is
 * rounded once (half to even) to its type.  NaN and infinities propagate as in the formulas.
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
    DENSE_FP32 = 5,
    DENSE_E4M3 = 6, /* 8-bit floating point: up to 448, NaN, no infinities */
    DENSE_E5M2 = 7, /* up to 57344, infinities and NaN */
    DENSE_E8M0 = 8  /* a scale 2^(byte - 127); byte 255 is NaN */
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
 * zeros has scale 0).  mean and rstd (M of FP32) may be absent.  Squares are summed
 * in 32 bits: a row whose squared distances from its mean add up to 2^128 or more
 * has rstd 0 and becomes its bias.
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

/*
 * Rows of 8-bit floating point.  x [M, K] (BF16, FP16 or FP32, col_stride 1)
 * becomes q [M, K] (E4M3 or E5M2) with a scale for each block: 128 values of a
 * row (scale [M, ceil(K/128)]) or 128 x 128 values (scale [ceil(M/128),
 * ceil(K/128)]); the blocks at the ends of rows and columns may have fewer.  A
 * block's scale is 2^e, e the least exponent (at least -127) with which its
 * largest magnitude times 2^-e does not exceed the type's largest value;
 * q = x 2^-e, rounded half to even.  Dividing by such a scale is exact, so q is
 * the rounding of x itself.  Values that are not finite become NaN and do not
 * count for the scale.
 *
 * qt [K, M] and scale_t ([K, ceil(M/128)], or by tiles) are the same of the
 * transpose of x, in one pass over it.  q with scale, or qt with scale_t, may be
 * absent, not both.  One type for both.
 */
typedef struct {
    dense_mat_t x;
    dense_mat_t q, scale;      /* dtype DENSE_NONE: not written */
    dense_mat_t qt, scale_t;   /* dtype DENSE_NONE: not written */
} dense_quantize_t;

conv_i8_status_t dense_quantize(const dense_quantize_t *args, void *stream);

/* x = q 2^e, rounded to x's type (BF16, FP16 or FP32): exact where the value is in
 * the type's range.  q and scale as above, both with col_stride 1. */
typedef struct {
    dense_mat_t q, scale, x;
} dense_dequantize_t;

conv_i8_status_t dense_dequantize(const dense_dequantize_t *args, void *stream);

/*
 * Dense layer on such operands: x [M, K] (E4M3 or E5M2) with scales for blocks
 * of a row, w [N, K] (E4M3) with scales for blocks of a row or tiles:
 *   z = sum over k of (x x_scale)(w w_scale) + bias; y = act(z) + residual
 * Scales have col_stride 1.  y, preact and residual share one type: BF16, FP16
 * or FP32; their strides, bias and the activation as in dense_linear.
 *
 * For a 16-bit y of more than 32 rows (of more than 16 where w has more than 4096, of
 * any number where x or w cannot be read in place) the matrix unit takes the operands as they
 * are: it adds the products of eight consecutive k at a time, cutting off what is
 * more than 13 bits below the largest of them, and sums those in 32 bits.  For a
 * 32-bit y, and for fewer rows, the operands are taken to BF16 first, which holds
 * them exactly (magnitudes of 2^-126 and more), and all sums are those of 32 bits;
 * x and w then have col_stride 1.
 */
typedef struct {
    dense_mat_t x, w, y;
    dense_mat_t residual, preact;  /* dtype DENSE_NONE: none */
    dense_mat_t x_scale;           /* [M, ceil(K/128)] of E8M0 */
    dense_mat_t w_scale;           /* [N, ceil(K/128)] or [ceil(N/128), ceil(K/128)] of E8M0 */
    dense_vec_t bias;
    int64_t activation;
} dense_linear_fp8_t;

conv_i8_status_t dense_linear_fp8_workspace_size(const dense_linear_fp8_t *args, size_t *bytes);
conv_i8_status_t dense_linear_fp8(const dense_linear_fp8_t *args, void *workspace, size_t bytes, void *stream);
conv_i8_status_t dense_linear_fp8_plan(const dense_linear_fp8_t *args, char *buf, size_t len);

/*
 * Its gradients, from the operands transposed: xt [K, M] and wt [K, N] (E4M3,
 * scales for blocks of a row or tiles).  dy and preact [M, N] (one type, BF16 or
 * FP16; preact is not read without an activation) give g = dy act'(preact),
 * which is quantised twice, to g_dtype (DENSE_E4M3 or DENSE_E5M2) with scales for
 * blocks of a row: as it is for dx = g w, transposed for dw = g^T x.  dbias sums
 * the unrounded g.  Any of dx [M, K], dw [N, K] and dbias (N), of dy's type, may
 * be absent; xt (wt) is not needed without dw (dx).
 */
typedef struct {
    dense_mat_t dy, preact;
    dense_mat_t xt, xt_scale, wt, wt_scale;
    dense_mat_t dx, dw;
    dense_vec_t dbias;
    int64_t activation;
    int64_t g_dtype;
} dense_linear_fp8_backward_t;

conv_i8_status_t dense_linear_fp8_backward_workspace_size(const dense_linear_fp8_backward_t *args, size_t *bytes);
conv_i8_status_t dense_linear_fp8_backward(const dense_linear_fp8_backward_t *args, void *workspace, size_t bytes,
                                           void *stream);
conv_i8_status_t dense_linear_fp8_backward_plan(const dense_linear_fp8_backward_t *args, char *buf, size_t len);

/*
 * The norm between two blocks, fused with the residual connection:
 *   n = norm(h) post_weight, or h without it
 *   r = alpha x + gate n, or x without h;  rounded to x's type
 *   y = norm(r) weight + bias
 * norm(v) = (v - mean) rstd, rstd = 1 / sqrt(mean((v - mean)^2) + eps); with
 * kind DENSE_RMS_NORM mean stands for 0.  x, h, r and y are [M, D], all matrices
 * and vectors of one type (BF16, FP16 or FP32), col_stride 1, D >= 1.  gate
 * [G, D]: G divides M, and each of its rows is that of M / G consecutive rows.
 * Without h, gate, post_weight and r are absent as well.  r may be x or h
 * itself.  y may be E4M3, with a scale for each 128 of a row in y_scale
 * [M, ceil(D/128)], as dense_quantize gives of the unrounded y.
 *
 * Squares are summed in 32 bits, where they have to stay below 2^128 (a deviation of
 * 2^64 / sqrt(D), which FP16 does not reach): beyond, and with an infinity or NaN in it, a
 * row's rstd is NaN and with it the normed row.  Squares below 2^-126 lose digits, which
 * shows with an eps below 1e-22 only; eps is taken in 32 bits.
 */
typedef enum { DENSE_LAYER_NORM = 0, DENSE_RMS_NORM = 1 } dense_norm_t;

typedef struct {
    dense_mat_t x, h, r, y;
    dense_mat_t gate;               /* dtype DENSE_NONE: ones */
    dense_mat_t y_scale;            /* E8M0, for an E4M3 y only */
    dense_vec_t post_weight;        /* dtype DENSE_NONE: no norm of h */
    dense_vec_t weight, bias;       /* dtype DENSE_NONE: ones, zeros */
    dense_vec_t mean, rstd;         /* of r, M of FP32; dtype DENSE_NONE: not written */
    dense_vec_t post_mean, post_rstd; /* of h */
    double alpha, eps;              /* eps >= 0 */
    int64_t kind;
} dense_residual_norm_t;

conv_i8_status_t dense_residual_norm(const dense_residual_norm_t *args, void *stream);

/*
 * Its gradients from those of r (dr; dtype DENSE_NONE: zero) and y (dy), r, h and
 * the statistics of the forward pass (means are not read with DENSE_RMS_NORM):
 *   t = dr + the gradient of norm(r) weight by r, applied to dy
 *   dx = alpha t; dgate = sum over a gate row's rows of t n
 *   dh = the gradient of n by h, applied to gate t
 *   dweight = sum over rows of dy norm(r); dbias = sum over rows of dy;
 *   dpost_weight = sum over rows of gate t norm(h)
 * Without h, dh, dgate and dpost_weight are absent; h is not read without gate
 * and post_weight.  dweight, dbias, dgate and dpost_weight are absent together
 * with what they are the gradients of, or each where it is not wanted.
 */
typedef struct {
    dense_mat_t dr, dy, r, h, dx, dh;
    dense_mat_t gate, dgate;
    dense_vec_t weight, post_weight;
    dense_vec_t mean, rstd, post_mean, post_rstd;
    dense_vec_t dweight, dbias, dpost_weight;
    double alpha;
    int64_t kind;
} dense_residual_norm_backward_t;

conv_i8_status_t dense_residual_norm_backward_workspace_size(const dense_residual_norm_backward_t *args, size_t *bytes);
conv_i8_status_t dense_residual_norm_backward(const dense_residual_norm_backward_t *args, void *workspace, size_t bytes,
                                              void *stream);

/*
 * norm = sqrt(sum of squares of all elements of all tensors), summed in 64 bits;
 * out = in min(1, max_norm / norm), a product of 64 bits rounded to 32 and to the
 * type.  Where an element is infinite or NaN, `norm` is too and all values stay as
 * they are.  Finite elements always follow the formula, also where their norm is
 * beyond what 32 bits hold and `norm` reads as infinity.  in and out: `count`
 * vectors of BF16, FP16 or FP32; an out is its in itself, or of the same type and
 * size and overlaps no other vector.  No two vectors of `in` overlap where they are
 * written, and `norm` lies in none of them.
 */
typedef struct {
    const dense_vec_t *in, *out;
    int64_t count;
    double max_norm;   /* >= 0, not NaN */
    float *norm;       /* device memory */
} dense_clip_grads_t;

conv_i8_status_t dense_clip_grads_workspace_size(const dense_clip_grads_t *args, size_t *bytes);
conv_i8_status_t dense_clip_grads(const dense_clip_grads_t *args, void *workspace, size_t bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_H */
