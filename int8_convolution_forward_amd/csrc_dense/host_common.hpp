// Argument checks shared by the C entries.
#pragma once

#include <stdint.h>

#include "dense.h"

namespace dense {

inline bool is_float(int64_t dt) { return dt == DENSE_BF16 || dt == DENSE_FP16 || dt == DENSE_FP32; }
inline bool is_half(int64_t dt) { return dt == DENSE_BF16 || dt == DENSE_FP16; }

inline int64_t size_of(int64_t dt)
{
    return dt == DENSE_INT8 ? 1 : dt == DENSE_FP32 ? 4 : is_half(dt) ? 2 : 0;
}

// Largest dim: indexes along it then stay within 32 bits.
constexpr int64_t kMaxDim = (int64_t)1 << 30;
// A launch has fewer than 2^32 threads.
inline bool launch_fits(int64_t wgs, int threads) { return wgs < ((int64_t)1 << 32) / threads; }
// Largest stride: a byte offset of kMaxDim rows then stays within 63 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 30;

// dims and strides of a matrix; strides along dims of size 1 become 1 (columns) or the packed pitch (rows)
inline conv_i8_status_t check_mat(dense_mat_t *m, bool output)
{
    if (size_of(m->dtype) == 0)
        return CONV_I8_ERR_DTYPE;
    if (m->rows < 0 || m->cols < 0)
        return CONV_I8_ERR_DIMS;
    if (m->rows > kMaxDim || m->cols > kMaxDim)
        return CONV_I8_ERR_UNSUPPORTED;
    if (m->cols <= 1)
        m->col_stride = 1;
    if (m->rows <= 1)
        m->row_stride = m->cols * (m->col_stride > 0 ? m->col_stride : 1);
    if (m->row_stride < 0 || m->col_stride < 0)
        return CONV_I8_ERR_STRIDES;
    if (m->row_stride > kMaxStride || m->col_stride > kMaxStride)
        return CONV_I8_ERR_UNSUPPORTED;
    if (output && (m->col_stride != 1 || (m->rows > 1 && m->row_stride < m->cols)))
        return CONV_I8_ERR_STRIDES;
    if (m->rows > 0 && m->cols > 0) {
        if (!m->ptr)
            return CONV_I8_ERR_NULL;
        if ((uintptr_t)m->ptr % size_of(m->dtype))
            return CONV_I8_ERR_PARAM;
    }
    return CONV_I8_OK;
}

// a vector of n elements; an absent one (DENSE_NONE) gets a null pointer
inline conv_i8_status_t check_vec(dense_vec_t *v, int64_t n)
{
    if (v->dtype == DENSE_NONE) {
        v->ptr = nullptr;
        return CONV_I8_OK;
    }
    if (!is_float(v->dtype))
        return CONV_I8_ERR_DTYPE;
    if (v->n != n)
        return CONV_I8_ERR_DIMS;
    if (n > 0 && !v->ptr)
        return CONV_I8_ERR_NULL;
    if ((uintptr_t)v->ptr % size_of(v->dtype))
        return CONV_I8_ERR_PARAM;
    return CONV_I8_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

#define DENSE_TRY(x)                         \
    do {                                     \
        const conv_i8_status_t try_st = (x); \
        if (try_st != CONV_I8_OK)            \
            return try_st;                   \
    } while (0)

}  // namespace dense
