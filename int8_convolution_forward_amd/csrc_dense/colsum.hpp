// The last step of sums over rows (bias gradients, the gradients of a norm's
// weights): partial sums of blocks of rows, added in a fixed order.
#pragma once

#include "dense_common.hpp"

namespace dense {

// out[c] = sum over r of part[r][c].  Columns [0, split) go to out0 and [split,
// cols) to out1, the first `valid` of each.
struct ColSumArgs {
    const float *part;
    int64_t ld;
    int rows;
    int64_t cols, split, valid;
    void *out0, *out1;
    int dt;
};

constexpr int kSumGroups = 32;

// COLS columns by kSumGroups groups of COLS threads: a group takes every
// kSumGroups-th row, eight loads at a time, and the groups are added through
// LDS, so the order of the sum does not depend on COLS.  A few hundred rows are
// bound by the latency of their loads: 251 rows of 3088 columns 2.6 us, with 8
// groups and four loads at a time 5.3.
template <int COLS>
__device__ __forceinline__ void column_sums(const ColSumArgs &a, int block, float (*red)[COLS + 1])
{
    constexpr int G = kSumGroups, U = 8;
    const int c = threadIdx.x % COLS, grp = threadIdx.x / COLS;
    const int64_t col = (int64_t)block * COLS + c;
    const bool second = col >= a.split;
    const int64_t oc = second ? col - a.split : col;
    const bool live = col < a.cols && oc < a.valid;
    float s[U] = {};
    if (live) {
        const float *p = a.part + col;
        int r = grp;
        for (; r + (U - 1) * G < a.rows; r += U * G) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                s[k] += p[(r + G * k) * a.ld];
        }
        // the rest without a wait between the loads: rows past the end repeat the last one
        if (r < a.rows) {
            float v[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                v[k] = p[min(r + G * k, a.rows - 1) * a.ld];
#pragma unroll
            for (int k = 0; k < U; ++k)
                s[k] += r + G * k < a.rows ? v[k] : 0.0f;
        }
    }
    red[grp][c] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (grp == 0 && live) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < G; ++k)
            v += red[k][c];
        store_dt(second ? a.out1 : a.out0, a.dt, oc, v);
    }
}

// Workgroups of colsum_kernel: they walk over the columns where one each would
// be more threads than a launch may have (2^32).
inline dim3 colsum_grid(int64_t cols)
{
    const int64_t wgs = (cols + 31) / 32;
    return dim3((unsigned)(wgs < (1 << 21) ? wgs : 1 << 21));
}

template <int COLS = 32>
__global__ __launch_bounds__(COLS * kSumGroups) void colsum_kernel(const ColSumArgs a)
{
    __shared__ float red[kSumGroups][COLS + 1];
    const int blocks = (int)((a.cols + COLS - 1) / COLS);
    for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
        column_sums<COLS>(a, b, red);
        if (b + (int)gridDim.x < blocks)
            __syncthreads();  // the sums are read before the next columns overwrite them
    }
}

}  // namespace dense
