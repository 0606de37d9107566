// Dense layer for a few rows of x (single tokens, decode batches): bound by
// reading the weights once.
//
// A workgroup of W waves takes 16 rows of w (output columns) and all M <= 16 G
// rows of x.  The waves split the inner dimension into 128-byte blocks; each
// lane loads its 16-byte pieces of w straight into the registers that a
// 16x16 matrix instruction takes them from, so the weights never pass through
// LDS.  x comes from L2, which all workgroups share.  Rows past M (columns of
// the product) repeat the last row: their sums are not stored and do not mix
// with the others.  The waves' sums are added in order through LDS.
#pragma once

#include "dense_common.hpp"

namespace dense {

struct SkinnyArgs {
    const uint8_t *x, *w;
    int64_t ldx, ldw;  // bytes between rows
    int M, N;
    int64_t kbytes;    // inner dimension in bytes
    Epilogue epi;
};

// 16 bytes at any address that is a multiple of the element size
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Piece16 {
    v4i v;
};

template <typename T, bool ALIGNED>
__device__ __forceinline__ v4i load_piece(const uint8_t *p)
{
    if constexpr (ALIGNED)
        return *(const v4i *)p;
    else
        return ((const Piece16<T> *)p)->v;
}

// the first `valid` bytes of a piece, zeros after them
template <typename T, bool ALIGNED>
__device__ __forceinline__ v4i load_piece_tail(const uint8_t *p, int64_t valid)
{
    if (valid >= 16)
        return load_piece<T, ALIGNED>(p);
    union { v4i v; T e[16 / sizeof(T)]; } u;
    u.v = v4i{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i)
        if ((i + 1) * (int)sizeof(T) <= valid)
            u.e[i] = ((const T *)p)[i];
    return u.v;
}

template <typename T, int G, int W, bool ALIGNED>
__global__ __launch_bounds__(64 * W) void skinny_kernel(const SkinnyArgs g)
{
    typedef typename Acc4<T>::type acc_t;
    __shared__ acc_t red[W][G][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int r = lane & 15;
    const int q = (lane >> 4) * 16;

    const uint8_t *wp = g.w + (int64_t)min(n0 + r, g.N - 1) * g.ldw + q;
    const uint8_t *xp[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        xp[i] = g.x + (int64_t)min(16 * i + r, g.M - 1) * g.ldx + q;

    acc_t acc[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        acc[i] = acc_t{0, 0, 0, 0};

    // U blocks of 128 bytes a row in flight
    constexpr int U = 4;
    const int64_t blocks = g.kbytes >> 7;
    int64_t b = wave;
    for (; b + (U - 1) * W < blocks; b += U * W) {
        v4i wv[2 * U], xv[2 * U][G];
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
            const int64_t k = (b + (u >> 1) * W) * 128 + (u & 1) * 64;
            wv[u] = load_piece<T, ALIGNED>(wp + k);
#pragma unroll
            for (int i = 0; i < G; ++i)
                xv[u][i] = load_piece<T, ALIGNED>(xp[i] + k);
        }
#pragma unroll
        for (int u = 0; u < 2 * U; ++u)
#pragma unroll
            for (int i = 0; i < G; ++i)
                acc[i] = mfma16<T>(wv[u], xv[u][i], acc[i]);
    }
    for (; b < blocks; b += W) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const v4i wv = load_piece<T, ALIGNED>(wp + b * 128 + u * 64);
#pragma unroll
            for (int i = 0; i < G; ++i)
                acc[i] = mfma16<T>(wv, load_piece<T, ALIGNED>(xp[i] + b * 128 + u * 64), acc[i]);
        }
    }
    if (b == blocks) {  // the wave whose turn the last, partial block is
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t k = b * 128 + u * 64;
            const int64_t valid = g.kbytes - k - q;
            const v4i wv = load_piece_tail<T, ALIGNED>(wp + k, valid);
#pragma unroll
            for (int i = 0; i < G; ++i)
                acc[i] = mfma16<T>(wv, load_piece_tail<T, ALIGNED>(xp[i] + k, valid), acc[i]);
        }
    }

#pragma unroll
    for (int i = 0; i < G; ++i)
        red[wave][i][lane] = acc[i];
    __syncthreads();

    // sum v of lane l belongs to output column n0 + 4 (l / 16) + v of row l % 16
    for (int o = threadIdx.x; o < G * 256; o += 64 * W) {
        const int col = o & 15, row = o >> 4;
        const int i = row >> 4;
        const int src = (col >> 2) * 16 + (row & 15);
        const int m = row, n = n0 + col;
        if (m >= g.M || n >= g.N)
            continue;
        float z;
        if constexpr (sizeof(T) == 1) {
            int s = 0;
#pragma unroll
            for (int k = 0; k < W; ++k)
                s += red[k][i][src][col & 3];
            z = (float)s;
            z *= (g.epi.x_scale ? g.epi.x_scale[m] : 1.0f) * (g.epi.w_scale ? g.epi.w_scale[n] : 1.0f);
        } else {
            z = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
                z += red[k][i][src][col & 3];
        }
        if (g.epi.bias)
            z += load_dt(g.epi.bias, g.epi.bias_dt, n);
        if (g.epi.preact)
            store_dt(g.epi.preact, g.epi.out_dt, m * g.epi.ldp + n, z);
        float y = activate_rt(g.epi.act, z);
        if (g.epi.residual)
            y += load_dt(g.epi.residual, g.epi.out_dt, m * g.epi.ldr + n);
        store_dt(g.epi.out, g.epi.out_dt, m * g.epi.ldo + n, y);
    }
}

}  // namespace dense
