// Layer norm over the columns of a row, forward (in the input's type, or as
// INT8 rows with a scale) and backward, for gfx950.
//
// All are bound by HBM: every value is read once and held in registers from
// the mean to the output.  P threads share a row and hold V groups of eight
// columns each, group v at columns (v P + thread) 8, so that every load of a
// wave is one contiguous run.  With P = 64 a wave owns its row and the sums
// need no barrier; wider rows, or few of them, take a workgroup per row.
#pragma once

#include "dense_common.hpp"

namespace dense {

struct NormArgs {
    const void *x, *weight, *bias;  // weight, bias: null for ones, zeros
    void *y;
    int64_t ldx, ldy;
    int M, D;
    float eps;
    float d;                        // D; sums are divided by it, so that a constant row's mean is exact
    float *mean, *rstd, *scale;     // null: not written
};

// Sum (or maximum) over the P threads of a row.  For P > 64 the waves' values
// go through LDS; `red` holds two sets so that one barrier per call is enough.
template <int P, bool MAX = false>
__device__ __forceinline__ float row_reduce(float v, float *red, int set)
{
    v = MAX ? wave_max<64>(v) : wave_sum<64>(v);
    if constexpr (P > 64) {
        constexpr int NW = P / 64;
        float *r = red + set * NW;
        if ((threadIdx.x & 63) == 0)
            r[threadIdx.x >> 6] = v;
        __syncthreads();
        v = r[0];
#pragma unroll
        for (int i = 1; i < NW; ++i)
            v = MAX ? fmaxf(v, r[i]) : v + r[i];
    }
    return v;
}

// Scale of an INT8 row whose largest magnitude is `top`, and its inverse (0 for
// a row of zeros).  A row with a value that is not finite gets the scale NaN;
// callers pass infinity for a NaN, because a maximum skips NaN.
__device__ __forceinline__ float quant_scale(float top, float &inv)
{
    inv = top > 0.0f ? 127.0f / top : 0.0f;
    return top < INFINITY ? top / 127.0f : __builtin_nanf("");
}

// threads of a workgroup: at least 256, so that P = 64 packs four rows
constexpr int norm_threads(int P) { return P < 256 ? 256 : P; }

template <typename T, int P, int V, bool Q8>
__global__ __launch_bounds__(norm_threads(P)) void norm_kernel(const NormArgs a)
{
    constexpr int RPW = norm_threads(P) / P;  // rows per workgroup
    __shared__ float red[3 * (P > 64 ? P / 64 : 1)];
    const int t = threadIdx.x % P;
    const int64_t m = (int64_t)blockIdx.x * RPW + threadIdx.x / P;
    if (m >= a.M)
        return;  // whole waves; with P > 64 there is one row per workgroup
    const T *x = (const T *)a.x + m * a.ldx;

    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
        load_n(x + (i * P + t) * 8, a.D - (i * P + t) * 8, v[i]);

    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += v[i][k];
    const float mean = row_reduce<P>(s, red, 0) / a.d;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int cnt = a.D - (i * P + t) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[i][k] = k < cnt ? v[i][k] - mean : 0.0f;
            s = __builtin_fmaf(v[i][k], v[i][k], s);
        }
    }
    const float rstd = 1.0f / sqrtf(row_reduce<P>(s, red, 1) / a.d + a.eps);
    if (t == 0) {
        if (a.mean)
            a.mean[m] = mean;
        if (a.rstd)
            a.rstd[m] = rstd;
    }
    float top = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * P + t) * 8, cnt = a.D - c;
        if (cnt <= 0)
            continue;
        float w[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            w[k] = 1.0f;
            b[k] = 0.0f;
        }
        if (a.weight)
            load_n((const T *)a.weight + c, cnt, w);
        if (a.bias)
            load_n((const T *)a.bias + c, cnt, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[i][k] = __builtin_fmaf(v[i][k] * rstd, w[k], b[k]);
            if constexpr (Q8) {
                const float u = k < cnt ? v[i][k] : 0.0f;
                top = fmaxf(top, fabsf(u));
                nan |= u != u;
            }
        }
        if constexpr (!Q8)
            store_n((T *)a.y + m * a.ldy + c, cnt, v[i]);
    }
    if constexpr (Q8) {
        float inv;
        const float scale = quant_scale(row_reduce<P, true>(nan ? INFINITY : top, red, 2), inv);
        if (t == 0)
            a.scale[m] = scale;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * P + t) * 8, cnt = a.D - c;
            if (cnt <= 0)
                continue;
            struct __attribute__((packed)) Q { int8_t e[8]; } q;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                q.e[k] = (int8_t)(int)__builtin_rintf(fminf(fmaxf(v[i][k] * inv, -127.0f), 127.0f));
            int8_t *y = (int8_t *)a.y + m * a.ldy + c;
            if (cnt >= 8) {
                *(Q *)y = q;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < cnt)
                        y[k] = q.e[k];
            }
        }
    }
}

// Rows longer than the registers hold: the row is read again (from cache) for
// each step.
template <typename T, bool Q8>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a)
{
    __shared__ float red[3 * 16];
    const int t = threadIdx.x;
    const int64_t m = blockIdx.x;
    const T *x = (const T *)a.x + m * a.ldx;
    float s = 0.0f;
    for (int64_t c = t * 8; c < a.D; c += 8192) {
        float v[8];
        load_n(x + c, (int)(a.D - c), v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += v[k];
    }
    const float mean = row_reduce<1024>(s, red, 0) / a.d;
    s = 0.0f;
    for (int64_t c = t * 8; c < a.D; c += 8192) {
        float v[8];
        load_n(x + c, (int)(a.D - c), v, mean);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s = __builtin_fmaf(v[k] - mean, v[k] - mean, s);
    }
    const float rstd = 1.0f / sqrtf(row_reduce<1024>(s, red, 1) / a.d + a.eps);
    if (t == 0) {
        if (a.mean)
            a.mean[m] = mean;
        if (a.rstd)
            a.rstd[m] = rstd;
    }
    auto value = [&](int64_t c, int cnt, float (&v)[8]) {
        float w[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            w[k] = 1.0f;
            b[k] = 0.0f;
        }
        load_n(x + c, cnt, v);
        if (a.weight)
            load_n((const T *)a.weight + c, cnt, w);
        if (a.bias)
            load_n((const T *)a.bias + c, cnt, b);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = __builtin_fmaf((v[k] - mean) * rstd, w[k], b[k]);
    };
    float top = 0.0f;
    bool nan = false;
    for (int64_t c = t * 8; c < a.D; c += 8192) {
        const int cnt = (int)(a.D - c);
        float v[8];
        value(c, cnt, v);
        if constexpr (Q8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float u = k < cnt ? v[k] : 0.0f;
                top = fmaxf(top, fabsf(u));
                nan |= u != u;
            }
        } else {
            store_n((T *)a.y + m * a.ldy + c, cnt, v);
        }
    }
    if constexpr (Q8) {
        float inv;
        const float scale = quant_scale(row_reduce<1024, true>(nan ? INFINITY : top, red, 2), inv);
        if (t == 0)
            a.scale[m] = scale;
        for (int64_t c = t * 8; c < a.D; c += 8192) {
            const int cnt = (int)(a.D - c);
            float v[8];
            value(c, cnt, v);
            int8_t *y = (int8_t *)a.y + m * a.ldy + c;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < cnt)
                    y[k] = (int8_t)(int)__builtin_rintf(fminf(fmaxf(v[k] * inv, -127.0f), 127.0f));
        }
    }
}

struct NormBackArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void *dx;
    int64_t lddy, ldx, lddx;
    int M, D;
    float d;                        // D; sums are divided by it, so that a constant row's mean is exact
    float *part;              // [workgroup][2][part_ld]: column sums of dy xh and of dy; null: not computed
    int64_t part_ld;
};

// dx of one row after another, with the columns' sums of dy xh and dy kept in
// registers over all rows of a thread and written once per workgroup.
template <typename T, int P, int V, bool SUMS>
__global__ __launch_bounds__(norm_threads(P)) void norm_backward_kernel(const NormBackArgs a)
{
    constexpr int RPW = norm_threads(P) / P;
    constexpr int NWR = P > 64 ? P / 64 : 1;
    __shared__ float red[4 * NWR];
    const int t = threadIdx.x % P;
    const int sub = threadIdx.x / P;

    float w[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (a.weight) {
            load_n((const T *)a.weight + (i * P + t) * 8, a.D - (i * P + t) * 8, w[i]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[i][k] = 1.0f;
        }
    }
    float sw[V][8], sb[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sw[i][k] = sb[i][k] = 0.0f;

    int set = 0;
    for (int64_t m = (int64_t)blockIdx.x * RPW + sub; m < a.M; m += (int64_t)gridDim.x * RPW) {
        const float mean = a.mean[m], rstd = a.rstd[m];
        float xh[V][8], dy[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * P + t) * 8;
            load_n((const T *)a.x + m * a.ldx + c, a.D - c, xh[i]);
            load_n((const T *)a.dy + m * a.lddy + c, a.D - c, dy[i]);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                xh[i][k] = (xh[i][k] - mean) * rstd;
                const float c = dy[i][k] * w[i][k];
                s1 += c;
                s2 = __builtin_fmaf(c, xh[i][k], s2);
                if constexpr (SUMS) {
                    sw[i][k] = __builtin_fmaf(dy[i][k], xh[i][k], sw[i][k]);
                    sb[i][k] += dy[i][k];
                }
            }
        s1 = wave_sum<64>(s1);
        s2 = wave_sum<64>(s2);
        if constexpr (P > 64) {
            float *r = red + set * 2 * NWR;
            if ((threadIdx.x & 63) == 0) {
                r[threadIdx.x >> 6] = s1;
                r[NWR + (threadIdx.x >> 6)] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NWR; ++i) {
                s1 += r[i];
                s2 += r[NWR + i];
            }
            set ^= 1;  // the other set: a slow wave may still read this one
        }
        s1 /= a.d;
        s2 /= a.d;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * P + t) * 8;
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = rstd * (dy[i][k] * w[i][k] - s1 - xh[i][k] * s2);
            store_n((T *)a.dx + m * a.lddx + c, a.D - c, o);
        }
    }
    if constexpr (SUMS) {
        if constexpr (RPW > 1) {
            // rows of one workgroup: added in order through LDS, eight columns
            // a thread at a time
            __shared__ float cs[RPW][P * 8];
            for (int i = 0; i < 2 * V; ++i) {
                __syncthreads();
#pragma unroll
                for (int u = 0; u < 2 * V; ++u)  // registers are indexed by constants
                    if (u == i)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            cs[sub][k * P + t] = u < V ? sw[u % V][k] : sb[u % V][k];
                __syncthreads();
                const int c0 = (i % V) * P * 8;
                for (int e = threadIdx.x; e < P * 8; e += norm_threads(P)) {
                    const int col = c0 + e, src = (e & 7) * P + (e >> 3);
                    float v = 0.0f;
#pragma unroll
                    for (int r = 0; r < RPW; ++r)
                        v += cs[r][src];
                    if (col < a.D)
                        a.part[((int64_t)blockIdx.x * 2 + (i >= V)) * a.part_ld + col] = v;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * P + t) * 8;
                float *p = a.part + (int64_t)blockIdx.x * 2 * a.part_ld + c;
                store_n(p, a.D - c, sw[i]);
                store_n(p + a.part_ld, a.D - c, sb[i]);
            }
        }
    }
}

// Rows longer than the registers hold: dx with the row read twice ...
template <typename T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(const NormBackArgs a)
{
    __shared__ float red[2 * 16];
    const int t = threadIdx.x;
    const int64_t m = blockIdx.x;
    const T *x = (const T *)a.x + m * a.ldx, *g = (const T *)a.dy + m * a.lddy;
    const float mean = a.mean[m], rstd = a.rstd[m];
    auto load = [&](int64_t c, int cnt, float (&xh)[8], float (&cv)[8]) {
        float w[8];
        load_n(x + c, cnt, xh, mean);
        load_n(g + c, cnt, cv);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = 1.0f;
        if (a.weight)
            load_n((const T *)a.weight + c, cnt, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            xh[k] = (xh[k] - mean) * rstd;
            cv[k] *= w[k];
        }
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = t * 8; c < a.D; c += 8192) {
        float xh[8], cv[8];
        load(c, (int)(a.D - c), xh, cv);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s1 += cv[k];
            s2 = __builtin_fmaf(cv[k], xh[k], s2);
        }
    }
    s1 = row_reduce<1024>(s1, red, 0) / a.d;
    s2 = row_reduce<1024>(s2, red, 1) / a.d;
    for (int64_t c = t * 8; c < a.D; c += 8192) {
        float xh[8], cv[8];
        load(c, (int)(a.D - c), xh, cv);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            cv[k] = rstd * (cv[k] - s1 - xh[k] * s2);
        store_n((T *)a.dx + m * a.lddx + c, (int)(a.D - c), cv);
    }
}

// ... and the column sums of a block of rows, 2048 columns a workgroup.
template <typename T>
__global__ __launch_bounds__(256) void norm_backward_sums_kernel(const NormBackArgs a, int rows)
{
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    const int cnt = (int)(a.D - c);
    if (cnt <= 0)
        return;
    const int m1 = min(a.M, (int)(blockIdx.y + 1) * rows);
    float sw[8] = {}, sb[8] = {};
    for (int64_t m = (int64_t)blockIdx.y * rows; m < m1; ++m) {
        const float mean = a.mean[m], rstd = a.rstd[m];
        float xv[8], g[8];
        load_n((const T *)a.x + m * a.ldx + c, cnt, xv);
        load_n((const T *)a.dy + m * a.lddy + c, cnt, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sw[k] = __builtin_fmaf(g[k], (xv[k] - mean) * rstd, sw[k]);
            sb[k] += g[k];
        }
    }
    float *p = a.part + (int64_t)blockIdx.y * 2 * a.part_ld + c;
    store_n(p, cnt, sw);
    store_n(p + a.part_ld, cnt, sb);
}

}  // namespace dense
