// Layer norm over the columns of a row, forward (in the input's type, or as
// INT8 rows with a scale) and backward, for gfx950.
//
// All are bound by HBM: every value is read once and held in registers from
// the mean to the output.  P threads share a row and hold V groups of eight
// columns each, group v at columns (v P + thread) 8, so that every load of a
// wave is one contiguous run.  With P = 64 a wave owns its row and the sums
// need no barrier; wider rows, or few of them, take a workgroup per row.
//
// What they need is bytes in flight.  A thread group walks over rows and loads
// the next one, in the form it has in memory, before it works on the present
// one, and a load has no condition per lane (TAIL: D is no multiple of eight).
// 16384 x 4096 BF16: the forward kernel 43 us (6.2 TB/s; a copy of the same bytes
// reaches 5.9), with a workgroup per row that loads, reduces and stores in turn
// 82; a backward call 76 us with its column sums, without the next row's loads 133.
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
    v = MAX ? wave_max(v) : wave_sum(v);
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
// callers pass infinity for a NaN, because a maximum skips NaN.  The inverse of a
// row below kTinyRow would not be finite: it is that of the row times kTinyUp,
// by which callers multiply the values too.
constexpr float kTinyRow = 0x1p-100f, kTinyUp = 0x1p64f;

__device__ __forceinline__ float quant_scale(float top, float &inv)
{
    inv = top > 0.0f ? 127.0f / (top < kTinyRow ? top * kTinyUp : top) : 0.0f;
    return top < INFINITY ? top / 127.0f : __builtin_nanf("");
}

// v * inv, at most 127 in magnitude, rounded half to even, in the low byte: the
// sum with 1.5 2^23 has the integer in its last bits.
__device__ __forceinline__ int8_t quantise(float v, float inv)
{
    return (int8_t)__builtin_bit_cast(int, __builtin_fmaf(v, inv, 12582912.0f));
}

// columns of a row of D that wave `wave` of its P threads holds
template <int P, int V>
__device__ __forceinline__ int wave_columns(int D, int wave)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        n += min(max(D - (i * P + wave * 64) * 8, 0), 512);
    return n;
}

// threads of a workgroup: at least 256, so that P = 64 packs four rows
constexpr int norm_threads(int P) { return P < 256 ? 256 : P; }

// Group i of a thread's part of a row, as it lies in memory.  Whether a group
// can be partial does not depend on the thread.
template <typename T, int P, int V>
__device__ __forceinline__ void load_row(const T *p, int D, int t, Raw8<T> (&r)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        r[i] = load_raw(p, (i * P + t) * 8, D);
}

template <bool TAIL, int P, typename T>
__device__ __forceinline__ void widen_group(const Raw8<T> &r, int D, int i, int t, float (&v)[8])
{
    if ((i + 1) * P * 8 <= D)
        widen(r, v);
    else
        widen_part<TAIL>(r, (i * P + t) * 8, D, v);
}

// The same of a row of weights, or `absent` everywhere where there are none
template <typename T>
__device__ __forceinline__ Raw8<T> load_param(const T *p, float absent, int c, int D)
{
    typedef T vec __attribute__((ext_vector_type(8)));
    return p ? load_raw(p, c, D) : __builtin_bit_cast(Raw8<T>, (vec)(T)absent);
}

template <typename T, int P, int V>
__device__ __forceinline__ void load_params(const T *p, float absent, int D, int t, Raw8<T> (&r)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        r[i] = load_param(p, absent, (i * P + t) * 8, D);
}

// Keeps what is computed from r inside the loop it stands in: widened weights
// held over all rows would take twice the registers (16-bit types).
template <typename T>
__device__ __forceinline__ void pin(Raw8<T> &r)
{
    if constexpr (sizeof(T) == 2)
        asm volatile("" : "+v"(r.w[0]));
}

// Mean and sum of squared distances from it, of a row held by P threads.  A
// wave takes both of its own columns (cols of them), two passes over registers;
// the waves' pairs are joined through LDS with one barrier:
//   M2 = sum over waves of M2_w + n_w (mean_w - mean)^2
template <int P, int V>
__device__ __forceinline__ void row_moments(float (&v)[V][8], int D, int t, float cols, float d, float2 *red, float &mean,
                                            float &m2)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += v[i][k];
    mean = wave_sum(s) / cols;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int cnt = D - (i * P + t) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float c = v[i][k] - mean;
            s = (i + 1) * P * 8 <= D || k < cnt ? __builtin_fmaf(c, c, s) : s;
        }
    }
    m2 = wave_sum(s);
    if constexpr (P > 64) {
        constexpr int NW = P / 64;
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = make_float2(mean, m2);
        __syncthreads();
        float2 w[NW];
        float n[NW];
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            w[i] = red[i];
            n[i] = (float)wave_columns<P, V>(D, i);
            if (n[i] > 0.0f)
                s = __builtin_fmaf(n[i], w[i].x, s);
        }
        mean = s / d;
        m2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            if (n[i] > 0.0f) {
                const float c = w[i].x - mean;
                m2 += __builtin_fmaf(n[i] * c, c, w[i].y);
            }
    }
}

// Rows walk over the grid: a thread group takes every gridDim-th one, with the
// next row's loads in flight while it works on the present one and the weights
// held over all of them (HOLD).  Workgroups of 1024 threads have 128 registers
// each and do neither: 32 columns a thread would spill.  They take one row, or
// several where a launch could not have as many threads.
template <typename T, int P, int V, bool HOLD, bool TAIL, bool Q8>
__global__ __launch_bounds__(norm_threads(P)) void norm_kernel(const NormArgs a)
{
    constexpr int RPW = norm_threads(P) / P;  // rows per workgroup
    constexpr int NW = P > 64 ? P / 64 : 1;
    __shared__ float2 red[2][NW];
    __shared__ float redq[2][NW];
    const int t = threadIdx.x % P;
    int64_t m = (int64_t)blockIdx.x * RPW + threadIdx.x / P;
    if (m >= a.M)
        return;  // whole waves; with P > 64 there is one row per workgroup
    const int64_t step = (int64_t)gridDim.x * RPW;
    const float cols = (float)wave_columns<P, V>(a.D, P > 64 ? threadIdx.x >> 6 : 0);

    Raw8<T> row[V], w[V], b[V];
    if constexpr (HOLD) {
        load_row<T, P, V>((const T *)a.x + m * a.ldx, a.D, t, row);
        load_params<T, P, V>((const T *)a.weight, 1.0f, a.D, t, w);
        load_params<T, P, V>((const T *)a.bias, 0.0f, a.D, t, b);
    }

    int set = 0;
    for (;;) {
        if constexpr (!HOLD)
            load_row<T, P, V>((const T *)a.x + m * a.ldx, a.D, t, row);
        float v[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i)
            widen_group<TAIL, P>(row[i], a.D, i, t, v[i]);
        const int64_t next = m + step;
        if (HOLD && next < a.M)
            load_row<T, P, V>((const T *)a.x + next * a.ldx, a.D, t, row);
        float mean, m2;
        row_moments<P, V>(v, a.D, t, cols, a.d, red[set], mean, m2);
        const float rstd = 1.0f / sqrtf(m2 / a.d + a.eps);
        if (t == 0) {
            if (a.mean)
                a.mean[m] = mean;
            if (a.rstd)
                a.rstd[m] = rstd;
        }
        float top = 0.0f, bad = 0.0f;  // bad: NaN if a value is not finite
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * P + t) * 8, cnt = a.D - c;
            const bool whole = (i + 1) * P * 8 <= a.D;
            float wv[8], bv[8];
            if constexpr (!HOLD) {
                w[i] = load_param((const T *)a.weight, 1.0f, c, a.D);
                b[i] = load_param((const T *)a.bias, 0.0f, c, a.D);
            }
            pin(w[i]);
            pin(b[i]);
            widen_group<TAIL, P>(w[i], a.D, i, t, wv);
            widen_group<TAIL, P>(b[i], a.D, i, t, bv);
            if (Q8 && !whole) {  // past the row's end the value is 0, also where mean rstd is infinite
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[i][k] = (TAIL ? k < cnt : cnt > 0) ? v[i][k] : mean;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[i][k] = __builtin_fmaf((v[i][k] - mean) * rstd, wv[k], bv[k]);
                if constexpr (Q8) {
                    top = fmaxf(top, fabsf(v[i][k]));
                    bad = __builtin_fmaf(v[i][k], 0.0f, bad);
                }
            }
            if constexpr (!Q8) {
                T *y = (T *)a.y + m * a.ldy + c;
                if (whole || (!TAIL && cnt > 0))
                    store_all(y, v[i]);
                else if constexpr (TAIL)
                    store_n(y, cnt, v[i]);
            }
        }
        if constexpr (Q8) {
            float inv;
            top = row_reduce<P, true>(bad == 0.0f ? top : INFINITY, redq[set], 0);
            const float scale = quant_scale(top, inv);
            if (t == 0)
                a.scale[m] = scale;
            if (top < kTinyRow) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[i][k] *= kTinyUp;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * P + t) * 8, cnt = a.D - c;
                const bool whole = (i + 1) * P * 8 <= a.D;
                struct __attribute__((packed)) Q { int8_t e[8]; } q;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    q.e[k] = quantise(v[i][k], inv);
                int8_t *y = (int8_t *)a.y + m * a.ldy + c;
                if (whole || (TAIL ? cnt >= 8 : cnt > 0)) {
                    *(Q *)y = q;
                } else if constexpr (TAIL) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < cnt)
                            y[k] = q.e[k];
                }
            }
        }
        if (next >= a.M)
            break;
        m = next;
        set ^= 1;  // the other set: a slow wave may still read this one
    }
}

// Rows longer than the registers hold: the row is read again (from cache) for
// each step.  Of the three sets of `red`, a row's next use of one comes after
// another set's barrier, so rows need none between them.
template <typename T, bool Q8>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormArgs a)
{
    __shared__ float red[3 * 16];
    const int t = threadIdx.x;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
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
            top = row_reduce<1024, true>(nan ? INFINITY : top, red, 2);
            const float scale = quant_scale(top, inv), up = top < kTinyRow ? kTinyUp : 1.0f;
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
                        y[k] = quantise(v[k] * up, inv);
            }
        }
    }
}

// Rows of fewer than eight columns, which the loads above need: a thread per
// row.  4 000 000 rows of 7 BF16 values take 22 us, bound by HBM (144 MB); with a
// workgroup per row 24 ms.
constexpr int kNarrow = 7;

template <typename T, bool Q8>
__global__ __launch_bounds__(256) void norm_narrow_kernel(const NormArgs a)
{
    const int D = a.D;
    float w[kNarrow], b[kNarrow];
#pragma unroll
    for (int k = 0; k < kNarrow; ++k) {
        w[k] = 1.0f;
        b[k] = 0.0f;
    }
    if (a.weight)
        load_n((const T *)a.weight, D, w);
    if (a.bias)
        load_n((const T *)a.bias, D, b);
    for (int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x; m < a.M; m += (int64_t)gridDim.x * 256) {
        float v[kNarrow];
        load_n((const T *)a.x + m * a.ldx, D, v);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kNarrow; ++k)
            s += v[k];
        const float mean = s / a.d;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kNarrow; ++k)
            s = k < D ? __builtin_fmaf(v[k] - mean, v[k] - mean, s) : s;
        const float rstd = 1.0f / sqrtf(s / a.d + a.eps);
        if (a.mean)
            a.mean[m] = mean;
        if (a.rstd)
            a.rstd[m] = rstd;
        float top = 0.0f;
        bool nan = false;
#pragma unroll
        for (int k = 0; k < kNarrow; ++k) {
            v[k] = k < D ? __builtin_fmaf((v[k] - mean) * rstd, w[k], b[k]) : 0.0f;
            top = fmaxf(top, fabsf(v[k]));
            nan |= v[k] != v[k];
        }
        if constexpr (Q8) {
            float inv;
            top = nan ? INFINITY : top;
            a.scale[m] = quant_scale(top, inv);
            const float up = top < kTinyRow ? kTinyUp : 1.0f;
#pragma unroll
            for (int k = 0; k < kNarrow; ++k)
                if (k < D)
                    ((int8_t *)a.y + m * a.ldy)[k] = quantise(v[k] * up, inv);
        } else {
            store_n((T *)a.y + m * a.ldy, D, v);
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
    void *dweight, *dbias;    // norm_backward_once_kernel only
};

// dx of one row after another, with the columns' sums of dy xh and dy kept in
// registers over all rows of a thread and written once per workgroup.  AHEAD
// rows are in flight while one is worked on; with none (workgroups of 1024
// threads, which have 128 registers each) the weights are read again for each
// row too.
template <typename T, int P, int V, int AHEAD, bool TAIL, bool SUMS>
__device__ __forceinline__ void backward_rows(const NormBackArgs &a, int block, int blocks)
{
    constexpr int RPW = norm_threads(P) / P;
    constexpr int NWR = P > 64 ? P / 64 : 1;
    __shared__ float2 red[2][NWR];
    const int t = threadIdx.x % P;
    const int sub = threadIdx.x / P;

    Raw8<T> w[V];
    if constexpr (AHEAD > 0)
        load_params<T, P, V>((const T *)a.weight, 1.0f, a.D, t, w);
    float sw[V][8], sb[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sw[i][k] = sb[i][k] = 0.0f;

    struct Rows {
        Raw8<T> x[V], dy[V];
        float mean, rstd;
    } ring[AHEAD > 0 ? AHEAD : 1];
    const int64_t step = (int64_t)blocks * RPW;
    auto load = [&](int64_t m, Rows &r) __attribute__((always_inline)) {
        if (m < a.M) {
            load_row<T, P, V>((const T *)a.x + m * a.ldx, a.D, t, r.x);
            load_row<T, P, V>((const T *)a.dy + m * a.lddy, a.D, t, r.dy);
            r.mean = a.mean[m];
            r.rstd = a.rstd[m];
        }
    };
    int64_t m = (int64_t)block * RPW + sub;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        load(m + i * step, ring[i]);

    int set = 0;
    auto work = [&](Rows &r) __attribute__((always_inline)) {
        if constexpr (AHEAD == 0) {
            load(m, r);
            load_params<T, P, V>((const T *)a.weight, 1.0f, a.D, t, w);
        }
        const Rows cur = r;
        const float mean = cur.mean, rstd = cur.rstd;
        if constexpr (AHEAD > 0)
            load(m + AHEAD * step, r);
        float xh[V][8], c[V][8];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float wv[8], dy[8];
            pin(w[i]);
            widen_group<TAIL, P>(w[i], a.D, i, t, wv);
            widen_group<TAIL, P>(cur.x[i], a.D, i, t, xh[i]);
            widen_group<TAIL, P>(cur.dy[i], a.D, i, t, dy);
            if ((i + 1) * P * 8 > a.D) {  // past the row's end xh is 0, also where mean rstd is infinite
                const int cnt = a.D - (i * P + t) * 8;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    xh[i][k] = (TAIL ? k < cnt : cnt > 0) ? xh[i][k] : mean;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                xh[i][k] = (xh[i][k] - mean) * rstd;
                c[i][k] = dy[k] * wv[k];
                s1 += c[i][k];
                s2 = __builtin_fmaf(c[i][k], xh[i][k], s2);
                if constexpr (SUMS) {
                    sw[i][k] = __builtin_fmaf(dy[k], xh[i][k], sw[i][k]);
                    sb[i][k] += dy[k];
                }
            }
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if constexpr (P > 64) {
            if ((threadIdx.x & 63) == 0)
                red[set][threadIdx.x >> 6] = make_float2(s1, s2);
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NWR; ++i) {
                s1 += red[set][i].x;
                s2 += red[set][i].y;
            }
            set ^= 1;  // the other set: a slow wave may still read this one
        }
        s1 /= a.d;
        s2 /= a.d;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = (i * P + t) * 8;
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = rstd * (c[i][k] - s1 - xh[i][k] * s2);
            T *dx = (T *)a.dx + m * a.lddx + at;
            if ((i + 1) * P * 8 <= a.D || (!TAIL && at < a.D))
                store_all(dx, o);
            else if constexpr (TAIL)
                store_n(dx, a.D - at, o);
        }
        m += step;
    };
    while (m < a.M) {
        // m is the same for all of a workgroup where its threads share a row
        for_each<(AHEAD > 0 ? AHEAD : 1)>([&](auto ic) __attribute__((always_inline)) {
            if (m < a.M)
                work(ring[decltype(ic)::value]);
        });
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
                        a.part[((int64_t)block * 2 + (i >= V)) * a.part_ld + col] = v;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * P + t) * 8;
                float *p = a.part + (int64_t)block * 2 * a.part_ld + c;
                store_n(p, a.D - c, sw[i]);
                store_n(p + a.part_ld, a.D - c, sb[i]);
            }
        }
    }
}

template <typename T, int P, int V, int AHEAD, bool TAIL, bool SUMS>
__global__ __launch_bounds__(norm_threads(P)) void norm_backward_kernel(const NormBackArgs a)
{
    backward_rows<T, P, V, AHEAD, TAIL, SUMS>(a, blockIdx.x, gridDim.x);
}

// Everything in one launch, for few rows: the first workgroups sum 32 columns
// each over all rows, four threads to a row, the others take one row per thread
// group.  x and dy are read twice, the second time from cache; what it saves is
// the partial sums on their way out and back, and a launch.  With many rows the
// walk down the columns lasts longest, sooner in wide rows, of which one launch
// has few in flight: 256 x 4096 BF16 6.2 us (two launches 10.5), 1000 x 4096 11.6
// (14.8), 1000 x 256 6.1 (7.7), 1000 x 1537 FP32 11.7 (12.5), 1000 x 8192 FP32 26.9
// (27.3); but 1000 x 9001 BF16 41 (31), 1000 x 16384 FP32 66 (54), 512 x 16384 FP32
// 33.8 (34.2).
constexpr int64_t once_rows(int64_t D) { return D <= 8192 ? 1024 : 512; }
constexpr int kOnceCols = 32;

template <typename T, int P, int V, bool TAIL>
__global__ __launch_bounds__(norm_threads(P)) void norm_backward_once_kernel(const NormBackArgs a, int col_blocks)
{
    if ((int)blockIdx.x >= col_blocks) {
        backward_rows<T, P, V, 0, TAIL, false>(a, blockIdx.x - col_blocks, gridDim.x - col_blocks);
        return;
    }
    constexpr int LANES = kOnceCols / 8, G = norm_threads(P) / LANES, U = 16 / sizeof(T);
    __shared__ float sums[2][norm_threads(P) / 64][kOnceCols];
    const int c = blockIdx.x * kOnceCols + (threadIdx.x % LANES) * 8, grp = threadIdx.x / LANES;
    float sw[8] = {}, sb[8] = {};
    for (int m = grp; m < a.M; m += U * G) {
        Raw8<T> x[U], dy[U];
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // rows past the end repeat the last one
            const int64_t r = min(m + u * G, a.M - 1);
            x[u] = load_raw((const T *)a.x + r * a.ldx, c, a.D);
            dy[u] = load_raw((const T *)a.dy + r * a.lddy, c, a.D);
            mean[u] = a.mean[r];
            rstd[u] = a.rstd[r];
        }
        // without the branches of TAIL the loads would be moved to their uses, a wait for each
        // (1000 x 2048 BF16 18.1 us; 10.4 with them together)
        if constexpr (!TAIL)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (m + u * G >= a.M)
                break;
            float xv[8], g[8];
            widen_part<TAIL>(x[u], c, a.D, xv);
            widen_part<TAIL>(dy[u], c, a.D, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sw[k] = __builtin_fmaf(g[k], (xv[k] - mean[u]) * rstd[u], sw[k]);
                sb[k] += g[k];
            }
        }
    }
    // the wave's sixteen rows by shuffles, the waves through LDS
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int o = 32; o >= LANES; o >>= 1) {
            sw[k] += __shfl_xor(sw[k], o, 64);
            sb[k] += __shfl_xor(sb[k], o, 64);
        }
    if ((threadIdx.x & 63) < LANES)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sums[0][threadIdx.x >> 6][(threadIdx.x % LANES) * 8 + k] = sw[k];
            sums[1][threadIdx.x >> 6][(threadIdx.x % LANES) * 8 + k] = sb[k];
        }
    __syncthreads();
    const int col = blockIdx.x * kOnceCols + threadIdx.x % kOnceCols, which = threadIdx.x / kOnceCols;
    if (which < 2 && col < a.D) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < norm_threads(P) / 64; ++i)
            v += sums[which][i][threadIdx.x % kOnceCols];
        ((T *)(which ? a.dbias : a.dweight))[col] = (T)v;
    }
}

// Rows longer than the registers hold: dx with the row read twice (the two sets
// of `red` alternate, so rows need no barrier between them) ...
template <typename T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(const NormBackArgs a)
{
    __shared__ float red[2 * 16];
    const int t = threadIdx.x;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
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

// Rows of fewer than eight columns: a thread per row, the columns' sums over a
// workgroup's rows in registers, then over its waves.  4 000 000 rows of 7 BF16
// values: 45 us with the column sums, 40 without (200 MB).
template <typename T>
__global__ __launch_bounds__(256) void norm_backward_narrow_kernel(const NormBackArgs a)
{
    __shared__ float red[4][2 * kNarrow];
    const int D = a.D;
    float w[kNarrow], sw[kNarrow] = {}, sb[kNarrow] = {};
#pragma unroll
    for (int k = 0; k < kNarrow; ++k)
        w[k] = 1.0f;
    if (a.weight)
        load_n((const T *)a.weight, D, w);
    for (int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x; m < a.M; m += (int64_t)gridDim.x * 256) {
        const float mean = a.mean[m], rstd = a.rstd[m];
        float xh[kNarrow], g[kNarrow], c[kNarrow];
        load_n((const T *)a.x + m * a.ldx, D, xh, mean);
        load_n((const T *)a.dy + m * a.lddy, D, g);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < kNarrow; ++k) {
            xh[k] = (xh[k] - mean) * rstd;
            c[k] = g[k] * w[k];
            s1 += c[k];
            s2 = __builtin_fmaf(c[k], xh[k], s2);
            sw[k] = __builtin_fmaf(g[k], xh[k], sw[k]);
            sb[k] += g[k];
        }
        s1 /= a.d;
        s2 /= a.d;
#pragma unroll
        for (int k = 0; k < kNarrow; ++k)
            c[k] = rstd * (c[k] - s1 - xh[k] * s2);
        store_n((T *)a.dx + m * a.lddx, D, c);
    }
    if (!a.part)
        return;
#pragma unroll
    for (int k = 0; k < kNarrow; ++k) {
        sw[k] = wave_sum(sw[k]);
        sb[k] = wave_sum(sb[k]);
        if ((threadIdx.x & 63) == 0) {
            red[threadIdx.x >> 6][k] = sw[k];
            red[threadIdx.x >> 6][kNarrow + k] = sb[k];
        }
    }
    __syncthreads();
    const int k = threadIdx.x % kNarrow, which = threadIdx.x / kNarrow;
    if (which < 2 && k < D)
        a.part[((int64_t)blockIdx.x * 2 + which) * a.part_ld + k] =
            (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
}

}  // namespace dense
