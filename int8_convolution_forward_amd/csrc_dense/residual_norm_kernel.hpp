// The norm between two blocks fused with the residual connection, forward and
// backward, for gfx950:
//
//   n = norm(h) post_weight, or h;  r = alpha x + gate n;  y = norm(r) weight + bias
//
// Bound by HBM, as layer norm (whose split of a row over P threads of V groups of
// eight columns this shares): every row is read once, held in registers through
// both norms, and written once.  r is rounded to its type before its norm is
// taken: the backward pass, which reads it back, then works on the same values.
//
// A thread group walks over rows and has the next one's loads in flight while it
// works on the present one (HOLD).  Workgroups of 1024 threads, for rows of more than
// 8192 columns, have 128 registers each and do neither that nor keep the weights;
// layer norm spills all the same, 16 to 39 registers of BF16 and 43 to 72 of FP32 (rms
// none and up to 6), which shows: r and y of 4096 x 16384 BF16 106 us as rms (537 MB,
// 5.1 TB/s), 157 as layer norm, 4096 x 12288 82 and 146.
#pragma once

#include "colsum.hpp"
#include "fp8_kernel.hpp"
#include "norm_kernel.hpp"

namespace dense {

struct ResNormArgs {
    const void *x, *h, *gate, *weight, *bias, *post_weight;  // null: absent
    void *r, *y;                   // r null: not written (it is x)
    uint8_t *y_scale;              // for an e4m3 y
    int64_t ldx, ldh, ldg, ldr, ldy, ldys;
    int M, D;
    int gate_rows;                 // rows that share a row of the gate
    float alpha, eps, d;
    float *mean, *rstd, *post_mean, *post_rstd;  // null: not written
};

template <int CTRL>
__device__ __forceinline__ float add_dpp(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, i, CTRL, 0xf, 0xf, true));
}

// Sum of the sixteen lanes of a row, in all of them
__device__ __forceinline__ float row16_sum(float v)
{
    return add_dpp<0x140>(add_dpp<0x141>(add_dpp<0x4E>(add_dpp<0xB1>(v))));
}

// Mean and sum of squared distances from it; RMS: 0 and the sum of squares.
template <int P, int V, bool RMS>
__device__ __forceinline__ void moments(float (&v)[V][8], int D, int t, float cols, float d, float2 *red, float &mean,
                                        float &m2)
{
    if constexpr (!RMS) {
        row_moments<P, V>(v, D, t, cols, d, red, mean, m2);
    } else {
        mean = m2 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                m2 = __builtin_fmaf(v[i][k], v[i][k], m2);
        m2 = row_reduce<P>(m2, (float *)red, 0);
    }
}

// 1 / deviation from the sum of squares m2 of d columns.  NaN, as 0 times m2, where 32 bits
// do not hold m2: by the formula that row, finite as its values may be, would become
// its bias with no gradient, and nobody would see it.  One instruction: a comparison
// takes 51.3 us for 4096 x 8192 BF16 as layer norm, this 49.2 as without.  (Taking such a
// row again, divided by a power of two, costs the registers of the usual ones: 8192 x 4096
// BF16 with both norms and gates 62.3 us instead of 57.5, 4096 x 8192 54.0.)
__device__ __forceinline__ float inverse_deviation(float m2, float d, float eps)
{
    return __builtin_fmaf(m2, 0.0f, 1.0f / sqrtf(m2 / d + eps));
}

template <typename T, int P, int V, bool HOLD, bool TAIL, bool RMS, bool Q8>
__global__ __launch_bounds__(norm_threads(P)) void residual_norm_kernel(const ResNormArgs a)
{
    constexpr int RPW = norm_threads(P) / P;  // rows per workgroup
    constexpr int NW = P > 64 ? P / 64 : 1;
    __shared__ float2 red[2][NW];
    const int t = threadIdx.x % P;
    int64_t m = (int64_t)blockIdx.x * RPW + (RPW > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / P) : 0);
    if (m >= a.M)
        return;  // whole waves; with P > 64 there is one row per workgroup
    const int64_t step = (int64_t)gridDim.x * RPW;
    const float cols = (float)wave_columns<P, V>(a.D, P > 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0);

    Raw8<T> x[V], h[V], g[V], w[V], b[V], pw[V];
    auto load = [&](int64_t m) __attribute__((always_inline)) {
        load_row<T, P, V>((const T *)a.x + m * a.ldx, a.D, t, x);
        if (a.h)
            load_row<T, P, V>((const T *)a.h + m * a.ldh, a.D, t, h);
        if (a.gate)
            load_row<T, P, V>((const T *)a.gate + (int64_t)((unsigned)m / (unsigned)a.gate_rows) * a.ldg, a.D, t, g);
    };
    if constexpr (HOLD) {
        load(m);
        load_params<T, P, V>((const T *)a.weight, 1.0f, a.D, t, w);
        load_params<T, P, V>((const T *)a.bias, 0.0f, a.D, t, b);
        load_params<T, P, V>((const T *)a.post_weight, 1.0f, a.D, t, pw);
    }
    int set = 0;
    for (;;) {
        if constexpr (!HOLD)
            load(m);
        float v[V][8], n[V][8], gv[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            widen_group<TAIL, P>(x[i], a.D, i, t, v[i]);
            if (a.h)
                widen_group<TAIL, P>(h[i], a.D, i, t, n[i]);
            if (a.gate)
                widen_group<TAIL, P>(g[i], a.D, i, t, gv[i]);
        }
        const int64_t next = m + step;
        if (HOLD && next < a.M)
            load(next);
        float mean, m2;
        if (a.h) {
            if (a.post_weight) {
                moments<P, V, RMS>(n, a.D, t, cols, a.d, red[set], mean, m2);
                set ^= 1;  // the other set: a slow wave may still read this one
                const float rstd = inverse_deviation(m2, a.d, a.eps);
                if (t == 0) {
                    if (a.post_mean)
                        a.post_mean[m] = mean;
                    if (a.post_rstd)
                        a.post_rstd[m] = rstd;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float pv[8];
                    if constexpr (!HOLD)
                        pw[i] = load_param((const T *)a.post_weight, 1.0f, (i * P + t) * 8, a.D);
                    pin(pw[i]);
                    widen_group<TAIL, P>(pw[i], a.D, i, t, pv);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        n[i][k] = (n[i][k] - mean) * rstd * pv[k];
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * P + t) * 8, cnt = a.D - c;
                const bool whole = (i + 1) * P * 8 <= a.D;
                typedef T vec __attribute__((ext_vector_type(8)));
                vec kept;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float s = a.gate ? gv[i][k] * n[i][k] : n[i][k];
                    kept[k] = (T)__builtin_fmaf(a.alpha, v[i][k], s);
                    v[i][k] = (float)kept[k];
                }
                T *r = (T *)a.r + m * a.ldr + c;
                if (whole || (!TAIL && cnt > 0))
                    *(Pack<T, 8> *)r = __builtin_bit_cast(Pack<T, 8>, kept);
                else if constexpr (TAIL)
                    store_n(r, cnt, v[i]);
                if (!whole) {  // past the row's end r is 0, also where a norm is infinite
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[i][k] = (TAIL ? k < cnt : cnt > 0) ? v[i][k] : 0.0f;
                }
            }
        }
        moments<P, V, RMS>(v, a.D, t, cols, a.d, red[set], mean, m2);
        set ^= 1;
        const float rstd = inverse_deviation(m2, a.d, a.eps);
        if (t == 0) {
            if (a.mean)
                a.mean[m] = mean;
            if (a.rstd)
                a.rstd[m] = rstd;
        }
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
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[i][k] = __builtin_fmaf((v[i][k] - mean) * rstd, wv[k], bv[k]);
            if constexpr (Q8) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    top = fmaxf(top, whole || k < cnt ? finite_size(v[i][k]) : 0.0f);
                const int byte = scale_byte(block_max(top), false);
                if (whole || cnt > 0) {
                    store_bytes((uint8_t *)a.y + m * a.ldy + c, whole ? 8 : cnt, encode8(v[i], inverse_scale(byte), false));
                    if ((threadIdx.x & 15) == 0)
                        a.y_scale[m * a.ldys + (c >> 7)] = (uint8_t)byte;
                }
            } else {
                T *y = (T *)a.y + m * a.ldy + c;
                if (whole || (!TAIL && cnt > 0))
                    store_all(y, v[i]);
                else if constexpr (TAIL)
                    store_n(y, cnt, v[i]);
            }
        }
        if (next >= a.M)
            break;
        m = next;
    }
}

// Rows of any other length: fewer than eight columns, or more than the registers
// hold.  A row is read again, from cache, for each step; each thread reads only
// columns of r that it wrote itself.
template <typename T, int P, bool RMS, bool Q8>
__global__ __launch_bounds__(P) void residual_norm_any_kernel(const ResNormArgs a)
{
    constexpr int NW = P > 64 ? P / 64 : 1;
    __shared__ float red[2 * NW];
    const int t = threadIdx.x;
    int set = 0;
    // the sets take turns: a slow wave may still read the last one
    auto sum = [&](float v) __attribute__((always_inline)) { return row_reduce<P>(v, red, set ^= 1); };
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const T *x = (const T *)a.x + m * a.ldx;
        auto stats = [&](const T *p, float &mean, float &rstd) {
            mean = 0.0f;
            if constexpr (!RMS) {
                float s = 0.0f;
                for (int64_t c = t * 8; c < a.D; c += P * 8) {
                    float v[8];
                    load_n(p + c, (int)(a.D - c), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        s += v[k];
                }
                mean = sum(s) / a.d;
            }
            float s = 0.0f;
            for (int64_t c = t * 8; c < a.D; c += P * 8) {
                float v[8];
                load_n(p + c, (int)(a.D - c), v, mean);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s = __builtin_fmaf(v[k] - mean, v[k] - mean, s);
            }
            rstd = inverse_deviation(sum(s), a.d, a.eps);
        };
        float mean, rstd;
        const T *src = x;
        if (a.h) {
            const T *h = (const T *)a.h + m * a.ldh;
            if (a.post_weight) {
                stats(h, mean, rstd);
                if (t == 0) {
                    if (a.post_mean)
                        a.post_mean[m] = mean;
                    if (a.post_rstd)
                        a.post_rstd[m] = rstd;
                }
            }
            T *r = (T *)a.r + m * a.ldr;
            const T *gate = a.gate ? (const T *)a.gate + (int64_t)((unsigned)m / (unsigned)a.gate_rows) * a.ldg : nullptr;
            for (int64_t c = t * 8; c < a.D; c += P * 8) {
                const int cnt = (int)(a.D - c);
                float v[8], n[8], p[8];
                load_n(x + c, cnt, v);
                load_n(h + c, cnt, n);
                if (a.post_weight) {
                    load_n((const T *)a.post_weight + c, cnt, p);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        n[k] = (n[k] - mean) * rstd * p[k];
                }
                if (gate) {
                    load_n(gate + c, cnt, p);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        n[k] *= p[k];
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = __builtin_fmaf(a.alpha, v[k], n[k]);
                store_n(r + c, cnt, v);
            }
            src = r;
        }
        stats(src, mean, rstd);
        if (t == 0) {
            if (a.mean)
                a.mean[m] = mean;
            if (a.rstd)
                a.rstd[m] = rstd;
        }
        // all lanes of a wave go round together: the blocks' largest magnitudes pass between them
        for (int64_t c0 = 0; c0 < a.D; c0 += P * 8) {
            const int64_t c = c0 + t * 8;
            const int cnt = c < a.D ? (int)(a.D - c) : 0;
            float v[8], w[8], b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                w[k] = 1.0f;
                b[k] = 0.0f;
            }
            load_n(src + c, cnt, v);
            if (a.weight)
                load_n((const T *)a.weight + c, cnt, w);
            if (a.bias)
                load_n((const T *)a.bias + c, cnt, b);
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = __builtin_fmaf((v[k] - mean) * rstd, w[k], b[k]);
                top = fmaxf(top, k < cnt ? finite_size(v[k]) : 0.0f);
            }
            if constexpr (Q8) {
                const int byte = scale_byte(block_max(top), false);
                if (cnt > 0) {
                    store_bytes((uint8_t *)a.y + m * a.ldy + c, cnt, encode8(v, inverse_scale(byte), false));
                    if ((t & 15) == 0)
                        a.y_scale[m * a.ldys + (c >> 7)] = (uint8_t)byte;
                }
            } else {
                store_n((T *)a.y + m * a.ldy + c, cnt, v);
            }
        }
    }
}

// ---- gradients -----------------------------------------------------------------
//
//   rh = (r - mean) rstd, c = dy weight:  t = dr + rstd (c - mean(c) - rh mean(c rh));  dx = alpha t
//   hh = (h - post_mean) post_rstd, n = hh post_weight (or h), u = gate t, e = u post_weight:
//   dh = post_rstd (e - mean(e) - hh mean(e hh)), or u
//   dweight = sum dy rh, dbias = sum dy, dpost_weight = sum u hh, dgate = sum t n over the gate's rows
//
// The columns' sums stay in registers over all rows of a workgroup.  Its rows are
// either part of those of one row of the gate (chunks > 1; the partial sums are
// added by residual_norm_sums_kernel) or those of whole rows of the gate, for which
// it writes dgate itself.
//
// Bound by HBM and, nearly as much, by the vector unit (about 40 operations a value
// with the widening of four inputs): 16384 x 4096 BF16 with both norms and eight
// gates 154 us, 806 MB, 5.2 TB/s.  What took it there from 176: sums of a wave
// folded two into one register before they are added up (a lane permutation for
// each sum by itself takes four times the operations), means by a product instead
// of a division, no condition per value inside a row.  A second workgroup on a CU
// instead of the next row's loads in flight is slower (279 us: 128 registers spill),
// so are two rows at a time (158).

struct ResNormBackArgs {
    const void *dr, *dy, *r, *h, *gate, *weight, *post_weight;  // null: absent (dr: zeros)
    const float *mean, *rstd, *post_mean, *post_rstd;
    void *dx, *dh, *dgate;            // dh null: no block before the norm
    int64_t lddr, lddy, ldr, ldh, ldg, lddx, lddh, lddg;
    int M, D;
    int gate_rows;                    // rows of a group: those that share a row of the gate, or all
    int groups, chunks;               // groups; workgroups of a group (1: a workgroup takes every so many groups)
    float alpha, d, inv_d;
    float *part;                      // [workgroup][4][part_ld]: dweight, dbias, dpost_weight, dgate; null: not computed
    int64_t part_ld;
    float2 *row_sums;                 // residual_norm_backward_any_kernel: both means of a row's first norm
};

// A thread group has the next row's loads in flight (AHEAD).  Between its steps it
// keeps a row as it lies in memory and widens it again: the values in 32 bits would
// take twice the registers.
template <typename T>
__device__ __forceinline__ void as_in_memory(Raw8<T> &r)
{
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
        asm volatile("" : "+v"(r.w[i]));
}

template <typename T, int P, int V, bool AHEAD, int OCC, bool TAIL, bool RMS, bool POST>
__global__ __launch_bounds__(norm_threads(P), OCC) void residual_norm_backward_kernel(const ResNormBackArgs a)
{
    constexpr int RPW = norm_threads(P) / P;
    constexpr int NW = P > 64 ? P / 64 : 1;
    constexpr int NS = POST ? 4 : 3;      // sums: dweight, dbias, dgate, dpost_weight
    __shared__ __attribute__((aligned(16))) float red[2][NW][4];
    __shared__ float cs[RPW > 1 ? RPW : 1][RPW > 1 ? P * 8 : 1];
    const int t = threadIdx.x % P, sub = RPW > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / P) : 0;
    const bool use_h = POST || a.gate;

    Raw8<T> w[V], pw[V], g[V];
    load_params<T, P, V>((const T *)a.weight, 1.0f, a.D, t, w);
    if constexpr (POST)
        load_params<T, P, V>((const T *)a.post_weight, 1.0f, a.D, t, pw);
    float sum[NS][V][8];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum[s][i][k] = 0.0f;

    // Sum s over the workgroup's rows: f(column, how many of the values exist, values), each column once.
    auto emit = [&](auto sc, auto f) __attribute__((always_inline)) {
        constexpr int s = decltype(sc)::value;
        if constexpr (RPW > 1) {
            for_each<V>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    cs[sub][k * P + t] = sum[s][i][k];
                __syncthreads();
                for (int e = threadIdx.x; e < P * 8; e += norm_threads(P)) {
                    const int col = i * P * 8 + e, src = (e & 7) * P + (e >> 3);
                    float v[1] = {0.0f};
#pragma unroll
                    for (int r = 0; r < RPW; ++r)
                        v[0] += cs[r][src];
                    if (col < a.D)
                        f(col, 1, v);
                }
            });
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                f((i * P + t) * 8, a.D - (i * P + t) * 8, sum[s][i]);
        }
    };

    struct Row {
        Raw8<T> r[V], dy[V], dr[V], h[V];
        float mean, rstd, post_mean, post_rstd;
    } ring;
    auto load = [&](int64_t m) __attribute__((always_inline)) {
        load_row<T, P, V>((const T *)a.r + m * a.ldr, a.D, t, ring.r);
        load_row<T, P, V>((const T *)a.dy + m * a.lddy, a.D, t, ring.dy);
        if (a.dr)
            load_row<T, P, V>((const T *)a.dr + m * a.lddr, a.D, t, ring.dr);
        if (use_h)
            load_row<T, P, V>((const T *)a.h + m * a.ldh, a.D, t, ring.h);
        ring.rstd = a.rstd[m];
        ring.mean = RMS ? 0.0f : a.mean[m];
        if constexpr (POST) {
            ring.post_rstd = a.post_rstd[m];
            ring.post_mean = RMS ? 0.0f : a.post_mean[m];
        }
    };
    int set = 0;
    // Both sums of a lane's numbers over a row's threads, as means.  A wave folds them into one register
    // first, so that two sums cost little more than one.
    auto means = [&](float &s1, float &s2) __attribute__((always_inline)) {
        // lanes 0 to 31 hold s1's parts, 32 to 63 s2's
        const float v = row16_sum(fold_halves(s1, s2, [](float x, float y) { return x + y; }));
        float r[4];
        if constexpr (P > 64) {
            if ((threadIdx.x & 15) == 0)
                red[set][threadIdx.x >> 6][(threadIdx.x >> 4) & 3] = v;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                r[q] = red[set][0][q];
#pragma unroll
            for (int i = 1; i < NW; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    r[q] += red[set][i][q];
            set ^= 1;  // the other set: a slow wave may still read this one
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                r[q] = lane_value(v, 16 * q);
        }
        s1 = RMS ? 0.0f : (r[0] + r[1]) * a.inv_d;
        s2 = (r[2] + r[3]) * a.inv_d;
    };
    // (v - mean) rstd of group i, 0 past the row's end, also where mean rstd is infinite
    auto normed = [&](const Raw8<T> &raw, int i, float mean, float rstd, float (&v)[8]) __attribute__((always_inline)) {
        widen_group<TAIL, P>(raw, a.D, i, t, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = (v[k] - mean) * rstd;
        if ((i + 1) * P * 8 > a.D) {
            asm volatile("");  // keeps the branch
            const int cnt = a.D - (i * P + t) * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = (TAIL ? k < cnt : cnt > 0) ? v[k] : 0.0f;
        }
    };

    const int step = RPW * a.chunks;
    for (int grp = blockIdx.x / a.chunks; grp < a.groups; grp += gridDim.x / a.chunks) {
        const int64_t base = (int64_t)grp * a.gate_rows, m1 = base + a.gate_rows;
        const int64_t m0 = base + blockIdx.x % a.chunks * RPW + sub;
        if (a.gate)
            load_row<T, P, V>((const T *)a.gate + (int64_t)grp * a.ldg, a.D, t, g);
        if (AHEAD && m0 < m1)
            load(m0);
        for (int64_t m = m0; m < m1; m += step) {
            if constexpr (!AHEAD)
                load(m);
            Row cur = ring;
            if (AHEAD && m + step < m1)
                load(m + step);
            float s1 = 0.0f, s2 = 0.0f, p1 = 0.0f, p2 = 0.0f, e[V][8];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float wv[8], dy[8], rh[8];
                as_in_memory(w[i]);
                widen_group<TAIL, P>(w[i], a.D, i, t, wv);
                widen_group<TAIL, P>(cur.dy[i], a.D, i, t, dy);
                normed(cur.r[i], i, cur.mean, cur.rstd, rh);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float c = dy[k] * wv[k];
                    s1 += c;
                    s2 = __builtin_fmaf(c, rh[k], s2);
                    sum[0][i][k] = __builtin_fmaf(dy[k], rh[k], sum[0][i][k]);
                    sum[1][i][k] += dy[k];
                }
            }
            means(s1, s2);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = (i * P + t) * 8, cnt = a.D - at;
                const bool whole = (i + 1) * P * 8 <= a.D;
                auto put = [&](void *p, int64_t ld, const float (&o)[8]) __attribute__((always_inline)) {
                    T *q = (T *)p + m * ld + at;
                    if (whole || (!TAIL && cnt > 0))
                        store_all(q, o);
                    else if constexpr (TAIL)
                        store_n(q, cnt, o);
                };
                float tv[8], o[8], wv[8], rh[8];
                as_in_memory(w[i]);
                as_in_memory(cur.r[i]);
                as_in_memory(cur.dy[i]);
                widen_group<TAIL, P>(w[i], a.D, i, t, wv);
                widen_group<TAIL, P>(cur.dy[i], a.D, i, t, tv);
                normed(cur.r[i], i, cur.mean, cur.rstd, rh);
                if (a.dr) {
                    widen_group<TAIL, P>(cur.dr[i], a.D, i, t, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    tv[k] = __builtin_fmaf(tv[k], wv[k], -s1);
                    tv[k] = __builtin_fmaf(cur.rstd, __builtin_fmaf(-rh[k], s2, tv[k]), o[k]);
                    o[k] = a.alpha * tv[k];
                }
                put(a.dx, a.lddx, o);
                if (!a.dh)
                    continue;
                if (!whole) {  // what mean(c) leaves past the row's end
                    asm volatile("");
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tv[k] = (TAIL ? k < cnt : cnt > 0) ? tv[k] : 0.0f;
                }
                float hh[8], gv[8], pv[8];
                if constexpr (POST) {
                    normed(cur.h[i], i, cur.post_mean, cur.post_rstd, hh);
                    as_in_memory(pw[i]);
                    widen_group<TAIL, P>(pw[i], a.D, i, t, pv);
                } else if (use_h) {
                    widen_group<TAIL, P>(cur.h[i], a.D, i, t, hh);
                }
                if (a.gate) {
                    as_in_memory(g[i]);
                    widen_group<TAIL, P>(g[i], a.D, i, t, gv);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        sum[2][i][k] = __builtin_fmaf(tv[k], POST ? hh[k] * pv[k] : hh[k], sum[2][i][k]);
                        tv[k] *= gv[k];  // u
                    }
                }
                if constexpr (POST) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        sum[NS - 1][i][k] = __builtin_fmaf(tv[k], hh[k], sum[NS - 1][i][k]);
                        e[i][k] = tv[k] * pv[k];
                        p1 += e[i][k];
                        p2 = __builtin_fmaf(e[i][k], hh[k], p2);
                    }
                } else {
                    put(a.dh, a.lddh, tv);
                }
            }
            if constexpr (POST) {
                means(p1, p2);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int at = (i * P + t) * 8;
                    float o[8], hh[8];
                    as_in_memory(cur.h[i]);
                    normed(cur.h[i], i, cur.post_mean, cur.post_rstd, hh);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = cur.post_rstd * (e[i][k] - p1 - hh[k] * p2);
                    T *q = (T *)a.dh + m * a.lddh + at;
                    if ((i + 1) * P * 8 <= a.D || (!TAIL && at < a.D))
                        store_all(q, o);
                    else if constexpr (TAIL)
                        store_n(q, a.D - at, o);
                }
            }
        }
        if (a.dgate && a.chunks == 1) {
            emit(Size<2>{}, [&](int col, int n, const auto &v) { store_n((T *)a.dgate + grp * a.lddg + col, n, v); });
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sum[2][i][k] = 0.0f;
        }
    }
    if (!a.part)
        return;
    float *p = a.part + (int64_t)blockIdx.x * 4 * a.part_ld;
    emit(Size<0>{}, [&](int col, int n, const auto &v) { store_n(p + col, n, v); });
    emit(Size<1>{}, [&](int col, int n, const auto &v) { store_n(p + a.part_ld + col, n, v); });
    if constexpr (POST)
        emit(Size<3>{}, [&](int col, int n, const auto &v) { store_n(p + 2 * a.part_ld + col, n, v); });
    if (a.dgate && a.chunks > 1)
        emit(Size<2>{}, [&](int col, int n, const auto &v) { store_n(p + 3 * a.part_ld + col, n, v); });
}

// Rows of any other length: dx and dh, with the row read again for each step ...
template <typename T, int P, bool RMS, bool POST>
__global__ __launch_bounds__(P) void residual_norm_backward_any_kernel(const ResNormBackArgs a)
{
    constexpr int NW = P > 64 ? P / 64 : 1;
    __shared__ float red[4 * NW];  // a set's next use comes after another set's barrier
    const int t = threadIdx.x;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const float mean = RMS ? 0.0f : a.mean[m], rstd = a.rstd[m];
        const float post_mean = RMS || !POST ? 0.0f : a.post_mean[m], post_rstd = POST ? a.post_rstd[m] : 0.0f;
        const T *gate = a.gate ? (const T *)a.gate + m / a.gate_rows * a.ldg : nullptr;
        auto load = [&](int64_t c, int cnt, float (&rh)[8], float (&cv)[8]) {
            float w[8];
            load_n((const T *)a.r + m * a.ldr + c, cnt, rh, mean);
            load_n((const T *)a.dy + m * a.lddy + c, cnt, cv);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k] = 1.0f;
            if (a.weight)
                load_n((const T *)a.weight + c, cnt, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                rh[k] = (rh[k] - mean) * rstd;
                cv[k] *= w[k];
            }
        };
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = t * 8; c < a.D; c += P * 8) {
            float rh[8], cv[8];
            load(c, (int)(a.D - c), rh, cv);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s1 += cv[k];
                s2 = __builtin_fmaf(cv[k], rh[k], s2);
            }
        }
        s1 = row_reduce<P>(s1, red, 0) / a.d;
        s2 = row_reduce<P>(s2, red, 1) / a.d;
        if (RMS)
            s1 = 0.0f;
        if (t == 0 && a.row_sums)
            a.row_sums[m] = make_float2(s1, s2);
        // t of eight columns, and (e, hh) where there is a norm of h
        auto through = [&](int64_t c, int cnt, float (&tv)[8], float (&hh)[8]) {
            float rh[8], dr[8] = {};
            load(c, cnt, rh, tv);
            if (a.dr)
                load_n((const T *)a.dr + m * a.lddr + c, cnt, dr);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                tv[k] = rstd * (tv[k] - s1 - rh[k] * s2) + dr[k];
            if constexpr (POST) {
                load_n((const T *)a.h + m * a.ldh + c, cnt, hh, post_mean);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    hh[k] = (hh[k] - post_mean) * post_rstd;
            }
        };
        auto gated = [&](int64_t c, int cnt, float (&v)[8]) {
            float p[8];
            if (gate) {
                load_n(gate + c, cnt, p);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] *= p[k];
            }
            if constexpr (POST) {
                load_n((const T *)a.post_weight + c, cnt, p);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = k < cnt ? v[k] * p[k] : 0.0f;
            }
        };
        float p1 = 0.0f, p2 = 0.0f;
        for (int64_t c = t * 8; c < a.D; c += P * 8) {
            const int cnt = (int)(a.D - c);
            float v[8], hh[8], o[8];
            through(c, cnt, v, hh);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k] = a.alpha * v[k];
            store_n((T *)a.dx + m * a.lddx + c, cnt, o);
            if (!a.dh)
                continue;
            gated(c, cnt, v);
            if constexpr (POST) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    p1 += v[k];
                    p2 = __builtin_fmaf(v[k], hh[k], p2);
                }
            } else {
                store_n((T *)a.dh + m * a.lddh + c, cnt, v);
            }
        }
        if constexpr (POST) {
            p1 = row_reduce<P>(p1, red, 2) / a.d;
            p2 = row_reduce<P>(p2, red, 3) / a.d;
            if (RMS)
                p1 = 0.0f;
            for (int64_t c = t * 8; c < a.D; c += P * 8) {
                const int cnt = (int)(a.D - c);
                float v[8], hh[8];
                through(c, cnt, v, hh);
                gated(c, cnt, v);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = post_rstd * (v[k] - p1 - hh[k] * p2);
                store_n((T *)a.dh + m * a.lddh + c, cnt, v);
            }
        }
    }
}

// ... and the columns' sums of the rows of workgroup blockIdx.y of the kernel above,
// 2048 columns a workgroup here.  Both read every operand, so that a call with a norm
// of h takes 410 us for 4096 x 12288 BF16 (its 604 MB once: 112 at a copy's rate) and
// 486 for 4096 x 16384.
template <typename T, bool RMS, bool POST>
__global__ __launch_bounds__(256) void residual_norm_columns_kernel(const ResNormBackArgs a)
{
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    const int cnt = (int)(a.D - c);
    if (cnt <= 0)
        return;
    const int wg = blockIdx.y;
    float w[8], pw[8], sum[4][8] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        w[k] = 1.0f;
    if (a.weight)
        load_n((const T *)a.weight + c, cnt, w);
    if constexpr (POST)
        load_n((const T *)a.post_weight + c, cnt, pw);
    for (int grp = wg / a.chunks; grp < a.groups; grp += gridDim.y / a.chunks) {
        const int64_t base = (int64_t)grp * a.gate_rows, m1 = base + a.gate_rows;
        float g[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            g[k] = 1.0f;
        if (a.gate)
            load_n((const T *)a.gate + (int64_t)grp * a.ldg + c, cnt, g);
        for (int64_t m = base + wg % a.chunks; m < m1; m += a.chunks) {
            const float mean = RMS ? 0.0f : a.mean[m], rstd = a.rstd[m];
            const float2 s = a.row_sums[m];
            float r[8], dy[8], dr[8] = {}, h[8] = {};
            load_n((const T *)a.r + m * a.ldr + c, cnt, r);
            load_n((const T *)a.dy + m * a.lddy + c, cnt, dy);
            if (a.dr)
                load_n((const T *)a.dr + m * a.lddr + c, cnt, dr);
            if (POST || a.gate)
                load_n((const T *)a.h + m * a.ldh + c, cnt, h);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float rh = (r[k] - mean) * rstd;
                sum[0][k] = __builtin_fmaf(dy[k], rh, sum[0][k]);
                sum[1][k] += dy[k];
                const float tv = rstd * (dy[k] * w[k] - s.x - rh * s.y) + dr[k];
                if constexpr (POST) {
                    const float hh = (h[k] - (RMS ? 0.0f : a.post_mean[m])) * a.post_rstd[m];
                    sum[2][k] = __builtin_fmaf(g[k] * tv, hh, sum[2][k]);
                    sum[3][k] = __builtin_fmaf(tv, hh * pw[k], sum[3][k]);
                } else {
                    sum[3][k] = __builtin_fmaf(tv, h[k], sum[3][k]);
                }
            }
        }
        if (a.dgate && a.chunks == 1) {
            store_n((T *)a.dgate + (int64_t)grp * a.lddg + c, cnt, sum[3]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum[3][k] = 0.0f;
        }
    }
    if (!a.part)
        return;
    float *p = a.part + (int64_t)wg * 4 * a.part_ld + c;
#pragma unroll
    for (int s = 0; s < 4; ++s)
        store_n(p + s * a.part_ld, cnt, sum[s]);
}

}  // namespace dense
