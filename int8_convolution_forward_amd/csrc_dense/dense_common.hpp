// Shared pieces of the dense layer's and layer norm's kernels for gfx950:
// element types, unaligned 16-byte loads and stores, activations and their
// slopes, direct-to-LDS loads, wave reductions and the tile order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense.h"

namespace dense {

typedef __bf16 bf16;
typedef _Float16 f16;
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kCUs = 256;
// Buffer offset outside every resource (ranges stay below 2^31): a load from
// it returns zeros.
constexpr int kOutOfRange = (int)0x80000000u;

template <typename T> struct Code;
template <> struct Code<int8_t> { static constexpr int v = DENSE_INT8; };
template <> struct Code<bf16> { static constexpr int v = DENSE_BF16; };
template <> struct Code<f16> { static constexpr int v = DENSE_FP16; };
template <> struct Code<float> { static constexpr int v = DENSE_FP32; };

// C values at any element-aligned address.  gfx950 runs with unaligned vector
// access enabled, so 16 bytes are one instruction whatever the address; an
// address that is a multiple of 16 costs nothing extra.
template <typename T, int C>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
    T e[C];
};

template <typename T, int C>
__device__ __forceinline__ void load_all(const T *p, float (&v)[C])
{
    const Pack<T, C> q = *(const Pack<T, C> *)p;
#pragma unroll
    for (int i = 0; i < C; ++i)
        v[i] = (float)q.e[i];
}

// Eight values as they lie in memory, so that what is on its way takes the
// registers of its type and not of 32-bit values.
template <typename T>
struct Raw8 {
    v4i w[sizeof(T) / 2];
};

// Values c .. c+7 of a row of D >= 8.  Past the end, and for a partial group, it
// reads the last eight of the row, which widen_part puts in their place: a load
// has no condition per lane, so nothing waits for it before it is used.
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *row, int c, int D)
{
    return __builtin_bit_cast(Raw8<T>, *(const Pack<T, 8> *)(row + min(c, D - 8)));
}

template <typename T>
__device__ __forceinline__ void widen(const Raw8<T> &r, float (&v)[8])
{
    typedef T vec __attribute__((ext_vector_type(8)));
    const vec q = __builtin_bit_cast(vec, r);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = (float)q[k];
}

// The same where only D - c of the values may exist: the others become zero.
// TAIL: D may be other than a multiple of eight.
template <bool TAIL, typename T>
__device__ __forceinline__ void widen_part(const Raw8<T> &r, int c, int D, float (&v)[8])
{
    widen(r, v);
    const int n = D - c;
    if constexpr (TAIL) {
        if (n < 8) {
            asm volatile("");  // keeps the branch: as selects, every lane would pay for them
            const int by = 8 - n;  // down by so many places
#pragma unroll
            for (int b = 4; b >= 1; b >>= 1)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = by & b ? (k + b < 8 ? v[k + b] : 0.0f) : v[k];
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = n > 0 ? v[k] : 0.0f;
}

template <typename T, int C>
__device__ __forceinline__ void store_all(T *p, const float (&v)[C])
{
    Pack<T, C> q;
#pragma unroll
    for (int i = 0; i < C; ++i)
        q.e[i] = (T)v[i];
    *(Pack<T, C> *)p = q;
}

// The first n of C values (n may be C or more); the others read as `fill`.
template <typename T, int C>
__device__ __forceinline__ void load_n(const T *p, int n, float (&v)[C], float fill = 0.0f)
{
    if (n >= C) {
        load_all(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            v[i] = i < n ? (float)p[i] : fill;
    }
}

template <typename T, int C>
__device__ __forceinline__ void store_n(T *p, int n, const float (&v)[C])
{
    if (n >= C) {
        store_all(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < n)
                p[i] = (T)v[i];
    }
}

// The same with the element type given at run time (uniform over the launch).
template <int C>
__device__ __forceinline__ void load_n_dt(const void *p, int dt, int64_t off, int n, float (&v)[C])
{
    if (dt == DENSE_BF16)
        load_n((const bf16 *)p + off, n, v);
    else if (dt == DENSE_FP16)
        load_n((const f16 *)p + off, n, v);
    else
        load_n((const float *)p + off, n, v);
}

template <int C>
__device__ __forceinline__ void store_n_dt(void *p, int dt, int64_t off, int n, const float (&v)[C])
{
    if (dt == DENSE_BF16)
        store_n((bf16 *)p + off, n, v);
    else if (dt == DENSE_FP16)
        store_n((f16 *)p + off, n, v);
    else
        store_n((float *)p + off, n, v);
}

__device__ __forceinline__ float load_dt(const void *p, int dt, int64_t i)
{
    return dt == DENSE_BF16 ? (float)((const bf16 *)p)[i]
         : dt == DENSE_FP16 ? (float)((const f16 *)p)[i]
                            : ((const float *)p)[i];
}

__device__ __forceinline__ void store_dt(void *p, int dt, int64_t i, float v)
{
    if (dt == DENSE_BF16)
        ((bf16 *)p)[i] = (bf16)v;
    else if (dt == DENSE_FP16)
        ((f16 *)p)[i] = (f16)v;
    else
        ((float *)p)[i] = v;
}

template <int N> struct Size { static constexpr int value = N; };

// f(Size<0>) .. f(Size<N-1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F f)
{
    if constexpr (I < N) {
        f(Size<I>{});
        for_each<N, I + 1>(f);
    }
}

// 16x16 matrix product of 64 bytes of the inner dimension: lane l gives row
// l % 16 of each operand at bytes 16 (l / 16), and holds column l % 16 (the
// second operand's row), rows 4 (l / 16) .. +3 of the result.
template <typename T> struct Acc4 { typedef v4f type; };
template <> struct Acc4<int8_t> { typedef v4i type; };

template <typename T>
__device__ __forceinline__ typename Acc4<T>::type mfma16(v4i a, v4i b, typename Acc4<T>::type c)
{
    if constexpr (sizeof(T) == 1)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    else if constexpr (__is_same(T, bf16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 1 / (1 + exp(-x)) from the hardware's exp2 and reciprocal (1 ulp each; the
// product with log2 e costs |x| 2^-24 relative, far below a 16-bit rounding).
// exp2 overflows to infinity and its reciprocal to 0, so both tails are exact.
__device__ __forceinline__ float sigmoid(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896f * x));
}

constexpr float kGeluC = 0.797884560802865f;   // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;
constexpr float kGeluE1 = -2.302208198144325f;  // -2 sqrt(2/pi) log2 e
constexpr float kGeluE3 = -0.102943239579983f;  // kGeluA times it
constexpr float kInvSqrt2Pi = 0.398942280401433f;

// 0.5 (1 + tanh u) = sigmoid(2u), so the tanh form of gelu is z sigmoid(2u).
// z2 is z^2; the constants of u and of the exponential are one, because the
// epilogue's arithmetic is not hidden by anything (7 operations a value).
__device__ __forceinline__ float gelu_tanh_gate(float z, float z2)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * __builtin_fmaf(z2, kGeluE3, kGeluE1)));
}

// exp(-z^2/2) and the normal distribution function.  With t = 1 / (1 + c |z|) the
// lower tail is t Q(t) exp(-z^2/2): Q, of degree 9, is a fit to
// exp(z^2/2) cdf(-|z|) / t with the least relative error over all z: 2^-24.5 with
// the constants as written, 2^-24.2 once they are rounded to 32 bits.
// Rounded to 32 bits everything is within 3 2^-24, and the tail keeps its
// relative precision (11 2^-24 down to z = -3; the rounding of z^2 in the
// exponent).  About 20 operations, where the library's erfc takes several times
// as many and branches.
__device__ __forceinline__ float normal_cdf(float z, float &bell)
{
    bell = __builtin_amdgcn_exp2f(-0.72134752044448f * (z * z));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 3.181980550e-01f, 1.0f));
    float q = -2.069549154e-02f;
    q = __builtin_fmaf(q, t, 9.534367189e-02f);
    q = __builtin_fmaf(q, t, -1.502907509e-01f);
    q = __builtin_fmaf(q, t, 7.120001795e-02f);
    q = __builtin_fmaf(q, t, -1.117871554e-02f);
    q = __builtin_fmaf(q, t, 5.997513579e-02f);
    q = __builtin_fmaf(q, t, 8.762607770e-02f);
    q = __builtin_fmaf(q, t, 1.141358198e-01f);
    q = __builtin_fmaf(q, t, 1.269415814e-01f);
    q = __builtin_fmaf(q, t, 1.269426604e-01f);
    const float tail = t * q * bell;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == DENSE_ACT_RELU)
        return z < 0.0f ? 0.0f : z;  // keeps a NaN
    else if constexpr (ACT == DENSE_ACT_GELU) {
        float bell;
        return z * normal_cdf(z, bell);
    } else if constexpr (ACT == DENSE_ACT_GELU_TANH)
        return z * gelu_tanh_gate(z, z * z);
    else if constexpr (ACT == DENSE_ACT_SILU)
        return z * sigmoid(z);
    else
        return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == DENSE_ACT_RELU) {
        return z > 0.0f ? 1.0f : z == z ? 0.0f : z;
    } else if constexpr (ACT == DENSE_ACT_GELU) {
        float bell;
        const float cdf = normal_cdf(z, bell);
        return __builtin_fmaf(z * kInvSqrt2Pi, bell, cdf);
    } else if constexpr (ACT == DENSE_ACT_GELU_TANH) {
        // p + z p (1 - p) 2u'(z); z^2 is bounded where p (1 - p) is already 0,
        // so that it cannot overflow against it
        const float z2 = fminf(z * z, 1.0e4f);
        const float p = gelu_tanh_gate(z, z2);
        return __builtin_fmaf(z * p * (1.0f - p), __builtin_fmaf(z2, 6.0f * kGeluC * kGeluA, 2.0f * kGeluC), p);
    } else if constexpr (ACT == DENSE_ACT_SILU) {
        const float p = sigmoid(z);
        return p * (1.0f + z * (1.0f - p));
    } else {
        return 1.0f;
    }
}

template <int U, int C>
__device__ __forceinline__ void activate_all(int act, float (&v)[U][C])
{
    auto all = [&](auto f) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i)
                v[u][i] = f(v[u][i]);
    };
    if (act == DENSE_ACT_RELU)
        all([](float z) { return activate<DENSE_ACT_RELU>(z); });
    else if (act == DENSE_ACT_GELU)
        all([](float z) { return activate<DENSE_ACT_GELU>(z); });
    else if (act == DENSE_ACT_GELU_TANH)
        all([](float z) { return activate<DENSE_ACT_GELU_TANH>(z); });
    else if (act == DENSE_ACT_SILU)
        all([](float z) { return activate<DENSE_ACT_SILU>(z); });
}

__device__ __forceinline__ float activate_rt(int act, float z)
{
    return act == DENSE_ACT_RELU        ? activate<DENSE_ACT_RELU>(z)
         : act == DENSE_ACT_GELU        ? activate<DENSE_ACT_GELU>(z)
         : act == DENSE_ACT_GELU_TANH   ? activate<DENSE_ACT_GELU_TANH>(z)
         : act == DENSE_ACT_SILU        ? activate<DENSE_ACT_SILU>(z)
                                        : z;
}

// Chunk permutation of an LDS row of SB bytes.  16 rows that read one
// chunk cover the 64 banks once: four 64-byte or two 128-byte rows make up the
// banks' 256 bytes, and the permutation differs between those that coincide.
template <int SB>
__device__ __forceinline__ int row_swizzle(int row, int chunk)
{
    return SB == 64 ? chunk ^ (((row >> 1) ^ (row >> 2)) & 3) : chunk ^ ((row >> 1) & 7);
}

// s_waitcnt immediate (gfx9 encoding): at most VM vector-memory operations
// outstanding, all LDS operations done.
template <int VM>
__device__ __forceinline__ void wait_vm_lgkm0()
{
    static_assert(VM >= 0 && VM < 64, "vmcnt out of range");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (0 << 8));
}

// All LDS operations done, any number of vector-memory operations outstanding.
__device__ __forceinline__ void wait_lgkm0()
{
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));
}

// Buffer resource (gfx9 layout): base address, stride 0, byte range, 32-bit
// data format.  Built from uniform values.
__device__ __forceinline__ v4i make_rsrc(const void *p, int range)
{
    const unsigned long long a = (unsigned long long)p;
    v4i d;
    d.x = (int)(unsigned)a;
    d.y = (int)((a >> 32) & 0xFFFFu);
    d.z = range;
    d.w = 0x00020000;
    return d;
}

// A load of 16 bytes per lane from buffer offset `voff` straight into LDS, lane
// i's bytes to M0 + 16*i, and the write of M0 that comes before it (with at
// least one other instruction between them: M0 needs a wait state).  An offset
// outside the range writes zeros.  The compiler does not see these loads, so
// the kernel counts them itself with s_waitcnt vmcnt; nothing between the two
// may use M0.
template <int OFFSET>
__device__ __forceinline__ void set_lds_target(unsigned lds_base)
{
    asm volatile("s_add_u32 m0, %0, %1" :: "s"(lds_base), "n"(OFFSET) : "m0", "scc");
}

__device__ __forceinline__ void load16_to_lds(v4i rsrc, int voff)
{
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" :: "v"(voff), "s"(rsrc) : "memory");
}

__device__ __forceinline__ unsigned lds_address(const void *p)
{
    return (unsigned)(unsigned long long)(lds_void *)p;
}

// Another lane's value, by a lane permutation that costs no trip through LDS
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xf, 0xf, false));
}

__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// f over the 64 lanes of a wave, the result in all of them: neighbours, pairs,
// halves of eight and of sixteen lanes exchanged, then the four rows of sixteen.
// (By shuffles, which go through LDS, a layer norm of 4096 columns spends more
// time on its reductions than on its arithmetic.)
template <typename F>
__device__ __forceinline__ float wave_reduce(float v, F f)
{
    v = f(v, dpp<0xB1>(v));   // lanes 1 0 3 2 of each four
    v = f(v, dpp<0x4E>(v));   // lanes 2 3 0 1
    v = f(v, dpp<0x141>(v));  // eight lanes mirrored
    v = f(v, dpp<0x140>(v));  // sixteen lanes mirrored
    return f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
}

__device__ __forceinline__ float wave_sum(float v)
{
    return wave_reduce(v, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// Workgroups are dealt round-robin to the 8 XCDs; each XCD gets one contiguous
// run of tiles.
__device__ __forceinline__ int xcd_tile(int bid, int tiles)
{
    const int per = tiles >> 3, rem = tiles & 7;
    const int xcd = bid & 7, idx = bid >> 3;
    return xcd * per + min(xcd, rem) + idx;
}

// Epilogue of one product (linear's, or a plain store for the gradients).
struct Epilogue {
    void *out;
    const void *residual;
    void *preact;
    const void *bias;
    const float *x_scale, *w_scale;
    int64_t ldo, ldr, ldp;  // row strides in elements
    int out_dt;             // of out, residual and preact
    int bias_dt;
    int act;
    int tile_offsets;       // 256 rows of every matrix above span less than 2^31 bytes
};

// The epilogue of U chunks of C columns, of which n .. n+cnt-1 exist, chunk u in row
// m + u*step: v holds the products' sums, ws and bs the columns' scales and
// biases.  Rows from M on are skipped.  All residuals are loaded first, so that
// their latencies overlap.
template <bool SCALED, int U, int C>
__device__ __forceinline__ void finish(const Epilogue &e, int64_t m, int step, int64_t M, int64_t n, int cnt,
                                       float (&v)[U][C], const float (&bs)[C], const float (&ws)[C])
{
    float r[U][C];
    if (e.residual) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (m + u * step < M)
                load_n_dt(e.residual, e.out_dt, (m + u * step) * e.ldr + n, cnt, r[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (SCALED) {
            const float xs = e.x_scale && m + u * step < M ? e.x_scale[m + u * step] : 1.0f;
#pragma unroll
            for (int i = 0; i < C; ++i)
                v[u][i] = __builtin_fmaf(v[u][i], xs * ws[i], bs[i]);
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
                v[u][i] += bs[i];
        }
    }
    if (e.preact) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (m + u * step < M)
                store_n_dt(e.preact, e.out_dt, (m + u * step) * e.ldp + n, cnt, v[u]);
    }
    activate_all(e.act, v);
    if (e.residual) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i)
                v[u][i] += r[u][i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (m + u * step < M)
            store_n_dt(e.out, e.out_dt, (m + u * step) * e.ldo + n, cnt, v[u]);
}

// Scales and biases of columns n .. n+cnt-1 (ones and zeros where absent).
template <int C>
__device__ __forceinline__ void column_params(const Epilogue &e, int64_t n, int cnt, float (&bs)[C], float (&ws)[C])
{
#pragma unroll
    for (int i = 0; i < C; ++i) {
        bs[i] = 0.0f;
        ws[i] = 1.0f;
    }
    if (e.bias)
        load_n_dt(e.bias, e.bias_dt, n, cnt, bs);
    if (e.w_scale)
        load_n(e.w_scale + n, cnt, ws);
}

}  // namespace dense
