// Rows of 8-bit floating point with a scale for each block of 128: quantising,
// with the slope of an activation and the transposed copy where they are wanted,
// and back.
//
// A scale is 2^e, kept as the byte e + 127.  Multiplying by 2^-e is exact, so a
// value is rounded once, by the instruction that converts it, and a block's scale
// follows from the bits of its largest magnitude: no division, and the same bytes
// in whatever precision it is computed.
//
// All are bound by HBM, which takes reads and writes together at 5.4 to 5.9 TB/s here
// (a copy of 256 and of 134 MB); times are given at each kernel.
#pragma once

#include "rows_kernel.hpp"

namespace dense {

// The byte of the least scale with which magnitudes up to `top` stay in range:
// 448 = 1.75 2^8 for e4m3, 57344 = 1.75 2^15 for e5m2.
__device__ __forceinline__ int scale_byte(float top, bool e5)
{
    const int bits = __builtin_bit_cast(int, top);
    return max((bits >> 23) - (e5 ? 15 : 8) + ((bits & 0x7fffff) > 0x600000), 0);
}

// 2^-e for the scale's byte (0 .. 247), a normal number
__device__ __forceinline__ float inverse_scale(int byte) { return __builtin_bit_cast(float, (254 - byte) << 23); }

// The magnitude that counts for a scale: 0 for what is not finite
__device__ __forceinline__ float finite_size(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; }

// Four values times `inv`, rounded half to even; what is not finite becomes NaN
__device__ __forceinline__ int encode4(float v0, float v1, float v2, float v3, float inv, bool e5)
{
    auto scaled = [&](float v) { return fabsf(v) < INFINITY ? v * inv : __builtin_nanf(""); };
    const float s0 = scaled(v0), s1 = scaled(v1), s2 = scaled(v2), s3 = scaled(v3);
    return e5 ? __builtin_amdgcn_cvt_pk_bf8_f32(s2, s3, __builtin_amdgcn_cvt_pk_bf8_f32(s0, s1, 0, false), true)
              : __builtin_amdgcn_cvt_pk_fp8_f32(s2, s3, __builtin_amdgcn_cvt_pk_fp8_f32(s0, s1, 0, false), true);
}

__device__ __forceinline__ Pack<uint8_t, 8> encode8(const float (&v)[8], float inv, bool e5)
{
    typedef int v2i __attribute__((ext_vector_type(2)));
    const v2i w = {encode4(v[0], v[1], v[2], v[3], inv, e5), encode4(v[4], v[5], v[6], v[7], inv, e5)};
    return __builtin_bit_cast(Pack<uint8_t, 8>, w);
}

// The first n of eight bytes
__device__ __forceinline__ void store_bytes(uint8_t *p, int n, const Pack<uint8_t, 8> &q)
{
    if (n >= 8) {
        *(Pack<uint8_t, 8> *)p = q;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n)
                p[k] = q.e[k];
    }
}

// Largest of the sixteen lanes that hold a block of a row, in all of them
__device__ __forceinline__ float block_max(float v)
{
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    return fmaxf(v, dpp<0x140>(v));
}

struct QuantArgs {
    const void *x, *z;        // z: where the values are x act'(z)
    int64_t ldx, ldz;
    int M, K;
    int strips, blocks;       // workgroups along a row, and of all rows
    bool e5, tiles, tiles_t;
    uint8_t *q, *scale;       // null: not written
    int64_t ldq, lds;
    int q_cols;               // columns of q that are written: K, or more as zeros
    uint8_t *qt, *scale_t;
    int64_t ldqt, ldst;
    int qt_cols;
    float *colsum;            // [row of tiles][sum_ld], or null: sums of the tile's columns
    int64_t sum_ld;
};

// Rows of 1 x 128 blocks: a wave takes 512 columns of four rows, eight a lane, so
// that sixteen lanes hold a block.  Four rows' loads are in flight at once.  Without
// a transposed copy or tiles nothing passes between waves, so this takes the place
// of the kernel below, with its barriers and LDS.  8192 x 8192 BF16: 36 us (202 MB, 5.6 TB/s);
// 16 x 4096, 64 x 8192 and 777 x 1032 3.9 to 4.4, a launch.
template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantArgs a)
{
    constexpr int U = 4;
    const int rb = blockIdx.x / a.strips, strip = blockIdx.x - rb * a.strips;
    const int lane = threadIdx.x & 63, c = strip * 512 + lane * 8, cnt = a.K - c;
    const int m0 = (rb * 4 + (threadIdx.x >> 6)) * U;
    float v[U][8];
    if (a.K >= 8) {
        Raw8<T> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            r[u] = load_raw((const T *)a.x + (int64_t)min(m0 + u, a.M - 1) * a.ldx, c, a.K);
        if (strip * 512 + 512 <= a.K) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                widen(r[u], v[u]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                widen_part<true>(r[u], c, a.K, v[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_n((const T *)a.x + (int64_t)min(m0 + u, a.M - 1) * a.ldx + c, cnt, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            top = fmaxf(top, finite_size(v[u][k]));
        const int byte = scale_byte(block_max(top), a.e5);
        if (m0 + u < a.M && cnt > 0) {
            const int64_t m = m0 + u;
            store_bytes(a.q + m * a.ldq + c, cnt, encode8(v[u], inverse_scale(byte), a.e5));
            if ((lane & 15) == 0)
                a.scale[m * a.lds + (c >> 7)] = (uint8_t)byte;
        }
    }
}

// A 128 x 128 tile a workgroup: a thread holds four rows of eight columns, from
// which it has the largest magnitudes of its rows (by lane permutations), of its
// columns and of the tile (through LDS).  The transposed values turn as bytes in LDS.
// So x is read once for both copies and their scales.  8192 x 8192 BF16, both
// copies: 59 to 64 us (270 MB, 4.2 to 4.6 TB/s: lines of 128 bytes to 2 x 8192
// places); with the slope of gelu_tanh, from two inputs, and the columns' sums 86 to
// 95 us (404 MB, 4.2 to 4.7 TB/s).  By 256 threads of twice the rows, with the
// columns' maxima by a permutation each instead of folding, that pass took 110 us,
// and 777 x 1032 9.7 us instead of 7.1.  More workgroups on a CU by fewer registers
// spill; square or XCD-contiguous orders of the tiles change nothing.
//
// The workgroups after those of the tiles copy operands of the products that
// follow (none where it only quantises).
constexpr int kTileThreads = 512;

template <typename T, int ACT>
__global__ __launch_bounds__(kTileThreads) void quantize_tile_kernel(const QuantArgs a, const PackArgs pack)
{
    if ((int)blockIdx.x >= a.blocks) {
        pack_chunk<uint8_t, kTileThreads>(pack, blockIdx.x - a.blocks);
        return;
    }
    constexpr int R = 4, W = kTileThreads / 64, PITCH = 136;
    // rows of the transposed tile: those that a wave writes together, eight apart, lie four banks apart
    auto turned_at = [](int row) __attribute__((always_inline)) { return row * PITCH + (row >> 5) * 16; };
    __shared__ __attribute__((aligned(16))) float cols[W][128];
    __shared__ __attribute__((aligned(16))) float inv[128];
    __shared__ __attribute__((aligned(16))) uint8_t turned[128 * PITCH + 48];
    __shared__ float wave_top[W];
    const int tr = blockIdx.x / a.strips, tc = blockIdx.x - tr * a.strips;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6, q = rg & 3;
    const int m0 = tr * 128 + rg * R, c = tc * 128 + cg * 8;
    float v[R][8];
    {
        Raw8<T> x[R], z[R];
        if (a.K >= 8) {
#pragma unroll
            for (int p = 0; p < R; ++p) {
                const int64_t m = min(m0 + p, a.M - 1);
                x[p] = load_raw((const T *)a.x + m * a.ldx, c, a.K);
                if constexpr (ACT != DENSE_ACT_NONE)
                    z[p] = load_raw((const T *)a.z + m * a.ldz, c, a.K);
            }
        }
#pragma unroll
        for (int p = 0; p < R; ++p) {
            const int64_t m = min(m0 + p, a.M - 1);
            float s[8];
            if (a.K < 8) {
                load_n((const T *)a.x + m * a.ldx + c, a.K - c, v[p]);
                if constexpr (ACT != DENSE_ACT_NONE)
                    load_n((const T *)a.z + m * a.ldz + c, a.K - c, s);
            } else if (tc * 128 + 128 <= a.K) {
                widen(x[p], v[p]);
                if constexpr (ACT != DENSE_ACT_NONE)
                    widen(z[p], s);
            } else {
                widen_part<true>(x[p], c, a.K, v[p]);
                if constexpr (ACT != DENSE_ACT_NONE)
                    widen_part<true>(z[p], c, a.K, s);
            }
            if constexpr (ACT != DENSE_ACT_NONE) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[p][k] *= act_slope<ACT>(s[k]);
            }
        }
    }
    if (tr * 128 + 128 > a.M) {
#pragma unroll
        for (int p = 0; p < R; ++p)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[p][k] = m0 + p < a.M ? v[p][k] : 0.0f;
    }

    // f over the rows of each column, of a wave's rows by folding two columns into one register and four
    // into one (lane 16 q + cg then holds columns 8 cg + 2 q' and the next, q' = q with its bits as they
    // fold), then of the waves through LDS: thread i < 128 has column i's
    auto columns = [&](float (&s)[8], auto f) __attribute__((always_inline)) {
        float h[4], w[2];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            h[k] = fold_halves(s[k], s[k + 4], f);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = fold_rows(h[k], h[k + 2], f);
        store_all(&cols[wave][cg * 8 + (q >> 1) * 4 + (q & 1) * 2], w);
        __syncthreads();
        float t = 0.0f;
        if (threadIdx.x < 128) {
            t = cols[0][threadIdx.x];
#pragma unroll
            for (int i = 1; i < W; ++i)
                t = f(t, cols[i][threadIdx.x]);
        }
        return t;
    };
    if (a.colsum) {
        float s[8] = {};
#pragma unroll
        for (int p = 0; p < R; ++p)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                s[k] += v[p][k];
        const float t = columns(s, [](float x, float y) { return x + y; });
        if (threadIdx.x < 128 && tc * 128 + (int)threadIdx.x < a.K)
            a.colsum[tr * a.sum_ld + tc * 128 + threadIdx.x] = t;
        __syncthreads();
    }

    float row_top[R], col_top[8] = {}, all = 0.0f;
#pragma unroll
    for (int p = 0; p < R; ++p) {
        row_top[p] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s = finite_size(v[p][k]);
            row_top[p] = fmaxf(row_top[p], s);
            col_top[k] = fmaxf(col_top[k], s);
        }
        all = fmaxf(all, row_top[p]);
        row_top[p] = block_max(row_top[p]);
    }
    int tile_byte = 0;
    if (a.tiles || a.tiles_t) {
        all = wave_max(all);
        if ((threadIdx.x & 63) == 0)
            wave_top[wave] = all;
        __syncthreads();
        all = wave_top[0];
#pragma unroll
        for (int i = 1; i < W; ++i)
            all = fmaxf(all, wave_top[i]);
        tile_byte = scale_byte(all, a.e5);
    }

    if (a.q) {
#pragma unroll
        for (int p = 0; p < R; ++p) {
            const int byte = a.tiles ? tile_byte : scale_byte(row_top[p], a.e5);
            if (m0 + p < a.M) {
                const int64_t m = m0 + p;
                store_bytes(a.q + m * a.ldq + c, a.q_cols - c, encode8(v[p], inverse_scale(byte), a.e5));
                if (!a.tiles && cg == 0)
                    a.scale[m * a.lds + tc] = (uint8_t)byte;
            }
        }
        if (a.tiles && threadIdx.x == 0)
            a.scale[tr * a.lds + tc] = (uint8_t)tile_byte;
    }
    if (!a.qt)
        return;
    float by[8];
    if (a.tiles_t) {
        if (threadIdx.x == 0)
            a.scale_t[tc * a.ldst + tr] = (uint8_t)tile_byte;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            by[k] = inverse_scale(tile_byte);
    } else {
        const float t = columns(col_top, [](float x, float y) { return fmaxf(x, y); });
        if (threadIdx.x < 128) {
            const int byte = scale_byte(t, a.e5);
            inv[threadIdx.x] = inverse_scale(byte);
            if (tc * 128 + (int)threadIdx.x < a.K)
                a.scale_t[(int64_t)(tc * 128 + threadIdx.x) * a.ldst + tr] = (uint8_t)byte;
        }
        __syncthreads();
        load_all(&inv[cg * 8], by);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *(int *)&turned[turned_at(cg * 8 + k) + rg * R] = encode4(v[0][k], v[1][k], v[2][k], v[3][k], by[k], a.e5);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i * 32 + rg, n = tc * 128 + row, m = tr * 128 + cg * 8;
        typedef int v2i __attribute__((ext_vector_type(2)));
        const v2i w = *(const v2i *)&turned[turned_at(row) + cg * 8];
        if (n < a.K)
            store_bytes(a.qt + (int64_t)n * a.ldqt + m, a.qt_cols - m, __builtin_bit_cast(Pack<uint8_t, 8>, w));
    }
}

struct DequantArgs {
    const uint8_t *q, *scale;
    void *x;
    int64_t ldq, lds, ldx;
    int M, K, strips;
    int x_cols;               // columns of x that are written: K, or more as zeros
    int shift;                // 7: one row of scales for 128 rows, 0: for each
    bool e5;
};

// The same split as quantize_rows_kernel's.  8192 x 8192 to BF16: 39 to 50 us (205 MB,
// 4.1 to 5.3 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void dequantize_kernel(const DequantArgs a)
{
    constexpr int U = 4;
    typedef int v2i __attribute__((ext_vector_type(2)));
    typedef float v2f __attribute__((ext_vector_type(2)));
    const int rb = blockIdx.x / a.strips, strip = blockIdx.x - rb * a.strips;
    const int c = strip * 512 + (threadIdx.x & 63) * 8, cnt = a.K - c;
    const int m0 = (rb * 4 + (threadIdx.x >> 6)) * U;
    if (c >= a.x_cols)
        return;
    Pack<uint8_t, 8> q[U];
    int byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t m = min(m0 + u, a.M - 1);
        const uint8_t *p = a.q + m * a.ldq + c;
        byte[u] = cnt > 0 ? a.scale[(m >> a.shift) * a.lds + (c >> 7)] : 0;
        if (cnt >= 8) {
            q[u] = *(const Pack<uint8_t, 8> *)p;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                q[u].e[k] = k < cnt ? p[k] : 0;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (m0 + u >= a.M)
            break;
        const v2i w = __builtin_bit_cast(v2i, q[u]);
        float v[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v2f lo, hi;
            if (a.e5) {
                lo = __builtin_amdgcn_cvt_pk_f32_bf8(w[i], false);
                hi = __builtin_amdgcn_cvt_pk_f32_bf8(w[i], true);
            } else {
                lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false);
                hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
            }
            v[4 * i] = lo.x;
            v[4 * i + 1] = lo.y;
            v[4 * i + 2] = hi.x;
            v[4 * i + 3] = hi.y;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = k >= cnt ? 0.0f : byte[u] == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(v[k], byte[u] - 127);
        store_n((T *)a.x + (int64_t)(m0 + u) * a.ldx + c, a.x_cols - c, v);
    }
}

}  // namespace dense
