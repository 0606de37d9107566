// The dense layer on 8-bit floating point for a few rows of x: bound by reading
// the weights once.
//
// As in skinny_kernel.hpp a workgroup of W waves takes 16 R rows of w and all M <=
// 16 G rows of x, and the waves split the inner dimension; here into groups of
// four blocks of 128, whose four scales are one word of a row.  A group's loads go
// out together: the weights (and x, for more than four rows) into the wave's own
// part of LDS, scales and x otherwise into registers.
//
// The values are taken to BF16, which holds them and their scale exactly, on the
// way into the matrix unit: the vector unit has the time for it, and the sums are
// then those of 32 bits, which the 8-bit instructions' are not (gemm_kernel.hpp).
// 1 x 8192 x 2048 in 5.3 us a call (16.8 MB of weights, kept by the caches in part:
// 5.6 us in a trace), 1 x 16384 x 4096 in 15.7 (4.3 TB/s).
#pragma once

#include "gemm_kernel.hpp"
#include "skinny_kernel.hpp"

namespace dense {

struct SkinnyF8Args {
    SkinnyArgs s;
    const uint8_t *sx, *sw;   // exponents of the scales, a byte for a block
    int64_t ldsx, ldsw;
    int sw_shift;             // 7: one row of them for 128 rows of w, 0: for each
    int kblocks;
};

// Eight values and the power of two 2^(byte - 127)
template <typename T>
__device__ __forceinline__ v8bf to_bf16(int a, int b, float scale)
{
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    v2bf p[4];
    if constexpr (__is_same(T, f8e4)) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, scale, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(a, scale, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, scale, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(b, scale, true);
    }
    return __builtin_bit_cast(v8bf, p);
}

__device__ __forceinline__ float scale_of(int word, int d)
{
    return __builtin_bit_cast(float, ((unsigned)word >> (8 * d) & 255) << 23);
}

template <typename T, int G, int R, int W, bool XL>
__global__ __launch_bounds__(64 * W) void skinny_f8_kernel(const SkinnyF8Args a)
{
    constexpr int D = 4;
    constexpr int BLOCK = 2048 * (R + (XL ? G : 0));   // LDS bytes of one block: 16 rows of 128 bytes each
    constexpr int L = BLOCK / 1024;                    // loads of one block
    constexpr int RED = W * R * G * 1024;
    static_assert(D * L < 64, "loads in flight");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[W * D * BLOCK > RED ? W * D * BLOCK : RED];
    const SkinnyArgs &g = a.s;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16 * R;
    const int r = lane & 15, q = lane >> 4;

    // load h of 16 rows: row 8 h + lane / 8, the chunk that belongs at lane % 8
    int chunk[2], woff[R][2], xoff[G][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = h * 8 + (lane >> 3);
        chunk[h] = row_swizzle<128>(row, lane & 7) * 16;
#pragma unroll
        for (int i = 0; i < R; ++i)
            woff[i][h] = n0 + 16 * i + row < g.N ? (16 * i + row) * (int)g.ldw + chunk[h] : kOutOfRange;
#pragma unroll
        for (int i = 0; i < G; ++i)
            xoff[i][h] = 16 * i + row < g.M ? (16 * i + row) * (int)g.ldx + chunk[h] : kOutOfRange;
    }
    uint8_t *mine = smem + wave * D * BLOCK;
    const unsigned lds = lds_address(mine);
    const uint8_t *wbase = g.w + (int64_t)n0 * g.ldw;

    // block b into slot d; what lies past the inner dimension loads zeros
    auto issue = [&](int b, auto dc) __attribute__((always_inline)) {
        constexpr int d = decltype(dc)::value;
        const int range = b < a.kblocks ? 0x7fffffff : 0;
        const v4i wr = make_rsrc(wbase + (int64_t)b * 128, range), xr = make_rsrc(g.x + (int64_t)b * 128, range);
        const int64_t left = g.kbytes - (int64_t)b * 128;
        auto put = [&](auto at, v4i rsrc, int off, int h) __attribute__((always_inline)) {
            set_lds_target<d * BLOCK + decltype(at)::value>(lds);
            const int v = chunk[h] < left ? off : kOutOfRange;
            asm volatile("s_nop 0");
            load16_to_lds(rsrc, v);
        };
        for_each<2 * R>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            put(Size<i * 1024>{}, wr, woff[i / 2][i & 1], i & 1);
        });
        if constexpr (XL)
            for_each<2 * G>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                put(Size<2048 * R + i * 1024>{}, xr, xoff[i / 2][i & 1], i & 1);
            });
    };
    // x straight from memory: the few rows of a 16-lane group coincide
    auto load_x = [&](int b, v4i (&xv)[2][G]) __attribute__((always_inline)) {
        const __amdgpu_buffer_rsrc_t xr =
            __builtin_amdgcn_make_buffer_rsrc((void *)(g.x + (int64_t)b * 128), (short)0, b < a.kblocks ? 0x7fffffff : 0, 0x00020000);
        const int64_t left = g.kbytes - (int64_t)b * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int k = h * 64 + q * 16;
                const int off = min(16 * i + r, g.M - 1) * (int)g.ldx + k;
                xv[h][i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(xr, k < left ? off : kOutOfRange, 0, 0));
            }
    };

    v4f acc[R][G];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k)
            acc[i][k] = v4f{0, 0, 0, 0};
    for (int grp = wave; grp * D < a.kblocks; grp += W) {
        // the compiler counts these loads but not those to LDS: they go first
        int sx[G], sw[R];
        load_scale_words([&](int i) { return a.sx + (int64_t)min(16 * i + r, g.M - 1) * a.ldsx; }, grp * D, a.kblocks, sx);
        load_scale_words([&](int i) { return a.sw + (int64_t)(min(n0 + 16 * i + r, g.N - 1) >> a.sw_shift) * a.ldsw; }, grp * D,
                         a.kblocks, sw);
        v4i xv[XL ? 1 : D][2][G];
        if constexpr (!XL)
#pragma unroll
            for (int d = 0; d < D; ++d)
                load_x(grp * D + d, xv[d]);
        __builtin_amdgcn_sched_barrier(0);
        for_each<D>([&](auto dc) __attribute__((always_inline)) { issue(grp * D + decltype(dc)::value, dc); });
        shift_scale_words(grp * D, a.kblocks, sx);
        shift_scale_words(grp * D, a.kblocks, sw);
        for_each<D>([&](auto dc) __attribute__((always_inline)) {
            constexpr int d = decltype(dc)::value;
            __builtin_amdgcn_sched_barrier(0);
            wait_vm_lgkm0<(D - 1 - d) * L>();
            __builtin_amdgcn_sched_barrier(0);
            const uint8_t *s = mine + d * BLOCK;
            const int at[2] = {r * 128 + row_swizzle<128>(r, q) * 16, r * 128 + row_swizzle<128>(r, 4 + q) * 16};
            float by_w[R], by_x[G];
#pragma unroll
            for (int i = 0; i < R; ++i)
                by_w[i] = scale_of(sw[i], d);
#pragma unroll
            for (int i = 0; i < G; ++i)
                by_x[i] = scale_of(sx[i], d);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i wv[R], x[G];
#pragma unroll
                for (int i = 0; i < R; ++i)
                    wv[i] = *(const v4i *)(s + i * 2048 + at[h]);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    if constexpr (XL)
                        x[i] = *(const v4i *)(s + (R + i) * 2048 + at[h]);
                    else
                        x[i] = xv[d][h][i];
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    v8bf wb[R], xb[G];
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        wb[i] = to_bf16<f8e4>(wv[i][e], wv[i][e + 1], by_w[i]);
#pragma unroll
                    for (int i = 0; i < G; ++i)
                        xb[i] = to_bf16<T>(x[i][e], x[i][e + 1], by_x[i]);
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int k = 0; k < G; ++k)
                            acc[i][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[i], xb[k], acc[i][k], 0, 0, 0);
                }
            }
        });
        __builtin_amdgcn_sched_barrier(0);
        wait_lgkm0();  // the reads are done before the next group's loads write
    }
    wait_vm_lgkm0<0>();
    __syncthreads();
    v4f(*red)[R * G][64] = (v4f(*)[R * G][64])smem;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k)
            red[wave][i * G + k][lane] = acc[i][k];
    __syncthreads();
    skinny_finish<T, G, R, W>(g, red, n0);
}

}  // namespace dense
