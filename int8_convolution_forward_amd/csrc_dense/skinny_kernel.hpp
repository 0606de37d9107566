// Dense layer for a few rows of x (single tokens, decode batches): bound by
// reading the weights once.
//
// A workgroup of W waves takes 16 R rows of w (output columns) and all M <= 16 G
// rows of x; the waves split the inner dimension into 128-byte blocks and add
// their sums in order through LDS at the end.  Rows past M and N are loaded as
// zeros (or repeat the last row) and their sums are not stored.
//
// Where rows are 16-byte aligned, skinny_kernel streams the blocks of w -- and,
// for more than four rows, of x -- through a part of LDS that is the wave's own
// (no barriers), by loads in which eight lanes take 128 contiguous bytes of a
// row.  Loading a fragment straight into registers makes 16 lanes touch 16 rows
// at a time, and the cache then delivers 16 bytes a cycle instead of 64: one bf16
// token through
// [8192, 2048] takes 7.2 us that way and 6.7 through LDS (33.5 MB, 5.0 TB/s,
// what a large copy reaches), 16 int8 tokens through [2048, 8192] 9.1 and 5.4.
// Splitting the inner dimension over workgroups as well, with a second launch
// to join them, costs more than it gives (6.9 us for the latter).
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

template <typename T>
__device__ __forceinline__ v4i load_piece(const uint8_t *p)
{
    return ((const Piece16<T> *)p)->v;
}

// the first `valid` bytes of a piece, zeros after them
template <typename T>
__device__ __forceinline__ v4i load_piece_tail(const uint8_t *p, int64_t valid)
{
    if (valid >= 16)
        return load_piece<T>(p);
    union { v4i v; T e[16 / sizeof(T)]; } u;
    u.v = v4i{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i)
        if ((i + 1) * (int)sizeof(T) <= valid)
            u.e[i] = ((const T *)p)[i];
    return u.v;
}

// Adds the waves' sums, in order, and finishes 16 R columns of every row.  Sum v
// of lane l belongs to column 4 (l / 16) + v of row l % 16 of its block.
template <typename T, int G, int R, int W>
__device__ __forceinline__ void skinny_finish(const SkinnyArgs &g, typename Acc4<T>::type (*red)[R * G][64], int n0)
{
    for (int o = threadIdx.x; o < R * G * 256; o += 64 * W) {
        const int c = o % (16 * R), m = o / (16 * R), n = n0 + c;
        const int src = ((c & 15) >> 2) * 16 + (m & 15), f = (c >> 4) * G + (m >> 4);
        if (m >= g.M || n >= g.N)
            continue;
        float z;
        if constexpr (is_int<T>) {
            int s = 0;
#pragma unroll
            for (int k = 0; k < W; ++k)
                s += red[k][f][src][c & 3];
            z = (float)s;
            z *= (g.epi.x_scale ? g.epi.x_scale[m] : 1.0f) * (g.epi.w_scale ? g.epi.w_scale[n] : 1.0f);
        } else {
            z = 0.0f;
#pragma unroll
            for (int k = 0; k < W; ++k)
                z += red[k][f][src][c & 3];
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

// D: blocks a wave has in flight; XL: x goes through LDS too
template <typename T, int G, int R, int W, int D, bool XL>
__global__ __launch_bounds__(64 * W) void skinny_kernel(const SkinnyArgs g)
{
    typedef typename Acc4<T>::type acc_t;
    constexpr int BLOCK = 2048 * (R + (XL ? G : 0));   // LDS bytes of one block: 16 rows of 128 bytes each
    constexpr int L = BLOCK / 1024;                    // loads of one block
    constexpr int RED = W * R * G * 1024;
    static_assert(D * L < 64, "loads in flight");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[W * D * BLOCK > RED ? W * D * BLOCK : RED];
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
    const int blocks = (int)((g.kbytes + 127) >> 7);
    uint8_t *mine = smem + wave * D * BLOCK;
    const unsigned lds = lds_address(mine);
    const uint8_t *wbase = g.w + (int64_t)n0 * g.ldw;

    // block b into slot d; a block past the end, and what lies past the inner
    // dimension in the last one, loads zeros
    auto issue = [&](int b, int d) {
        const int range = b < blocks ? 0x7fffffff : 0;
        const v4i wr = make_rsrc(wbase + (int64_t)b * 128, range), xr = make_rsrc(g.x + (int64_t)b * 128, range);
        const unsigned to = lds + d * BLOCK;
        const int64_t left = g.kbytes - (int64_t)b * 128;
        auto put = [&](auto at, v4i rsrc, int off, int h) {
            set_lds_target<decltype(at)::value>(to);
            const int v = chunk[h] < left ? off : kOutOfRange;
            asm volatile("s_nop 0");
            load16_to_lds(rsrc, v);
        };
        for_each<2 * R>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
            put(Size<i * 1024>{}, wr, woff[i / 2][i & 1], i & 1);
        });
        if constexpr (XL)
            for_each<2 * G>([&](auto ic) {
                constexpr int i = decltype(ic)::value;
                put(Size<2048 * R + i * 1024>{}, xr, xoff[i / 2][i & 1], i & 1);
            });
    };
    // x straight from memory: the few rows of a 16-lane group coincide
    auto load_x = [&](int b, v4i (&xv)[2][G]) {
        const __amdgpu_buffer_rsrc_t xr =
            __builtin_amdgcn_make_buffer_rsrc((void *)(g.x + (int64_t)b * 128), (short)0, b < blocks ? 0x7fffffff : 0, 0x00020000);
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

    acc_t acc[R][G];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k)
            acc[i][k] = acc_t{0, 0, 0, 0};
    auto multiply = [&](int d, const v4i (&xv)[2][G]) {
        const uint8_t *s = mine + d * BLOCK;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = r * 128 + row_swizzle<128>(r, h * 4 + q) * 16;
            v4i wv[R], x[G];
#pragma unroll
            for (int i = 0; i < R; ++i)
                wv[i] = *(const v4i *)(s + i * 2048 + at);
#pragma unroll
            for (int i = 0; i < G; ++i)
                x[i] = XL ? *(const v4i *)(s + (R + i) * 2048 + at) : xv[h][i];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int k = 0; k < G; ++k)
                    acc[i][k] = mfma16<T>(wv[i], x[k], acc[i][k]);
        }
    };

    int b = wave;
    if constexpr (XL) {
        // a ring: the slot of a block takes the block D ahead once its reads are done
        if (b < blocks)
#pragma unroll
            for (int d = 0; d < D; ++d)
                issue(b + d * W, d);
        for (; b < blocks; b += D * W) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const v4i none[2][G] = {};
                __builtin_amdgcn_sched_barrier(0);
                wait_vm_lgkm0<(D - 1) * L>();
                __builtin_amdgcn_sched_barrier(0);
                multiply(d, none);
                __builtin_amdgcn_sched_barrier(0);
                wait_lgkm0();
                issue(b + (d + D) * W, d);
            }
        }
    } else {
        // D blocks at a time: the compiler counts the loads of x but not those
        // to LDS, and waits for more of them than a ring could afford
        for (; b < blocks; b += D * W) {
            v4i xv[D][2][G];
#pragma unroll
            for (int d = 0; d < D; ++d)
                load_x(b + d * W, xv[d]);
#pragma unroll
            for (int d = 0; d < D; ++d)
                issue(b + d * W, d);
            for_each<D>([&](auto dc) {
                constexpr int d = decltype(dc)::value;
                __builtin_amdgcn_sched_barrier(0);
                wait_vm_lgkm0<(D - 1 - d) * L>();
                __builtin_amdgcn_sched_barrier(0);
                multiply(d, xv[d]);
            });
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkm0();
        }
    }
    wait_vm_lgkm0<0>();  // trailing loads of zeros still write to LDS
    __syncthreads();
    acc_t(*red)[R * G][64] = (acc_t(*)[R * G][64])smem;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < G; ++k)
            red[wave][i * G + k][lane] = acc[i][k];
    __syncthreads();
    skinny_finish<T, G, R, W>(g, red, n0);
}

// Rows that are not 16-byte aligned: the same loads, eight lanes to 128 bytes of
// a row, but by way of registers (a load into LDS needs aligned chunks), U
// blocks of w and x at a time.  One fp16 token through [6736, 4313]: 14 us, with
// fragments loaded straight from memory 25.
template <typename T, int G, int W, int U>
__global__ __launch_bounds__(64 * W) void skinny_unaligned_kernel(const SkinnyArgs g)
{
    typedef typename Acc4<T>::type acc_t;
    constexpr int BLOCK = 2048 * (1 + G);              // LDS bytes of one block: w's 16 rows, then x's
    constexpr int RED = W * G * 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[W * U * BLOCK > RED ? W * U * BLOCK : RED];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int r = lane & 15, q = lane >> 4;

    // load h of 16 rows: row 8 h + lane / 8, chunk lane % 8; rows past the end repeat the last one
    const int chunk = (lane & 7) * 16;
    const uint8_t *src[2 * (1 + G)];
    int dst[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = h * 8 + (lane >> 3);
        dst[h] = row * 128 + row_swizzle<128>(row, lane & 7) * 16;
        src[h] = g.w + (int64_t)min(n0 + row, g.N - 1) * g.ldw + chunk;
#pragma unroll
        for (int i = 0; i < G; ++i)
            src[2 + 2 * i + h] = g.x + (int64_t)min(16 * i + row, g.M - 1) * g.ldx + chunk;
    }
    uint8_t *mine = smem + wave * U * BLOCK;

    acc_t acc[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        acc[i] = acc_t{0, 0, 0, 0};
    // LAST: the block in which the inner dimension may end before the block does
    auto blocks_at = [&](auto nc, auto last, int64_t b) __attribute__((always_inline)) {
        constexpr int N = decltype(nc)::value;
        v4i v[N][2 * (1 + G)];
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < 2 * (1 + G); ++i) {
                const int64_t k = (b + u * W) * 128;
                if constexpr (decltype(last)::value)
                    v[u][i] = load_piece_tail<T>(src[i] + k, g.kbytes - k - chunk);
                else
                    v[u][i] = load_piece<T>(src[i] + k);
            }
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int i = 0; i < 2 * (1 + G); ++i)
                *(v4i *)(mine + u * BLOCK + (i >> 1) * 2048 + dst[i & 1]) = v[u][i];
        // the wave's own LDS, whose operations run in order: only the compiler
        // must not move the reads up (or the next block's writes)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *s = mine + u * BLOCK + r * 128 + row_swizzle<128>(r, h * 4 + q) * 16;
                const v4i wv = *(const v4i *)s;
#pragma unroll
                for (int i = 0; i < G; ++i)
                    acc[i] = mfma16<T>(wv, *(const v4i *)(s + (1 + i) * 2048), acc[i]);
            }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    const int64_t blocks = g.kbytes >> 7;
    int64_t b = wave;
    for (; b + (U - 1) * W < blocks; b += U * W)
        blocks_at(Size<U>{}, Size<0>{}, b);
    for (; b < blocks; b += W)
        blocks_at(Size<1>{}, Size<0>{}, b);
    if (b == blocks)  // the wave whose turn the last, partial block is
        blocks_at(Size<1>{}, Size<1>{}, b);

    __syncthreads();
    acc_t(*red)[G][64] = (acc_t(*)[G][64])smem;
#pragma unroll
    for (int i = 0; i < G; ++i)
        red[wave][i][lane] = acc[i];
    __syncthreads();
    skinny_finish<T, G, 1, W>(g, red, n0);
}

}  // namespace dense
