// Memory-bound passes around the products: copies of operands into the form
// the product kernel reads in place, and the gradient of the activation with the
// column sums of the bias gradient.
#pragma once

#include "colsum.hpp"
#include "dense_common.hpp"

namespace dense {

// One operand copied to rows of 16-byte chunks: dst row r holds `cols`
// elements of src row r and zeros up to the chunk's end.
struct PackJob {
    const void *src;
    void *dst;
    int64_t rows, cols;      // elements
    int64_t rs, cs;          // source strides in elements
    int64_t chunks;          // 16-byte chunks per destination row
    int64_t items;           // rows * chunks, 0 for an unused job
};

struct PackArgs {
    PackJob job[2];
    int first;               // workgroups of job 0
};

// One thread copies one chunk; both operands of a product go in one launch.
// U is an unsigned integer of the element's size, THREADS those of a workgroup.
template <typename U, int THREADS = 256>
__device__ __forceinline__ void pack_chunk(const PackArgs &a, int block)
{
    constexpr int E = 16 / sizeof(U);
    struct __attribute__((packed, aligned(sizeof(U)))) Piece { U e[E]; };
    const bool second = block >= a.first;
    const PackJob &j = a.job[second];
    const int64_t i = (int64_t)(second ? block - a.first : block) * THREADS + threadIdx.x;
    if (i >= j.items)
        return;
    // a 64-bit division costs more than the copy
    const int64_t r = j.items <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)j.chunks) : i / j.chunks;
    const int64_t c = (i - r * j.chunks) * E;
    const U *s = (const U *)j.src + r * j.rs + c * j.cs;
    Piece p;
    if (j.cs == 1 && c + E <= j.cols) {
        p = *(const Piece *)s;
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
            p.e[k] = c + k < j.cols ? s[k * j.cs] : U(0);
    }
    *(v4i *)((U *)j.dst + i * E) = __builtin_bit_cast(v4i, p);
}

template <typename U>
__global__ __launch_bounds__(256) void pack_kernel(const PackArgs a)
{
    pack_chunk<U>(a, blockIdx.x);
}

// g = dy act'(z), written with a row pitch of whole 16-byte chunks (zeros past
// N), and column sums of the unrounded g over a block of rows.  g is rounded to
// the operands' type, since the matrix unit takes both of a product's operands in
// it: relative errors of half a step, as dy's and z's own roundings have, and in
// FP16, below 2^-14, errors of up to 2^-25, where g is smaller than both.  A
// caller who needs g's further digits has it in two terms: what the rounding
// takes away, raised by second_term_up, goes to g2.
// 8192 x 8192 BF16 with the slope of gelu's tanh form: 75 us (403 MB, 5.4 TB/s);
// with loads of one row at a time, each under a condition, 100.
template <typename T> constexpr float second_term_up();
template <> constexpr float second_term_up<bf16>() { return 1.0f; }
template <> constexpr float second_term_up<f16>() { return 2048.0f; }  // at most half a step of 65504: 2^15

struct ActGradArgs {
    const void *dy, *z;       // z null: g = dy
    int64_t ldy, ldz;
    int M, N;
    int rows;                 // rows per workgroup
    int strips, blocks;       // workgroups along a row, and of this pass
    void *g, *g2;             // g null: only the column sums; g2: the second term
    int64_t ldg;
    float *colsum;            // [row block][sum_ld], or null
    int64_t sum_ld;
};

// A wave takes 512 columns (eight per lane) of every fourth row of its block,
// so that each load is one contiguous 1 KiB; the four waves' column sums are
// added through LDS in order.  The workgroups after those copy operands.  WIDE: g
// has two terms (asked for at run time, one term pays 0.3 us for it).
template <typename T, int ACT, bool WIDE>
__global__ __launch_bounds__(256) void act_grad_kernel(const ActGradArgs a, const PackArgs pack)
{
    if ((int)blockIdx.x >= a.blocks) {
        pack_chunk<uint16_t>(pack, blockIdx.x - a.blocks);
        return;
    }
    const int rb = blockIdx.x / a.strips, strip = blockIdx.x - rb * a.strips;
    __shared__ float red[4][512];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = strip * 512 + lane * 8;
    const int cnt = a.N - n;
    const int m0 = rb * a.rows, m1 = min(a.M, m0 + a.rows);
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum[i] = 0.0f;
    // FORM 2: eight columns for every lane, 1: eight or none, 0: any number;
    // -1: fewer than eight columns in all
    auto some = [&](auto form, auto uc, int m) __attribute__((always_inline)) {
        constexpr int FORM = decltype(form)::value, U = decltype(uc)::value;
        float v[U][8];
        if constexpr (FORM < 0) {
            load_n((const T *)a.dy + m * a.ldy + n, cnt, v[0]);
            if constexpr (ACT != DENSE_ACT_NONE) {
                float z[8];
                load_n((const T *)a.z + m * a.ldz + n, cnt, z);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[0][i] *= act_slope<ACT>(z[i]);
            }
        } else {
            Raw8<T> dy[U], z[U];
            auto wide = [&](const Raw8<T> &r, float (&w)[8]) {
                if constexpr (FORM == 2)
                    widen(r, w);
                else
                    widen_part<FORM == 0>(r, n, a.N, w);
            };
#pragma unroll
            for (int u = 0; u < U; ++u) {  // the loads of all rows go out together
                dy[u] = load_raw((const T *)a.dy + (m + 4 * u) * a.ldy, n, a.N);
                if constexpr (ACT != DENSE_ACT_NONE)
                    z[u] = load_raw((const T *)a.z + (m + 4 * u) * a.ldz, n, a.N);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                wide(dy[u], v[u]);
                if constexpr (ACT != DENSE_ACT_NONE) {
                    float zv[8];
                    wide(z[u], zv);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[u][i] *= act_slope<ACT>(zv[i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (a.g && (FORM == 2 || cnt > 0)) {
                store_all((T *)a.g + (m + 4 * u) * a.ldg + n, v[u]);
                if constexpr (WIDE) {
                    float rest[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float d = v[u][i] - (float)(T)v[u][i];
                        rest[i] = fabsf(d) < INFINITY ? d * second_term_up<T>() : 0.0f;  // NaN, infinities: all in g
                    }
                    store_all((T *)a.g2 + (m + 4 * u) * a.ldg + n, rest);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[i] += v[u][i];
        }
    };
    auto rows = [&](auto form) __attribute__((always_inline)) {
        int m = m0 + wave;
        if constexpr (decltype(form)::value >= 0)
            for (; m + 12 < m1; m += 16)
                some(form, Size<4>{}, m);
        for (; m < m1; m += 4)
            some(form, Size<1>{}, m);
    };
    if (strip * 512 + 512 <= a.N)
        rows(Size<2>{});
    else if (a.N % 8 == 0)
        rows(Size<1>{});
    else if (a.N > 8)
        rows(Size<0>{});
    else
        rows(Size<-1>{});
    if (!a.colsum)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[wave][lane * 8 + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256)
        if (strip * 512 + c < a.N)
            a.colsum[rb * a.sum_ld + strip * 512 + c] =
                (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
}

}  // namespace dense
