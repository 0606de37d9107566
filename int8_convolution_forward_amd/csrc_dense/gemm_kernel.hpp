// Tiled matrix product for gfx950: C[m, n] = sum_k A(m, k) B(n, k) with the
// dense layer's epilogue, operands BF16, FP16 (32-bit float sums) or INT8
// (32-bit integer sums).
//
// A workgroup of four waves computes a TM x TN tile.  Both operands stream
// from memory straight into a ring of NS LDS stages (buffer_load ... lds, 16
// bytes a lane, no staging registers), NS-1 stages ahead of the one that is
// multiplied; one barrier per stage publishes the stage that landed and
// retires the slot the next loads overwrite.  A stage is 64 bytes of the inner
// dimension: 32 BF16/FP16 or 64 INT8 values, two matrix instructions deep.
//
// An operand is stored in one of two ways:
//  * rows (STR false): the inner dimension is contiguous.  LDS holds 64-byte
//    rows whose 16-byte chunks are permuted by row bits 1..2, so that the 32
//    rows a fragment read touches spread over all banks.
//  * columns (STR true, 16-bit types): the inner dimension has the stride.
//    LDS holds one row of TM (TN) values per inner index, 64-byte groups
//    permuted by the row's low bits; fragments come from transposing reads
//    (ds_read_tr16_b64: lane i of a 16-lane group gets value i % 4 of the
//    four 8-byte pieces that lanes 4b + i/4 address).
// A gradient therefore reads the same tensors as the forward product, with no
// transposed copies.
//
// What lies outside an operand is loaded from an offset past the buffer's
// range and reads as zeros: no branch guards an edge.  Host code gives the
// kernel only operands whose 16-byte chunks are aligned and do not straddle a
// row's end (others are copied into that form first).  Bases advance by 64-bit
// scalar adds, so only offsets within one tile have to fit 31 bits.
//
// Matrix operands are passed as (B, A): a lane then holds one row m and four
// consecutive columns n at a time.  The epilogue turns 32-row slabs of the
// wave's tile through its own part of LDS, so that every lane loads, computes
// and stores eight consecutive columns (16 bytes) and a wave writes whole
// 256-byte row segments.
#pragma once

#include "dense_common.hpp"

namespace dense {

struct GemmArgs {
    const uint8_t *a, *b;
    int64_t lda, ldb;      // bytes between rows (rows form) or inner indices (columns form)
    int M, N;
    int kbytes;            // inner dimension in bytes of a rows-form operand, a multiple of 16
    int K;                 // inner dimension in elements
    int nstages;           // stages of 64 bytes
    int kchunk;            // stages per split
    int tiles_m, tiles_n, tiles;
    int group;             // row tiles per group of the tile order
    int64_t part_stride;   // split: 32-bit values per partial copy
    int part_ld;
    void *part;            // split: partial sums [split][M][part_ld], or null
    Epilogue epi;
};

template <int N> struct Size { static constexpr int value = N; };

template <typename T> struct Acc { typedef v16f type; };
template <> struct Acc<int8_t> { typedef v16i type; };

template <typename T>
__device__ __forceinline__ typename Acc<T>::type mfma32(v4i a, v4i b, typename Acc<T>::type c)
{
    if constexpr (sizeof(T) == 1)
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
    else if constexpr (__is_same(T, bf16))
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Rows form: chunk permutation of a 64-byte row.
__device__ __forceinline__ int row_swizzle(int row, int chunk)
{
    return chunk ^ (((row >> 1) ^ (row >> 2)) & 3);
}

// Columns form: 64-byte group permutation of inner row kr.  The four rows of
// a transposing read must fall into different bank groups: rows of 256 bytes
// and more all start at bank 0, two 128-byte rows cover the banks once.
template <int TD>
__device__ __forceinline__ int col_swizzle(int kr)
{
    return TD >= 128 ? kr & 3 : (kr >> 1) & 1;
}

// OCC: workgroups a CU is to hold at a time (one wave of each per SIMD)
template <typename T, int TM, int TN, int WGM, int WGN, int NS, int OCC, bool ASTR, bool BSTR>
__global__ __launch_bounds__(64 * WGM * WGN, OCC) void gemm_kernel(const GemmArgs g)
{
    constexpr int NW = WGM * WGN;
    constexpr int ES = sizeof(T);
    constexpr int BKE = 64 / ES;                // inner elements per stage
    constexpr int AL = TM / (NW * 16), BL = TN / (NW * 16), LPS = AL + BL;
    constexpr int A_BYTES = TM * 64, STAGE = (TM + TN) * 64;
    constexpr int WM = TM / WGM, WN = TN / WGN;
    constexpr int FM = WM / 32, FN = WN / 32;
    constexpr int NMF = 2 * FM * FN;            // matrix instructions per stage
    constexpr int NRD = 2 * (FM + FN);          // fragment reads per stage
    static_assert(AL >= 1 && BL >= 1 && FM >= 1 && FN >= 1, "tile too small");
    static_assert(NS >= 2 && (NS - 1) * LPS < 64, "pipeline depth");
    static_assert(!(ASTR || BSTR) || ES == 2, "transposing reads take 16-bit values");

    // epilogue slab of one wave: 32 rows of WN values, padded by 4
    constexpr int SP = WN + 4;
    constexpr int SLAB = 32 * SP * 4;
    constexpr int LDS_BYTES = NS * STAGE > NW * SLAB ? NS * STAGE : NW * SLAB;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS_BYTES];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Tile order: each XCD walks a contiguous run; within it, groups of
    // `group` row tiles go column by column, so the tiles in flight on an XCD
    // share both operands' rows in its L2.
    const int t = xcd_tile(blockIdx.x, g.tiles);
    const int per_group = g.group * g.tiles_n;
    const int grp = t / per_group;
    const int rows_here = min(g.group, g.tiles_m - grp * g.group);
    const int in = t - grp * per_group;
    const int m0 = (grp * g.group + in % rows_here) * TM;
    const int n0 = (in / rows_here) * TN;

    const int stage0 = blockIdx.y * g.kchunk;
    const int stage_end = min(g.nstages, stage0 + g.kchunk);

    // ---- load geometry: load i of this wave fills the 1 KiB LDS block
    // i*NW+wave of its operand's part of the stage
    const int row0 = wave * 16 + (lane >> 2);
    const int j = row_swizzle(row0, lane & 3);  // the same for every i
    auto rows_off = [&](int i, int first, int dim, int64_t ld) {
        const int r = row0 + i * NW * 16;
        return first + r < dim ? r * (int)ld + j * 16 : kOutOfRange;
    };
    auto cols_off = [&](auto td, int i, int first, int dim, int64_t ld) {
        constexpr int TD = decltype(td)::value;
        constexpr int CPR = TD / 8;             // chunks per inner row
        const int kr = (i * NW + wave) * (64 / CPR) + lane / CPR;
        const int c = (lane % CPR) ^ (col_swizzle<TD>(kr) << 2);
        return first + c * 8 < dim ? kr * (int)ld + c * 16 : kOutOfRange;
    };
    typedef Size<TM> TMc;
    typedef Size<TN> TNc;
    int a_off[AL], b_off[BL];
#pragma unroll
    for (int i = 0; i < AL; ++i)
        a_off[i] = ASTR ? cols_off(TMc{}, i, m0, g.M, g.lda) : rows_off(i, m0, g.M, g.lda);
#pragma unroll
    for (int i = 0; i < BL; ++i)
        b_off[i] = BSTR ? cols_off(TNc{}, i, n0, g.N, g.ldb) : rows_off(i, n0, g.N, g.ldb);

    // bases of the tile at the next stage to load
    const uint8_t *a_base = g.a + (ASTR ? (int64_t)m0 * ES + (int64_t)stage0 * BKE * g.lda
                                        : m0 * g.lda + (int64_t)stage0 * 64);
    const uint8_t *b_base = g.b + (BSTR ? (int64_t)n0 * ES + (int64_t)stage0 * BKE * g.ldb
                                        : n0 * g.ldb + (int64_t)stage0 * 64);
    const int64_t a_step = ASTR ? BKE * g.lda : 64, b_step = BSTR ? BKE * g.ldb : 64;

    const unsigned smem_lds = lds_address(smem);
    int issued = stage0;
    v4i a_rsrc, b_rsrc;
    unsigned lbase = 0;
    bool chunk_live = false;  // rows form: this lane's chunk lies inside the inner dimension

    // Loads of the next stage go to ring slot `slot`.  A stage past the end
    // loads zeros, so that every iteration issues the same number of loads.
    auto begin_stage = [&](int slot) {
        const bool live = issued < stage_end;
        // columns form: the range ends with the last inner row of the stage
        // and the last 16-byte chunk of it inside the matrix
        const int krows = live ? min(BKE, g.K - issued * BKE) : 0;
        a_rsrc = make_rsrc(a_base, ASTR ? (krows > 0 ? (krows - 1) * (int)g.lda + min(TM, (g.M - m0 + 7) & ~7) * ES : 0)
                                        : (live ? 0x7fffffff : 0));
        b_rsrc = make_rsrc(b_base, BSTR ? (krows > 0 ? (krows - 1) * (int)g.ldb + min(TN, (g.N - n0 + 7) & ~7) * ES : 0)
                                        : (live ? 0x7fffffff : 0));
        chunk_live = issued * 64 + j * 16 < g.kbytes;
        lbase = smem_lds + slot * STAGE + wave * 1024;
    };
    auto dma_one = [&](int i) {
        if (i < AL)
            load16_to_lds(a_rsrc, lbase + i * NW * 1024, ASTR || chunk_live ? a_off[i] : kOutOfRange);
        else
            load16_to_lds(b_rsrc, lbase + A_BYTES + (i - AL) * NW * 1024,
                          BSTR || chunk_live ? b_off[i - AL] : kOutOfRange);
    };
    auto end_stage = [&]() {
        ++issued;
        a_base += a_step;
        b_base += b_step;
    };

    const int wm = (wave / WGN) * WM;
    const int wn = (wave % WGN) * WN;

    typename Acc<T>::type acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
            acc[x][y] = typename Acc<T>::type{};

    // fragments, double-buffered in registers: [0, FM) from A, [FM, FM+FN) from B
    v4i frag[2][2][FM + FN];
    auto read_rows = [&](const uint8_t *base, int first, int ks) {
        const int row = first + (lane & 31);
        return *(const v4i *)&base[row * 64 + row_swizzle(row, ks * 2 + (lane >> 5)) * 16];
    };
    auto read_cols = [&](auto td, const uint8_t *base, int first, int ks) {
        constexpr int TD = decltype(td)::value;
        const int jj = lane & 15;
        const int col = first + ((lane >> 4) & 1) * 16 + (jj & 3) * 4;
        v4s r[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kr = ks * 16 + (lane >> 5) * 8 + h * 4 + (jj >> 2);
            const uint8_t *p = base + kr * (TD * 2) + (((col >> 3) ^ (col_swizzle<TD>(kr) << 2)) << 4) + (col & 7) * 2;
            r[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
        }
        return __builtin_bit_cast(v4i, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read_one = [&](int buf, int slot, int i) {
        const int ks = i / (FM + FN), f = i % (FM + FN);
        const uint8_t *base = smem + slot * STAGE;
        if (f < FM) {
            if constexpr (ASTR)
                frag[buf][ks][f] = read_cols(TMc{}, base, wm + f * 32, ks);
            else
                frag[buf][ks][f] = read_rows(base, wm + f * 32, ks);
        } else {
            if constexpr (BSTR)
                frag[buf][ks][f] = read_cols(TNc{}, base + A_BYTES, wn + (f - FM) * 32, ks);
            else
                frag[buf][ks][f] = read_rows(base + A_BYTES, wn + (f - FM) * 32, ks);
        }
    };
    auto mfma_one = [&](int buf, int i) {
        const int ks = i / (FM * FN), x = (i / FN) % FM, y = i % FN;
        acc[x][y] = mfma32<T>(frag[buf][ks][FM + y], frag[buf][ks][x], acc[x][y]);
    };

    // One stage: the matrix instructions of stage `it` (fragments in registers
    // `buf`) are interleaved with the loads of stage it+NS into the slot that
    // stage `it` vacated and the fragment reads of stage it+1.  The first ones
    // need only registers and go out before the wait and the barrier.
    constexpr int NOTHER = LPS + NRD;
    constexpr int PRE = NMF / 4;
    int cur_slot = 0;
    auto body = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PRE; ++i)
            mfma_one(buf, i);
        __builtin_amdgcn_sched_barrier(0);
        wait_vm_lgkm0<(NS - 2) * LPS>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        begin_stage(cur_slot);
        const int nslot = cur_slot + 1 == NS ? 0 : cur_slot + 1;
#pragma unroll
        for (int i = PRE; i < NMF; ++i) {
            mfma_one(buf, i);
#pragma unroll
            for (int o = (i - PRE) * NOTHER / (NMF - PRE); o < (i - PRE + 1) * NOTHER / (NMF - PRE); ++o) {
                if (o < LPS)
                    dma_one(o);
                else
                    read_one(buf ^ 1, nslot, o - LPS);
            }
        }
        end_stage();
        cur_slot = nslot;
        __builtin_amdgcn_sched_barrier(0);
    };

    // An odd count runs one extra stage of zeros, so that the loop body holds
    // two stages, one per fragment buffer, without a branch.
    const int nloop = (max(stage_end - stage0, 0) + 1) & ~1;
    if (nloop > 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            begin_stage(s);
#pragma unroll
            for (int i = 0; i < LPS; ++i)
                dma_one(i);
            end_stage();
        }
        wait_vm_lgkm0<(NS - 1) * LPS>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int i = 0; i < NRD; ++i)
            read_one(0, 0, i);
        for (int it = 0; it < nloop; it += 2) {
            body(0);
            body(1);
        }
        wait_vm_lgkm0<0>();  // the trailing loads of zeros still write to the ring
    }
    __syncthreads();

    // ---- epilogue: 32-row slabs through the wave's own LDS -----------------
    float *slab = (float *)(smem + wave * SLAB);
    constexpr int CPR = WN / 8;                 // 8-column chunks per slab row
    static_assert(64 % CPR == 0, "a lane keeps its columns over all rows");
    const int cc = (lane % CPR) * 8;
    const int n = n0 + wn + cc;
    const int cnt = g.N - n;                    // columns of this chunk inside the matrix (8 or more: all)
    float bs[8], ws[8];
    if (!g.part && cnt > 0)
        column_params(g.epi, n, cnt, bs, ws);
    auto finish_slab = [&](auto xc) __attribute__((always_inline)) {
        constexpr int x = decltype(xc)::value;
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                typename Acc<T>::type &v = acc[x][y];
                v4f o;
                if constexpr (ES == 1) {
                    // partial sums stay integers (their bits travel as floats)
                    const v4i iv = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                    o = g.part ? __builtin_bit_cast(v4f, iv) : v4f{(float)iv.x, (float)iv.y, (float)iv.z, (float)iv.w};
                } else {
                    o = v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                }
                *(v4f *)&slab[(lane & 31) * SP + y * 32 + 8 * q + 4 * (lane >> 5)] = o;
            }
        // one wave's LDS operations run in order: only the compiler must not
        // move the reads up
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        constexpr int RS = 64 / CPR;            // rows apart of a lane's chunks
        constexpr int ITS = 32 / RS, U = ITS < 4 ? ITS : 4;
#pragma unroll 1
        for (int it = 0; it < ITS; it += U) {
            const int r = it * RS + lane / CPR;
            const int m = m0 + wm + x * 32 + r;
            float v[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                *(v4f *)&v[u][0] = *(const v4f *)&slab[(r + u * RS) * SP + cc];
                *(v4f *)&v[u][4] = *(const v4f *)&slab[(r + u * RS) * SP + cc + 4];
            }
            if (cnt <= 0)
                continue;
            if (g.part) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (m + u * RS < g.M) {
                        float *p = (float *)g.part + blockIdx.y * g.part_stride + (int64_t)(m + u * RS) * g.part_ld + n;
                        *(v4f *)p = *(v4f *)&v[u][0];
                        *(v4f *)(p + 4) = *(v4f *)&v[u][4];
                    }
            } else {
                finish8<ES == 1, U>(g.epi, m, RS, g.M, n, cnt, v, bs, ws);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    static_assert(FM == 1 || FM == 2 || FM == 4, "slabs");
    finish_slab(Size<0>{});
    if constexpr (FM >= 2)
        finish_slab(Size<1>{});
    if constexpr (FM >= 4) {
        finish_slab(Size<2>{});
        finish_slab(Size<3>{});
    }
}

// Sum of a split product's partial copies, in the order of the splits, and the
// epilogue.  One thread takes eight columns of one row.
template <bool INT>
__global__ __launch_bounds__(256) void split_finish_kernel(const GemmArgs g, int nsplit)
{
    const int cpr = g.part_ld / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / cpr;
    const int n = (int)(i - m * cpr) * 8;
    if (m >= g.M || n >= g.N)
        return;
    const float *p = (const float *)g.part + m * g.part_ld + n;
    float v[1][8];
    if constexpr (INT) {
        v4i s0 = *(const v4i *)p, s1 = *(const v4i *)(p + 4);
        for (int z = 1; z < nsplit; ++z) {
            s0 += *(const v4i *)(p + z * g.part_stride);
            s1 += *(const v4i *)(p + z * g.part_stride + 4);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[0][k] = (float)s0[k];
            v[0][4 + k] = (float)s1[k];
        }
    } else {
        v4f s0 = *(const v4f *)p, s1 = *(const v4f *)(p + 4);
        for (int z = 1; z < nsplit; ++z) {
            s0 += *(const v4f *)(p + z * g.part_stride);
            s1 += *(const v4f *)(p + z * g.part_stride + 4);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[0][k] = s0[k];
            v[0][4 + k] = s1[k];
        }
    }
    float bs[8], ws[8];
    column_params(g.epi, n, g.N - n, bs, ws);
    finish8<INT, 1>(g.epi, m, 1, g.M, n, g.N - n, v, bs, ws);
}

}  // namespace dense
