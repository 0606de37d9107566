// Tiled matrix product for gfx950: C[m, n] = sum_k A(m, k) B(n, k) with the
// dense layer's epilogue, operands BF16, FP16 (32-bit float sums) or INT8
// (32-bit integer sums).
//
// A workgroup of four waves computes a TM x TN tile.  Both operands stream from
// memory straight into rings of LDS stages (buffer_load ... lds, 16 bytes a
// lane, no staging registers); one barrier per stage publishes the stage that
// landed and retires the slots the next loads overwrite.  A stage is 128 bytes
// of the inner dimension: 64 BF16/FP16 or 128 INT8 values.  (Stages of 64 bytes
// make twice the requests to the cache for the same data: 709 us against 605
// for 8192^3 BF16 zeros.  The 256x256 tile has three slots for A and two for B,
// which fills the 160 KB: two for both leave 100 us of waits there.)
//
// An operand is stored in one of two ways:
//  * rows (STR false): the inner dimension is contiguous.  LDS holds 128-byte
//    rows whose 16-byte chunks are permuted so that the 16 rows a fragment read
//    touches cover the banks once.
//  * columns (STR true, 16-bit types): the inner dimension has the stride.
//    LDS holds one row of TM (TN) values per inner index, 32-byte groups
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
// Epilogue.  A lane holds one of 16 columns of each 16x16 block.  With B in rows
// form, lane i reads the fragment of block y from column FN i + y of the wave's
// part of B (FN blocks of 16 columns), so that it ends up with FN consecutive
// columns of a row and sixteen lanes with the row's whole segment of the wave's
// tile: bias, activation, residual and stores are 16 bytes a lane (FN = 8) and
// 256 contiguous bytes a row, straight from the accumulators.  Tiles at an edge,
// partial sums, 32-bit outputs and B in columns form (whose transposing reads
// cannot give that order) turn through LDS.
#pragma once

#include "colsum.hpp"
#include "dense_common.hpp"

namespace dense {

// Bytes of the inner dimension per stage: two halves, one matrix instruction deep each
constexpr int kStageBytes = 128;

struct GemmArgs {
    const uint8_t *a, *b;
    int64_t lda, ldb;      // bytes between rows (rows form) or inner indices (columns form)
    int M, N;
    int kbytes;            // inner dimension in bytes of a rows-form operand, a multiple of 16
    int K;                 // inner dimension in elements
    int nstages;           // stages of kStageBytes
    int kchunk;            // stages per split
    int tiles_m, tiles_n, tiles;
    int group;             // row tiles per group of the tile order
    int64_t part_stride;   // split: 32-bit values per partial copy
    int part_ld;
    void *part;            // split: partial sums [split][M][part_ld], or null
    Epilogue epi;
};

// acc += the 16x16 product, in place in accumulation registers.  Written as an
// instruction because the register allocator otherwise gives the result other
// registers than the addend and copies all of them around the loop.  The
// compiler then knows nothing of its latency: operands come from LDS reads
// (which it does wait for), one accumulator's instructions are FM*FN apart, and
// the kernel waits itself before it reads the sums (mfma_drain, tie).
// VGPR: the sums lie in ordinary registers instead.
template <typename T, bool VGPR>
__device__ __forceinline__ void mfma16_acc(v4i a, v4i b, typename Acc4<T>::type &c)
{
#define DENSE_MFMA(NAME)                                                             \
    if constexpr (VGPR)                                                              \
        asm volatile("v_mfma_" NAME " %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));   \
    else                                                                             \
        asm volatile("v_mfma_" NAME " %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b))
    if constexpr (sizeof(T) == 1) {
        DENSE_MFMA("i32_16x16x64_i8");
    } else if constexpr (__is_same(T, bf16)) {
        DENSE_MFMA("f32_16x16x32_bf16");
    } else {
        DENSE_MFMA("f32_16x16x32_f16");
    }
#undef DENSE_MFMA
}

// More wait states than a result of the instruction above needs.
__device__ __forceinline__ void mfma_drain()
{
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
}

// Makes what reads a sum depend on a statement after the drain: without it, only
// the scheduler's habits keep a copy of the sum from being placed before the drain.
template <bool VGPR, typename A>
__device__ __forceinline__ void tie(A &c)
{
    if constexpr (VGPR)
        asm volatile("" : "+v"(c));
    else
        asm volatile("" : "+a"(c));
}

// Columns form: permutation of inner row kr's 32-byte groups.  32 lanes of a
// transposing read take 32 bytes each of the eight rows k0 .. k0+3 and
// k0+8 .. k0+11, which must cover the banks once: rows of 256 bytes and more
// all start at bank 0, two 128-byte rows cover the banks once.
template <int TD>
__device__ __forceinline__ int col_swizzle(int kr)
{
    return TD >= 128 ? (kr & 3) | ((kr >> 1) & 4) : ((kr >> 1) & 1) | ((kr >> 2) & 2);
}

// B in rows form, in the order of the epilogue: a fragment read takes the rows
// FN i + y, i = 0 .. 15, all of one parity.  Two 128-byte rows make up the
// banks' 256 bytes, so the 16 slots of a pair of rows are permuted together, by
// the pair's number in units of the pairs a read skips.
template <int FN>
__device__ __forceinline__ int pair_swizzle(int pair, int slot)
{
    return slot ^ ((pair / (FN / 2)) & 15);
}

template <typename T> struct Type { typedef T type; };

// C values as the bits of 16-bit output type O, and back
template <typename O, int C> struct Bits { typedef O vec __attribute__((ext_vector_type(C))); };
template <int C> struct Words;
template <> struct Words<8> { typedef v4i type; };
template <> struct Words<4> { typedef int type __attribute__((ext_vector_type(2))); };
template <> struct Words<2> { typedef int type; };

template <int C>
__device__ __forceinline__ void buffer_store(typename Words<C>::type v, __amdgpu_buffer_rsrc_t r, int voff, int soff)
{
    if constexpr (C == 8)
        __builtin_amdgcn_raw_buffer_store_b128(v, r, voff, soff, 0);
    else if constexpr (C == 4)
        __builtin_amdgcn_raw_buffer_store_b64(v, r, voff, soff, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(v, r, voff, soff, 0);
}

template <int C>
__device__ __forceinline__ typename Words<C>::type buffer_load(__amdgpu_buffer_rsrc_t r, int voff, int soff)
{
    if constexpr (C == 8)
        return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
    else if constexpr (C == 4)
        return __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
}

// The epilogue of a wave's whole 16 FM x 16 FN tile at (m, n), values of 16-bit
// type O, straight from the accumulators: lane l holds rows 16 x + 4 (l / 16) + u
// and columns (l % 16) FN + y.
template <typename T, typename O, int ACT, int FM, int FN>
__device__ __forceinline__ void finish_whole(const Epilogue &e, typename Acc4<T>::type (&acc)[FM][FN], int m, int n,
                                             int lane)
{
    typedef typename Words<FN>::type words;
    typedef typename Bits<O, FN>::vec vec;
    const int col = (lane & 15) * FN, row = 4 * (lane >> 4);
    float bs[FN], ws[FN];
    column_params(e, n + col, FN, bs, ws);
    auto view = [&](const void *p, int64_t ld) {
        return __builtin_amdgcn_make_buffer_rsrc((O *)const_cast<void *>(p) + m * ld + n, (short)0, 0x7fffffff, 0x00020000);
    };
    // residuals of four blocks of rows at a time (64 registers)
    constexpr int RG = FM < 4 ? FM : 4;
    words res[RG][4];
    const __amdgpu_buffer_rsrc_t rsd = view(e.residual, e.ldr);
    const int vr = (row * (int)e.ldr + col) * 2;
    const __amdgpu_buffer_rsrc_t out = view(e.out, e.ldo), pre = view(e.preact, e.ldp);
    const int vo = (row * (int)e.ldo + col) * 2, vp = (row * (int)e.ldp + col) * 2;
    for_each<FM>([&](auto xc) __attribute__((always_inline)) {
        constexpr int x = decltype(xc)::value;
        if constexpr (x % RG == 0) {
            if (e.residual)
#pragma unroll
                for (int i = 0; i < RG; ++i)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        res[i][u] = buffer_load<FN>(rsd, vr, (16 * (x + i) + u) * (int)e.ldr * 2);
        }
        float xs[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if constexpr (sizeof(T) == 1) {
            if (e.x_scale)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    xs[u] = e.x_scale[m + 16 * x + row + u];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float z[FN];
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                if constexpr (sizeof(T) == 1)
                    z[y] = __builtin_fmaf((float)acc[x][y][u], xs[u] * ws[y], bs[y]);
                else
                    z[y] = acc[x][y][u] + bs[y];
            }
            if (e.preact) {
                vec b;
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    b[y] = (O)z[y];
                buffer_store<FN>(__builtin_bit_cast(words, b), pre, vp, (16 * x + u) * (int)e.ldp * 2);
            }
#pragma unroll
            for (int y = 0; y < FN; ++y)
                z[y] = activate<ACT>(z[y]);
            if (e.residual) {
                const vec b = __builtin_bit_cast(vec, res[x % RG][u]);
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    z[y] += (float)b[y];
            }
            vec b;
#pragma unroll
            for (int y = 0; y < FN; ++y)
                b[y] = (O)z[y];
            buffer_store<FN>(__builtin_bit_cast(words, b), out, vo, (16 * x + u) * (int)e.ldo * 2);
        }
        __builtin_amdgcn_sched_barrier(0);  // one block at a time, or the values of several are held at once
    });
}

// NSA, NSB: slots of the operands' rings, NSB or NSB + 1 and NSB; LH: loads per
// thread of a stage that go out in the half that frees their slots (the others
// in the half after it)
template <typename T, int TM, int TN, int WGM, int WGN, int NSA, int NSB, int LH, bool ASTR, bool BSTR>
struct TileCfg {
    static constexpr int NW = WGM * WGN;
    static constexpr int RING = (NSA * TM + NSB * TN) * kStageBytes;
    static constexpr int WM = TM / WGM, WN = TN / WGN;
    // epilogue slab of one wave: up to 64 rows of WN values, padded by 4
    static constexpr int SP = WN + 4;
    static constexpr int SLAB = (WM < 64 ? WM : 64) * SP * 4;
    static constexpr int LDS_BYTES = RING > NW * SLAB ? RING : NW * SLAB;
};

// One tile of one split.  smem: TileCfg::LDS_BYTES of LDS, aligned to 1024
template <typename T, int TM, int TN, int WGM, int WGN, int NSA, int NSB, int LH, bool ASTR, bool BSTR>
__device__ __forceinline__ void gemm_tile(const GemmArgs &g, uint8_t *smem, int block, int split)
{
    typedef TileCfg<T, TM, TN, WGM, WGN, NSA, NSB, LH, ASTR, BSTR> Cfg;
    constexpr int NW = Cfg::NW;
    constexpr int ES = sizeof(T);
    constexpr int SB = kStageBytes;
    constexpr int BKE = SB / ES;                // inner elements per stage
    constexpr int RPB = 1024 / SB;              // rows-form rows per 1 KiB block
    constexpr int AL = TM / (NW * RPB), BL = TN / (NW * RPB), LPS = AL + BL;
    constexpr int A_BYTES = TM * SB, B_BYTES = TN * SB;
    constexpr int WM = Cfg::WM, WN = Cfg::WN;
    constexpr int FM = WM / 16, FN = WN / 16;
    constexpr int NMF = FM * FN;                // matrix instructions per half
    constexpr int NRD = FM + FN;                // fragment reads per half
    static_assert(AL >= 1 && BL >= 1 && FM >= 2 && FN >= 2, "tile too small");
    static_assert(NSB >= 2 && (NSA == NSB || (NSA == 3 && NSB == 2)), "ring slots");
    static_assert((NSA - 1) * AL + (NSB - 1) * BL < 64, "pipeline depth");
    static_assert(LH <= LPS, "loads of a stage");
    constexpr int A_RING = NSA * A_BYTES;
    static_assert(!(ASTR || BSTR) || ES == 2, "transposing reads take 16-bit values");
    constexpr int SP = Cfg::SP, SLAB = Cfg::SLAB;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Tile order: each XCD walks a contiguous run; within it, groups of
    // `group` row tiles go column by column, so the tiles in flight on an XCD
    // share both operands' rows in its L2.
    const int t = xcd_tile(block, g.tiles);
    const int per_group = g.group * g.tiles_n;
    const int grp = t / per_group;
    const int rows_here = min(g.group, g.tiles_m - grp * g.group);
    const int in = t - grp * per_group;
    const int m0 = (grp * g.group + in % rows_here) * TM;
    const int n0 = (in / rows_here) * TN;

    const int stage0 = split * g.kchunk;
    const int stage_end = min(g.nstages, stage0 + g.kchunk);

    // ---- load geometry: load i of this wave fills the 1 KiB LDS block
    // i*NW+wave of its operand's part of the stage
    const int row0 = wave * RPB + lane / (SB / 16);
    const int j = row_swizzle<SB>(row0, lane % (SB / 16));  // the same for every i
    auto a_rows_off = [&](int i) {
        const int r = row0 + i * NW * RPB;
        return m0 + r < g.M ? r * (int)g.lda + j * 16 : kOutOfRange;
    };
    auto b_slot_of = [&](int i) {               // row * 8 + chunk that belongs at this lane's place
        const int pair = (i * NW + wave) * (RPB / 2) + (lane >> 4);
        return pair * 16 + pair_swizzle<FN>(pair, lane & 15);
    };
    auto b_rows_off = [&](int i) {
        const int rc = b_slot_of(i), r = rc >> 3;
        return n0 + r < g.N ? r * (int)g.ldb + (rc & 7) * 16 : kOutOfRange;
    };
    auto cols_off = [&](auto td, int i, int first, int dim, int64_t ld) {
        constexpr int TD = decltype(td)::value;
        constexpr int CPR = TD / 8;             // chunks per inner row
        const int kr = (i * NW + wave) * (64 / CPR) + lane / CPR;
        const int c = (lane % CPR) ^ (col_swizzle<TD>(kr) << 1);
        return first + c * 8 < dim ? kr * (int)ld + c * 16 : kOutOfRange;
    };
    typedef Size<TM> TMc;
    typedef Size<TN> TNc;
    int a_off[AL], b_off[BL];
#pragma unroll
    for (int i = 0; i < AL; ++i)
        a_off[i] = ASTR ? cols_off(TMc{}, i, m0, g.M, g.lda) : a_rows_off(i);
#pragma unroll
    for (int i = 0; i < BL; ++i)
        b_off[i] = BSTR ? cols_off(TNc{}, i, n0, g.N, g.ldb) : b_rows_off(i);

    // The operands' streams: buffer resource and ring slot of the next stage to
    // load.  `full` is the range of a whole stage: without limit in rows form
    // (offsets past an edge were set out of range above), up to the last chunk
    // of the last inner row in columns form, where a range also ends the last,
    // partial stage.
    const unsigned smem_lds = lds_address(smem);
    const int a_cols = min(TM, (g.M - m0 + 7) & ~7) * ES, b_cols = min(TN, (g.N - n0 + 7) & ~7) * ES;
    const int a_full = ASTR ? (BKE - 1) * (int)g.lda + a_cols : 0x7fffffff;
    const int b_full = BSTR ? (BKE - 1) * (int)g.ldb + b_cols : 0x7fffffff;
    const int64_t a_step = ASTR ? BKE * g.lda : SB, b_step = BSTR ? BKE * g.ldb : SB;
    // the stage in which the inner dimension ends before the stage does
    const int tail = (ASTR || BSTR ? g.K % BKE : g.kbytes % SB) ? g.nstages - 1 : -1;
    const int tail_k = g.K - tail * BKE;    // inner elements of it
    v4i a_rsrc = make_rsrc(g.a + (ASTR ? (int64_t)m0 * ES + stage0 * a_step : m0 * g.lda + stage0 * a_step), a_full);
    v4i b_rsrc = make_rsrc(g.b + (BSTR ? (int64_t)n0 * ES + stage0 * b_step : n0 * g.ldb + stage0 * b_step), b_full);
    int a_next = stage0, b_next = stage0, a_fill = 0, b_fill = 0;
    unsigned a_lds = smem_lds + wave * 1024, b_lds = smem_lds + A_RING + wave * 1024;

    // Before a stage's first load: its range (a stage past the end loads zeros,
    // so that every iteration issues the same number of loads), and in the tail
    // stage what lies past the inner dimension set out of range -- for good,
    // since nothing is loaded after it.
    auto open_a = [&]() {
        a_rsrc.z = a_next < stage_end ? a_full : 0;
        if (a_next == tail) {
            if constexpr (ASTR) {
                a_rsrc.z = a_next < stage_end ? (tail_k - 1) * (int)g.lda + a_cols : 0;
            } else {
                const bool in = a_next * SB + j * 16 < g.kbytes;
#pragma unroll
                for (int i = 0; i < AL; ++i)
                    a_off[i] = in ? a_off[i] : kOutOfRange;
            }
        }
    };
    auto open_b = [&]() {
        b_rsrc.z = b_next < stage_end ? b_full : 0;
        if (b_next == tail) {
            if constexpr (BSTR) {
                b_rsrc.z = b_next < stage_end ? (tail_k - 1) * (int)g.ldb + b_cols : 0;
            } else {
#pragma unroll
                for (int i = 0; i < BL; ++i)
                    b_off[i] = b_next * SB + (b_slot_of(i) & 7) * 16 < g.kbytes ? b_off[i] : kOutOfRange;
            }
        }
    };
    // After its last load: the base and the slot of the next one.
    auto advance = [&](v4i &r, int64_t step) {
        const uint64_t base = ((uint64_t)(unsigned)r.y << 32 | (unsigned)r.x) + step;
        r.x = (int)(unsigned)base;
        r.y = (int)(base >> 32);
    };
    auto next_a = [&]() {
        ++a_next;
        a_fill = a_fill + 1 == NSA ? 0 : a_fill + 1;
        a_lds = smem_lds + wave * 1024 + a_fill * A_BYTES;
    };
    auto next_b = [&]() {
        ++b_next;
        b_fill = b_fill + 1 == NSB ? 0 : b_fill + 1;
        b_lds = smem_lds + A_RING + wave * 1024 + b_fill * B_BYTES;
    };
    // Loads 0 .. BL-1 of a stage are B's: with one slot less, it is needed sooner.
    auto aim = [&](auto ic) {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < BL)
            set_lds_target<i * NW * 1024>(b_lds);
        else if constexpr (i < LPS)
            set_lds_target<(i - BL) * NW * 1024>(a_lds);
    };
    auto load_one = [&](auto ic) {
        constexpr int i = decltype(ic)::value;
        if constexpr (i < BL)
            load16_to_lds(b_rsrc, b_off[i]);
        else
            load16_to_lds(a_rsrc, a_off[i - BL]);
    };

    const int wm = (wave / WGN) * WM;
    const int wn = (wave % WGN) * WN;

    typename Acc4<T>::type acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
            acc[x][y] = typename Acc4<T>::type{};

    // fragments of a half, double-buffered in registers: [0, FN) from B,
    // [FN, FN+FM) from A
    v4i frag[2][FN + FM];
    auto read_rows = [&](const uint8_t *base, int first, int half) {
        const int row = first + (lane & 15);
        return *(const v4i *)&base[row * SB + row_swizzle<SB>(row, half * 4 + (lane >> 4)) * 16];
    };
    auto read_b_rows = [&](const uint8_t *base, int y, int half) {
        const int row = wn + (lane & 15) * FN + y;
        return *(const v4i *)&base[(row >> 1) * 256 + pair_swizzle<FN>(row >> 1, (row & 1) * 8 + half * 4 + (lane >> 4)) * 16];
    };
    auto read_cols = [&](auto td, const uint8_t *base, int first, int half) {
        constexpr int TD = decltype(td)::value;
        const int jj = lane & 15;
        const int col = first + (jj & 3) * 4;
        v4s r[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int kr = half * 32 + (lane >> 4) * 8 + h * 4 + (jj >> 2);
            const uint8_t *p = base + kr * (TD * 2) + (((col >> 3) ^ (col_swizzle<TD>(kr) << 1)) << 4) + (col & 7) * 2;
            r[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
        }
        return __builtin_bit_cast(v4i, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read_one = [&](int buf, int a_slot, int b_slot, int half, int i) {
        if (i < FN) {
            const uint8_t *base = smem + A_RING + b_slot * B_BYTES;
            if constexpr (BSTR)
                frag[buf][i] = read_cols(TNc{}, base, wn + i * 16, half);
            else
                frag[buf][i] = read_b_rows(base, i, half);
        } else {
            const uint8_t *base = smem + a_slot * A_BYTES;
            if constexpr (ASTR)
                frag[buf][i] = read_cols(TMc{}, base, wm + (i - FN) * 16, half);
            else
                frag[buf][i] = read_rows(base, wm + (i - FN) * 16, half);
        }
    };
    // A wave of the 256x256 tile has 256 sums, all the accumulation registers there
    // are; one row of blocks is kept in ordinary ones, since with none to spare the
    // allocator moves sums about inside the loop.
    constexpr int kLastAcc = FM * FN == 64 ? FM - 1 : FM;  // blocks of rows before it are in accumulation registers
    auto mfma_one = [&](int buf, auto ic) __attribute__((always_inline)) {
        constexpr int x = decltype(ic)::value / FN, y = decltype(ic)::value % FN;
        constexpr bool vgpr = x >= kLastAcc;
        if constexpr (BSTR)
            mfma16_acc<T, vgpr>(frag[buf][y], frag[buf][FN + x], acc[x][y]);
        else
            mfma16_acc<T, vgpr>(frag[buf][FN + x], frag[buf][y], acc[x][y]);
    };

    // A half: its matrix instructions (fragments in registers `buf`) with the
    // reads of the next half's fragments and the loads between them.  In the
    // last half of a stage the next half is the next stage's first: a wait and
    // a barrier come before its reads, and after them this stage's slots are
    // free, so the loads of the stage NSB (NSA) ahead go there, the last
    // LPS - LH of them in the next stage's first half.  The first PRE matrix
    // instructions need only registers and go out before the wait.
    //
    // The order is pinned instruction by instruction.  A wave is alone on its
    // SIMD (or shares it with one other), a matrix instruction lasts 16 cycles
    // and every other instruction takes 4 to issue: more than three of them
    // between two matrix instructions leave the matrix unit idle.  So reads,
    // loads, the writes of M0 and the scalar work of a new stage go into
    // different gaps.
    constexpr int PRE = NMF / 4;
    int a_slot = 0, b_slot = 0;
    auto half = [&](auto hc) __attribute__((always_inline)) {
        constexpr int h = decltype(hc)::value, buf = h;
        constexpr bool last = h == 1;
        constexpr int first = last ? PRE : 0;   // matrix instructions before reads may start
        constexpr int np = NMF - first, nr = np * 3 / 4 > 0 ? np * 3 / 4 : 1;
        constexpr int l0 = last ? 0 : LH, nl = last ? LH : LPS - LH;
        const int an = a_slot + 1 == NSA ? 0 : a_slot + 1, bn = b_slot + 1 == NSB ? 0 : b_slot + 1;
        for_each<NMF>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            if constexpr (last && i == PRE) {
                wait_vm_lgkm0<(NSA - 2) * AL + (NSB - 2) * BL>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
            mfma_one(buf, ic);
            if constexpr (last && i < PRE) {
                // the stage whose loads start after the barrier
                constexpr int step = PRE / 6 > 0 ? PRE / 6 : 1;
                if constexpr (i == 0)
                    advance(b_rsrc, b_step);
                if constexpr (i == (step < PRE ? step : 0))
                    next_b();
                if constexpr (i == (2 * step < PRE ? 2 * step : 0))
                    open_b();
                if constexpr (i == (3 * step < PRE ? 3 * step : 0))
                    advance(a_rsrc, a_step);
                if constexpr (i == (4 * step < PRE ? 4 * step : 0))
                    next_a();
                if constexpr (i == (5 * step < PRE ? 5 * step : 0))
                    open_a();
            }
            if constexpr (i == (first > 0 ? first - 1 : 0) && nl > 0)
                aim(Size<l0>{});
            if constexpr (i >= first) {
                constexpr int p = i - first;
                constexpr int r0 = p * NRD / nr < NRD ? p * NRD / nr : NRD;
                constexpr int r1 = (p + 1) * NRD / nr < NRD ? (p + 1) * NRD / nr : NRD;
                for_each<r1 - r0>([&](auto oc) __attribute__((always_inline)) {
                    read_one(buf ^ 1, last ? an : a_slot, last ? bn : b_slot, last ? 0 : h + 1, r0 + decltype(oc)::value);
                });
                constexpr int d0 = p * nl / np, d1 = (p + 1) * nl / np;
                for_each<d1 - d0>([&](auto oc) __attribute__((always_inline)) {
                    constexpr int o = l0 + d0 + decltype(oc)::value;
                    load_one(Size<o>{});
                    if constexpr (o + 1 < l0 + nl)
                        aim(Size<o + 1>{});
                });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (last) {
            a_slot = an;
            b_slot = bn;
        }
    };

    const int nloop = max(stage_end - stage0, 0);
    if (nloop > 0) {
        // The rings filled in the order of the loop: stage by stage, B before
        // A, and A's extra slot first of all
        auto load_part = [&](auto from, auto to) __attribute__((always_inline)) {
            for_each<decltype(to)::value - decltype(from)::value>([&](auto ic) __attribute__((always_inline)) {
                typedef Size<decltype(from)::value + decltype(ic)::value> I;
                aim(I{});
                asm volatile("s_nop 0");
                load_one(I{});
            });
        };
        if constexpr (NSA > NSB) {
            open_a();
            load_part(Size<BL>{}, Size<LPS>{});
            advance(a_rsrc, a_step);
            next_a();
        }
        for_each<NSB>([&](auto sc) __attribute__((always_inline)) {
            if constexpr (decltype(sc)::value > 0) {
                advance(b_rsrc, b_step);
                next_b();
                advance(a_rsrc, a_step);
                next_a();
            }
            open_b();
            open_a();
            load_part(Size<0>{}, Size<(decltype(sc)::value < NSB - 1 ? LPS : LH)>{});
        });
        // everything but the loads after stage 0's
        wait_vm_lgkm0<(NSB - 2) * LPS + LH + (NSA > NSB ? AL : 0)>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int i = 0; i < NRD; ++i)
            read_one(0, 0, 0, 0, i);
        for (int it = 0; it < nloop; ++it) {
            half(Size<0>{});
            half(Size<1>{});
        }
        wait_vm_lgkm0<0>();  // the trailing loads of zeros still write to the rings
        mfma_drain();
        for_each<NMF>([&](auto ic) __attribute__((always_inline)) {
            constexpr int x = decltype(ic)::value / FN, y = decltype(ic)::value % FN;
            tie<(x >= kLastAcc)>(acc[x][y]);
        });
    }
    __syncthreads();

    // ---- epilogue, whole tile, 16-bit output, B in rows form: straight from the
    // accumulators, one piece of code per activation without branches inside
    const Epilogue &e = g.epi;
    if constexpr (!BSTR) {
        // row strides that reach past a tile's 31-bit offsets take the other path
        const bool whole = !g.part && m0 + TM <= g.M && n0 + TN <= g.N && e.tile_offsets;
        if (whole && (ES == 2 ? e.out_dt == Code<T>::v : e.out_dt != DENSE_FP32)) {
            auto run = [&](auto act, auto out) __attribute__((always_inline)) {
                typedef typename decltype(out)::type O;
                finish_whole<T, O, decltype(act)::value, FM, FN>(e, acc, m0 + wm, n0 + wn, lane);
            };
            auto by_act = [&](auto out) __attribute__((always_inline)) {
                if (e.act == DENSE_ACT_NONE)
                    run(Size<DENSE_ACT_NONE>{}, out);
                else if (e.act == DENSE_ACT_RELU)
                    run(Size<DENSE_ACT_RELU>{}, out);
                else if (e.act == DENSE_ACT_GELU)
                    run(Size<DENSE_ACT_GELU>{}, out);
                else if (e.act == DENSE_ACT_GELU_TANH)
                    run(Size<DENSE_ACT_GELU_TANH>{}, out);
                else
                    run(Size<DENSE_ACT_SILU>{}, out);
            };
            if constexpr (ES == 2) {
                by_act(Type<T>{});
            } else if (e.out_dt == DENSE_BF16) {
                by_act(Type<bf16>{});
            } else {
                by_act(Type<f16>{});
            }
            return;
        }
    }

    // ---- epilogue, anything else: the sums go to the wave's own part of LDS, up
    // to 64 rows at a time, and one loop takes them from there row by row
    float *slab = (float *)(smem + wave * SLAB);
    constexpr int CPR = WN / 8;                 // 8-column chunks per row
    static_assert(64 % CPR == 0, "a lane keeps its columns over all rows");
    const int cc = (lane % CPR) * 8;
    const int n = n0 + wn + cc;
    const int cnt = g.N - n;                    // columns of this chunk inside the matrix (8 or more: all)
    float bs[8], ws[8];
    if (!g.part && cnt > 0)
        column_params(e, n, cnt, bs, ws);
    for_each<(FM + 3) / 4>([&](auto sc) __attribute__((always_inline)) {
        constexpr int x0 = decltype(sc)::value * 4, XS = FM - x0 < 4 ? FM - x0 : 4;
        for_each<XS * FN>([&](auto bc) __attribute__((always_inline)) {
            constexpr int x = decltype(bc)::value / FN, y = decltype(bc)::value % FN;
            const typename Acc4<T>::type v = acc[x0 + x][y];
            v4f o;
            if constexpr (ES == 1)  // partial sums stay integers (their bits travel as floats)
                o = g.part ? __builtin_bit_cast(v4f, v) : v4f{(float)v.x, (float)v.y, (float)v.z, (float)v.w};
            else
                o = v;
            if constexpr (BSTR) {
                *(v4f *)&slab[(x * 16 + (lane & 15)) * SP + y * 16 + 4 * (lane >> 4)] = o;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    slab[(x * 16 + 4 * (lane >> 4) + u) * SP + (lane & 15) * FN + y] = o[u];
            }
        });
        // one wave's LDS operations run in order: only the compiler must not
        // move the reads up
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        constexpr int RS = 64 / CPR;            // rows apart of a lane's chunks
        constexpr int ITS = XS * 16 / RS, U = ITS < 4 ? ITS : 4;
#pragma unroll 1
        for (int it = 0; it < ITS; it += U) {
            const int r = it * RS + lane / CPR;
            const int m = m0 + wm + x0 * 16 + r;
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
                        float *p = (float *)g.part + split * g.part_stride + (int64_t)(m + u * RS) * g.part_ld + n;
                        *(v4f *)p = *(v4f *)&v[u][0];
                        *(v4f *)(p + 4) = *(v4f *)&v[u][4];
                    }
            } else {
                finish<ES == 1, U, 8>(e, m, RS, g.M, n, cnt, v, bs, ws);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    });
}

// OCC: workgroups a CU is to hold at a time (one wave of each per SIMD)
template <typename T, int TM, int TN, int WGM, int WGN, int NSA, int NSB, int LH, int OCC, bool ASTR, bool BSTR>
__global__ __launch_bounds__(64 * WGM * WGN, OCC) void gemm_kernel(const GemmArgs g)
{
    __shared__ __attribute__((aligned(1024)))
    uint8_t smem[TileCfg<T, TM, TN, WGM, WGN, NSA, NSB, LH, ASTR, BSTR>::LDS_BYTES];
    gemm_tile<T, TM, TN, WGM, WGN, NSA, NSB, LH, ASTR, BSTR>(g, smem, blockIdx.x, blockIdx.y);
}

// Both products of the gradients, neither of them split, and the last step of
// the bias gradient, in one launch: where they are a few microseconds each the
// gaps between launches and the CUs that one alone leaves idle cost as much.
struct PairArgs {
    GemmArgs dx, dw;
    ColSumArgs sum;   // columns 0: no bias gradient
};

template <typename T, int TM, int TN, int WGM, int WGN, int NSA, int NSB, int LH, int OCC>
__global__ __launch_bounds__(64 * WGM * WGN, OCC) void gemm_pair_kernel(const PairArgs p)
{
    constexpr int kCols = 64 * WGM * WGN / kSumGroups;
    __shared__ __attribute__((aligned(1024)))
    uint8_t smem[TileCfg<T, TM, TN, WGM, WGN, NSA, NSB, LH, false, true>::LDS_BYTES];
    const int b = blockIdx.x;
    if (b < p.dx.tiles)
        gemm_tile<T, TM, TN, WGM, WGN, NSA, NSB, LH, false, true>(p.dx, smem, b, 0);
    else if (b < p.dx.tiles + p.dw.tiles)
        gemm_tile<T, TM, TN, WGM, WGN, NSA, NSB, LH, true, true>(p.dw, smem, b - p.dx.tiles, 0);
    else
        column_sums<kCols>(p.sum, b - p.dx.tiles - p.dw.tiles, (float(*)[kCols + 1])smem);
}

template <bool INT> struct Choice { typedef float type; };
template <> struct Choice<true> { typedef int8_t type; };

// The partial copies of a product's sums, from the splits of its inner dimension
// and the terms of its first operand.
struct JoinArgs {
    int copies, first;  // those from `first` on are of the second term
    float scale;        // by which the second term is taken
};

// Sum of the partial copies, in their order, and the epilogue.  One thread takes
// eight columns of one row.
template <bool INT>
__global__ __launch_bounds__(256) void split_finish_kernel(const GemmArgs g, const JoinArgs j)
{
    const int cpr = g.part_ld / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = i / cpr;
    const int n = (int)(i - m * cpr) * 8;
    if (m >= g.M || n >= g.N)
        return;
    const float *p = (const float *)g.part + m * g.part_ld + n;
    typedef typename Acc4<typename Choice<INT>::type>::type vec;
    auto sum = [&](int from, int to, vec (&s)[2]) {
        s[0] = *(const vec *)(p + from * g.part_stride);
        s[1] = *(const vec *)(p + from * g.part_stride + 4);
        for (int z = from + 1; z < to; ++z) {
            s[0] += *(const vec *)(p + z * g.part_stride);
            s[1] += *(const vec *)(p + z * g.part_stride + 4);
        }
    };
    vec s[2];
    sum(0, j.first, s);
    float v[1][8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[0][k] = (float)s[k / 4][k % 4];
    if (!INT && j.copies > j.first) {
        sum(j.first, j.copies, s);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[0][k] = __builtin_fmaf((float)s[k / 4][k % 4], j.scale, v[0][k]);
    }
    float bs[8], ws[8];
    column_params(g.epi, n, g.N - n, bs, ws);
    finish<INT, 1>(g.epi, m, 1, g.M, n, g.N - n, v, bs, ws);
}

}  // namespace dense
