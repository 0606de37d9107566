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

// acc += the 16x16 product, in place in accumulation registers.  Written as an
// instruction because the register allocator otherwise gives the result other
// registers than the addend and copies all of them around the loop.  The
// compiler then knows nothing of its latency: operands come from LDS reads
// (which it does wait for), one accumulator's instructions are FM*FN apart, and
// the kernel waits itself before it reads the sums (mfma_drain).
template <typename T>
__device__ __forceinline__ void mfma16_acc(v4i a, v4i b, typename Acc4<T>::type &c)
{
    if constexpr (sizeof(T) == 1)
        asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else if constexpr (__is_same(T, bf16))
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else
        asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// More wait states than a result of the instruction above needs.
__device__ __forceinline__ void mfma_drain()
{
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
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

// SB: bytes of the inner dimension per stage, 64 or 128; NSA, NSB: slots of the
// operands' rings, NSB or NSB + 1 and NSB; LH: loads per thread of a stage that
// go out in the half that frees their slots (the others in the half after it);
// OCC: workgroups a CU is to hold at a time (one wave of each per SIMD)
template <typename T, int TM, int TN, int WGM, int WGN, int SB, int NSA, int NSB, int LH, int OCC, bool ASTR, bool BSTR>
__global__ __launch_bounds__(64 * WGM * WGN, OCC) void gemm_kernel(const GemmArgs g)
{
    constexpr int NW = WGM * WGN;
    constexpr int ES = sizeof(T);
    constexpr int H = SB / 64;                  // halves of a stage, one matrix instruction deep each
    constexpr int BKE = SB / ES;                // inner elements per stage
    constexpr int RPB = 1024 / SB;              // rows-form rows per 1 KiB block
    constexpr int AL = TM / (NW * RPB), BL = TN / (NW * RPB), LPS = AL + BL;
    constexpr int A_BYTES = TM * SB, B_BYTES = TN * SB;
    constexpr int WM = TM / WGM, WN = TN / WGN;
    constexpr int FM = WM / 16, FN = WN / 16;
    constexpr int NMF = FM * FN;                // matrix instructions per half
    constexpr int NRD = FM + FN;                // fragment reads per half
    static_assert(AL >= 1 && BL >= 1 && FM >= 2 && FN >= 2, "tile too small");
    static_assert(NSB >= 2 && (NSA == NSB || (NSA == 3 && NSB == 2)), "ring slots");
    static_assert((NSA - 1) * AL + (NSB - 1) * BL < 64, "pipeline depth");
    static_assert(LH <= LPS && (H > 1 || LH == LPS), "loads of a stage");
    constexpr int RING = NSA * A_BYTES + NSB * B_BYTES, A_RING = NSA * A_BYTES;
    static_assert(!(ASTR || BSTR) || ES == 2, "transposing reads take 16-bit values");

    // epilogue slab of one wave: 32 rows of WN values, padded by 4
    constexpr int SP = WN + 4;
    constexpr int SLAB = 32 * SP * 4;
    constexpr int LDS_BYTES = RING > NW * SLAB ? RING : NW * SLAB;
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
    const int row0 = wave * RPB + lane / (SB / 16);
    const int j = row_swizzle<SB>(row0, lane % (SB / 16));  // the same for every i
    auto rows_off = [&](int i, int first, int dim, int64_t ld) {
        const int r = row0 + i * NW * RPB;
        return first + r < dim ? r * (int)ld + j * 16 : kOutOfRange;
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
        a_off[i] = ASTR ? cols_off(TMc{}, i, m0, g.M, g.lda) : rows_off(i, m0, g.M, g.lda);
#pragma unroll
    for (int i = 0; i < BL; ++i)
        b_off[i] = BSTR ? cols_off(TNc{}, i, n0, g.N, g.ldb) : rows_off(i, n0, g.N, g.ldb);

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
                const bool in = b_next * SB + j * 16 < g.kbytes;
#pragma unroll
                for (int i = 0; i < BL; ++i)
                    b_off[i] = in ? b_off[i] : kOutOfRange;
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
                frag[buf][i] = read_rows(base, wn + i * 16, half);
        } else {
            const uint8_t *base = smem + a_slot * A_BYTES;
            if constexpr (ASTR)
                frag[buf][i] = read_cols(TMc{}, base, wm + (i - FN) * 16, half);
            else
                frag[buf][i] = read_rows(base, wm + (i - FN) * 16, half);
        }
    };
    auto mfma_one = [&](int buf, int i) {
        const int x = i / FN, y = i % FN;
        mfma16_acc<T>(frag[buf][y], frag[buf][FN + x], acc[x][y]);
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
    auto half = [&](auto bufc, auto hc) __attribute__((always_inline)) {
        constexpr int buf = decltype(bufc)::value, h = decltype(hc)::value;
        constexpr bool last = h == H - 1;
        constexpr int first = last ? PRE : 0;   // matrix instructions before reads may start
        constexpr int np = NMF - first, nr = np * 3 / 4 > 0 ? np * 3 / 4 : 1;
        constexpr int l0 = last ? 0 : LH, nl = last ? LH : h == 0 ? LPS - LH : 0;
        const int an = a_slot + 1 == NSA ? 0 : a_slot + 1, bn = b_slot + 1 == NSB ? 0 : b_slot + 1;
        for_each<NMF>([&](auto ic) __attribute__((always_inline)) {
            constexpr int i = decltype(ic)::value;
            if constexpr (last && i == PRE) {
                wait_vm_lgkm0<(NSA - 2) * AL + (NSB - 2) * BL>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
            mfma_one(buf, i);
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

    // Fragment buffers alternate by half.  With one half per stage the loop
    // body holds two stages, and an odd count runs an extra stage of zeros.
    const int nloop = H == 1 ? (max(stage_end - stage0, 0) + 1) & ~1 : max(stage_end - stage0, 0);
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
        for (int it = 0; it < nloop; it += H == 1 ? 2 : 1) {
            half(Size<0>{}, Size<0>{});
            half(Size<1>{}, Size<H - 1>{});
        }
        wait_vm_lgkm0<0>();  // the trailing loads of zeros still write to the rings
        mfma_drain();
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
        for (int x2 = 0; x2 < 2; ++x2)
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                const typename Acc4<T>::type v = acc[2 * x + x2][y];
                v4f o;
                if constexpr (ES == 1)  // partial sums stay integers (their bits travel as floats)
                    o = g.part ? __builtin_bit_cast(v4f, v) : v4f{(float)v.x, (float)v.y, (float)v.z, (float)v.w};
                else
                    o = v;
                *(v4f *)&slab[(x2 * 16 + (lane & 15)) * SP + y * 16 + 4 * (lane >> 4)] = o;
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
    static_assert(FM == 2 || FM == 4 || FM == 8, "slabs");
    finish_slab(Size<0>{});
    if constexpr (FM >= 4)
        finish_slab(Size<1>{});
    if constexpr (FM >= 8) {
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
