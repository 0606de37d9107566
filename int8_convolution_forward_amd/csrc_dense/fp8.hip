// C entries of the dense layer on 8-bit floating point, its gradients, and the
// quantiser: argument checks, the choice of kernel and the launches.
#include "fp8_kernel.hpp"
#include "gemm_plan.hpp"
#include "skinny_f8_kernel.hpp"

namespace dense {
namespace {

// ---- quantising --------------------------------------------------------------

conv_i8_status_t check_fp8(dense_mat_t *m, bool output)
{
    return is_fp8(m->dtype) ? check_mat_of(m, output, 1) : CONV_I8_ERR_DTYPE;
}

struct QuantPlan {
    dense_quantize_t d;
    bool tiles = false, tiles_t = false;
};

conv_i8_status_t analyze(const dense_quantize_t *args, QuantPlan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_quantize_t &d = p->d;
    DENSE_TRY(check_mat(&d.x, false));
    if (!is_float(d.x.dtype))
        return CONV_I8_ERR_DTYPE;
    const int64_t M = d.x.rows, K = d.x.cols;
    const bool q = d.q.dtype != DENSE_NONE, qt = d.qt.dtype != DENSE_NONE;
    if (!q && !qt)
        return CONV_I8_ERR_NULL;
    if ((d.scale.dtype != DENSE_NONE) != q || (d.scale_t.dtype != DENSE_NONE) != qt)
        return CONV_I8_ERR_PARAM;
    if (q) {
        DENSE_TRY(check_fp8(&d.q, true));
        if (d.q.rows != M || d.q.cols != K)
            return CONV_I8_ERR_OUT_DIMS;
        DENSE_TRY(check_scales(&d.scale, M, K, true, &p->tiles));
    }
    if (qt) {
        DENSE_TRY(check_fp8(&d.qt, true));
        if (d.qt.rows != K || d.qt.cols != M)
            return CONV_I8_ERR_OUT_DIMS;
        DENSE_TRY(check_scales(&d.scale_t, K, M, true, &p->tiles_t));
    }
    if (q && qt && d.q.dtype != d.qt.dtype)
        return CONV_I8_ERR_DTYPE;
    if (d.x.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    const bool rows = !qt && !p->tiles;
    if (!launch_fits(rows ? ceil_div(M, 16) * ceil_div(K, 512) : ceil_div(M, kBlock) * ceil_div(K, kBlock), kTileThreads))
        return CONV_I8_ERR_UNSUPPORTED;
    return CONV_I8_OK;
}

void run_quantize(const QuantPlan &p, hipStream_t s)
{
    const dense_quantize_t &d = p.d;
    QuantArgs a;
    memset(&a, 0, sizeof a);
    a.x = d.x.ptr;
    a.ldx = d.x.row_stride;
    a.M = (int)d.x.rows;
    a.K = (int)d.x.cols;
    a.e5 = (d.q.dtype != DENSE_NONE ? d.q.dtype : d.qt.dtype) == DENSE_E5M2;
    a.tiles = p.tiles;
    a.tiles_t = p.tiles_t;
    if (d.q.dtype != DENSE_NONE) {
        a.q = (uint8_t *)const_cast<void *>(d.q.ptr);
        a.ldq = d.q.row_stride;
        a.scale = (uint8_t *)const_cast<void *>(d.scale.ptr);
        a.lds = d.scale.row_stride;
        a.q_cols = a.K;
    }
    if (d.qt.dtype != DENSE_NONE) {
        a.qt = (uint8_t *)const_cast<void *>(d.qt.ptr);
        a.ldqt = d.qt.row_stride;
        a.scale_t = (uint8_t *)const_cast<void *>(d.scale_t.ptr);
        a.ldst = d.scale_t.row_stride;
        a.qt_cols = a.M;
    }
    const bool rows = !a.qt && !a.tiles;
    a.strips = (int)ceil_div(a.K, rows ? 512 : kBlock);
    a.blocks = (int)(a.strips * ceil_div(a.M, rows ? 16 : kBlock));
    PackArgs none;
    memset(&none, 0, sizeof none);
    const dim3 grid((unsigned)a.blocks), block(256);
    auto launch = [&](auto t) {
        typedef typename decltype(t)::type T;
        if (rows)
            hipLaunchKernelGGL(quantize_rows_kernel<T>, grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((quantize_tile_kernel<T, DENSE_ACT_NONE>), grid, dim3(kTileThreads), 0, s, a, none);
    };
    if (d.x.dtype == DENSE_BF16)
        launch(Type<bf16>{});
    else if (d.x.dtype == DENSE_FP16)
        launch(Type<f16>{});
    else
        launch(Type<float>{});
}

conv_i8_status_t analyze(const dense_dequantize_t *args, dense_dequantize_t *d, bool *tiles)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    *d = *args;
    DENSE_TRY(check_fp8(&d->q, false));
    DENSE_TRY(check_mat(&d->x, true));
    if (!is_float(d->x.dtype))
        return CONV_I8_ERR_DTYPE;
    if (d->x.rows != d->q.rows || d->x.cols != d->q.cols)
        return CONV_I8_ERR_OUT_DIMS;
    if (d->q.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    DENSE_TRY(check_scales(&d->scale, d->q.rows, d->q.cols, false, tiles));
    return launch_fits(ceil_div(d->q.rows, 16) * ceil_div(d->q.cols, 512), 256) ? CONV_I8_OK : CONV_I8_ERR_UNSUPPORTED;
}

// x [rows of q, cols]: q's values and zeros after them
void run_dequantize(const dense_mat_t &q, const dense_mat_t &scale, bool tiles, int64_t dt, void *x, int64_t ldx, int cols,
                    hipStream_t s)
{
    if (q.rows == 0 || cols == 0)
        return;
    DequantArgs a;
    memset(&a, 0, sizeof a);
    a.q = (const uint8_t *)q.ptr;
    a.scale = (const uint8_t *)scale.ptr;
    a.x = x;
    a.ldq = q.row_stride;
    a.lds = scale.row_stride;
    a.ldx = ldx;
    a.M = (int)q.rows;
    a.K = (int)q.cols;
    a.x_cols = cols;
    a.strips = (int)ceil_div(cols, 512);
    a.shift = tiles ? 7 : 0;
    a.e5 = q.dtype == DENSE_E5M2;
    const dim3 grid((unsigned)(a.strips * ceil_div(a.M, 16))), block(256);
    if (dt == DENSE_BF16)
        hipLaunchKernelGGL(dequantize_kernel<bf16>, grid, block, 0, s, a);
    else if (dt == DENSE_FP16)
        hipLaunchKernelGGL(dequantize_kernel<f16>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(dequantize_kernel<float>, grid, block, 0, s, a);
}

// ---- linear_fp8 --------------------------------------------------------------

struct LinearF8Plan {
    dense_linear_fp8_t d;
    int64_t M, N, K;
    bool w_tiles = false;
    bool skinny = false;
    bool wide = false;  // the operands as BF16: for a 32-bit result
    int waves = 4;
    Operand a, b;
    GemmPlan gemm;
    int64_t ws_bytes = 0;
};

// An operand [dim, inner] taken to BF16 in the workspace
conv_i8_status_t plan_wide(const dense_mat_t &m, Operand *o)
{
    if (m.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    o->dim = m.rows;
    o->inner = m.cols;
    o->es = 2;
    o->packed = true;
    o->ld = round_up(m.cols * 2, 16);
    o->pack_bytes = round_up(o->ld * m.rows, kWsAlign);
    if (!launch_fits(ceil_div(m.rows, 16) * ceil_div(m.cols, 512), 256))
        return CONV_I8_ERR_UNSUPPORTED;
    return check_reach(*o);
}

// An operand [dim, inner] of bytes, read in rows form
conv_i8_status_t plan_bytes(const dense_mat_t &m, Operand *o)
{
    o->src = m.ptr;
    o->rs = m.row_stride;
    o->cs = m.col_stride;
    o->dim = m.rows;
    o->inner = m.cols;
    o->es = 1;
    plan_operand(o, true, false);
    return check_reach(*o);
}

conv_i8_status_t analyze(const dense_linear_fp8_t *args, LinearF8Plan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_linear_fp8_t &d = p->d;
    DENSE_TRY(check_fp8(&d.x, false));
    DENSE_TRY(check_fp8(&d.w, false));
    DENSE_TRY(check_mat(&d.y, true));
    if (d.w.dtype != DENSE_E4M3 || !is_float(d.y.dtype))
        return CONV_I8_ERR_DTYPE;
    p->M = d.x.rows;
    p->K = d.x.cols;
    p->N = d.w.rows;
    if (d.w.cols != p->K)
        return CONV_I8_ERR_CHANNELS;
    if (d.y.rows != p->M || d.y.cols != p->N)
        return CONV_I8_ERR_OUT_DIMS;
    DENSE_TRY(check_scales(&d.x_scale, p->M, p->K, false, nullptr));
    DENSE_TRY(check_scales(&d.w_scale, p->N, p->K, false, &p->w_tiles));
    dense_mat_t *same[2] = {&d.residual, &d.preact};
    for (int i = 0; i < 2; ++i) {
        if (same[i]->dtype == DENSE_NONE) {
            same[i]->ptr = nullptr;
            continue;
        }
        DENSE_TRY(check_mat(same[i], i == 1));
        if (same[i]->dtype != d.y.dtype)
            return CONV_I8_ERR_DTYPE;
        if (same[i]->rows != p->M || same[i]->cols != p->N)
            return CONV_I8_ERR_OUT_DIMS;
        if (same[i]->col_stride != 1)
            return CONV_I8_ERR_STRIDES;
    }
    DENSE_TRY(check_vec(&d.bias, p->N));
    if (d.activation < DENSE_ACT_NONE || d.activation > DENSE_ACT_SILU)
        return CONV_I8_ERR_PARAM;
    if (p->M == 0 || p->N == 0)
        return CONV_I8_OK;
    Forced forced;
    DENSE_TRY(forced_tile(&forced));
    DENSE_TRY(plan_bytes(d.x, &p->a));
    DENSE_TRY(plan_bytes(d.w, &p->b));
    // Without a copy, up to 32 rows (us, all of BF16 results; the other side is the best tile and split):
    //   rows x w         1 x 4096x4096    16 x 4096x4096    17 x 4096x4096    17 x 8192x4096    17 x 16384x4096
    //   few rows' / tiles   5.9 / 9.8        6.4 / 10.6        8.4 / 10.5       16.5 / 14.1        30.1 / 18.8
    // Above 16 rows the copies of x leave LDS for one workgroup on a CU, which has half the weights of
    // that in flight: it pays while each CU has one workgroup in all.  A 32-bit result costs the tiles twice.
    const bool one_each = ceil_div(p->N, 16) <= kCUs;
    p->skinny = p->M <= (one_each || d.y.dtype == DENSE_FP32 ? 32 : 16) && p->N <= ((int64_t)1 << 25) && !p->a.packed &&
                !p->b.packed && !forced.on;
    if (p->skinny) {
        // A wave for each group of four blocks of K, as far as LDS has room: 1 x 4096x4096 6.5 us with 4
        // waves, 5.9 with 8, 6.1 with 16; 1 x 1024x8192 7.0, 5.4, 5.2; 1 x 8192x1024 4.4, 4.5, 5.9.  With x
        // in LDS as well, 8 waves fill it: where CUs have several workgroups, two of 4 waves do more (16 x
        // 16384x4096: 22.4 us with 8, 18.9 with 4; 16 x 4096x4096: 6.5 and 7.3).
        const int64_t groups = ceil_div(p->K, 4 * kBlock);
        if (groups <= 4 || p->M > 16 || (p->M > 4 && !one_each))
            p->waves = 4;
        else
            p->waves = groups <= 8 || p->M > 4 ? 8 : 16;
        return CONV_I8_OK;
    }
    p->wide = d.y.dtype == DENSE_FP32;
    if (p->wide) {
        p->a = p->b = Operand();
        DENSE_TRY(plan_wide(d.x, &p->a));
        DENSE_TRY(plan_wide(d.w, &p->b));
    }
    plan_gemm(p->M, p->N, p->K, p->wide ? 2 : 1, forced, &p->gemm, p->wide ? kCost : kCostF8);
    if (!grid_fits(p->gemm, p->M) || !launch_fits(pack_wgs(p->a) + pack_wgs(p->b), 256))
        return CONV_I8_ERR_UNSUPPORTED;
    p->ws_bytes = p->a.pack_bytes + p->b.pack_bytes + p->gemm.part_bytes;
    return CONV_I8_OK;
}

template <typename T, int G, int R, bool XL>
void launch_skinny(const SkinnyF8Args &a, int waves, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(a.s.N, 16 * R));
    if constexpr (!XL) {
        if (waves == 16) {
            hipLaunchKernelGGL((skinny_f8_kernel<T, G, R, 16, XL>), grid, dim3(1024), 0, s, a);
            return;
        }
    }
    if constexpr (G == 1) {
        if (waves >= 8) {
            hipLaunchKernelGGL((skinny_f8_kernel<T, G, R, 8, XL>), grid, dim3(512), 0, s, a);
            return;
        }
    }
    hipLaunchKernelGGL((skinny_f8_kernel<T, G, R, 4, XL>), grid, dim3(256), 0, s, a);
}

template <typename T>
void launch_skinny(const SkinnyF8Args &a, int waves, hipStream_t s)
{
    if (a.s.M <= 4)
        launch_skinny<T, 1, 1, false>(a, waves, s);
    else if (a.s.M <= 16)
        launch_skinny<T, 1, 1, true>(a, waves, s);
    else
        launch_skinny<T, 2, 1, true>(a, waves, s);
}

void set_scales(GemmArgs *g, const void *sa, int64_t ldsa, const void *sb, int64_t ldsb, bool b_tiles, int64_t K)
{
    g->sa = (const uint8_t *)sa;
    g->sb = (const uint8_t *)sb;
    g->ldsa = ldsa;
    g->ldsb = ldsb;
    g->sb_shift = b_tiles ? 7 : 0;
    g->kblocks = (int)ceil_div(K, kBlock);
}

conv_i8_status_t run_linear(const LinearF8Plan &p, void *ws, hipStream_t stream)
{
    const dense_linear_fp8_t &d = p.d;
    Epilogue epi;
    memset(&epi, 0, sizeof epi);
    epi.out = const_cast<void *>(d.y.ptr);
    epi.ldo = d.y.row_stride;
    epi.residual = d.residual.ptr;
    epi.ldr = d.residual.row_stride;
    epi.preact = const_cast<void *>(d.preact.ptr);
    epi.ldp = d.preact.row_stride;
    epi.bias = d.bias.ptr;
    epi.bias_dt = (int)d.bias.dtype;
    epi.out_dt = (int)d.y.dtype;
    epi.act = (int)d.activation;
    if (p.skinny) {
        SkinnyF8Args a;
        memset(&a, 0, sizeof a);
        a.s.x = (const uint8_t *)d.x.ptr;
        a.s.w = (const uint8_t *)d.w.ptr;
        a.s.ldx = d.x.row_stride;
        a.s.ldw = d.w.row_stride;
        a.s.M = (int)p.M;
        a.s.N = (int)p.N;
        a.s.kbytes = p.K;
        a.s.epi = epi;
        a.sx = (const uint8_t *)d.x_scale.ptr;
        a.sw = (const uint8_t *)d.w_scale.ptr;
        a.ldsx = d.x_scale.row_stride;
        a.ldsw = d.w_scale.row_stride;
        a.sw_shift = p.w_tiles ? 7 : 0;
        a.kblocks = (int)ceil_div(p.K, kBlock);
        if (d.x.dtype == DENSE_E4M3)
            launch_skinny<f8e4>(a, p.waves, stream);
        else
            launch_skinny<f8e5>(a, p.waves, stream);
        return hipGetLastError() == hipSuccess ? CONV_I8_OK : CONV_I8_ERR_HIP;
    }
    uint8_t *pa = (uint8_t *)ws, *pb = pa + p.a.pack_bytes, *part = pb + p.b.pack_bytes;
    if (p.wide) {
        run_dequantize(d.x, d.x_scale, false, DENSE_BF16, pa, p.a.ld / 2, (int)(p.a.ld / 2), stream);
        run_dequantize(d.w, d.w_scale, p.w_tiles, DENSE_BF16, pb, p.b.ld / 2, (int)(p.b.ld / 2), stream);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
        const GemmArgs g = gemm_args(p.a, pa, p.b, pb, p.M, p.N, p.K, p.gemm, part, epi);
        return run_gemm(DENSE_BF16, p.a, p.b, p.gemm, g, stream) ? CONV_I8_OK : CONV_I8_ERR_HIP;
    }
    if (!launch_pack(p.a, pa, p.b, pb, stream))
        return CONV_I8_ERR_HIP;
    GemmArgs g = gemm_args(p.a, p.a.packed ? pa : p.a.src, p.b, p.b.packed ? pb : p.b.src, p.M, p.N, p.K, p.gemm, part, epi);
    set_scales(&g, d.x_scale.ptr, d.x_scale.row_stride, d.w_scale.ptr, d.w_scale.row_stride, p.w_tiles, p.K);
    return run_gemm(d.x.dtype, p.a, p.b, p.gemm, g, stream) ? CONV_I8_OK : CONV_I8_ERR_HIP;
}

// ---- linear_fp8_backward -----------------------------------------------------

struct BackwardF8Plan {
    dense_linear_fp8_backward_t d;
    int64_t M, N, K;
    bool want_dx, want_dw, want_db;
    bool pass;                          // the pass over dy (and preact)
    bool xt_tiles = false, wt_tiles = false;
    Operand ga, gt, wb, xb;             // g and g^T as quantised here, wt and xt
    int64_t g_bytes = 0, gs_bytes = 0, gt_bytes = 0, gts_bytes = 0, sum_bytes = 0, sum_ld = 0;
    GemmPlan dx, dw;
    int64_t part_bytes = 0, ws_bytes = 0;

    // Both products go out in one launch.
    bool pair() const
    {
        return want_dx && want_dw && dx.tile == kPairTile && dw.tile == kPairTile && dx.splits == 1 && dw.splits == 1 &&
               launch_fits((int64_t)dx.tiles_m * dx.tiles_n + (int64_t)dw.tiles_m * dw.tiles_n + ceil_div(N, 8), 256);
    }
};

conv_i8_status_t analyze(const dense_linear_fp8_backward_t *args, BackwardF8Plan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_linear_fp8_backward_t &d = p->d;
    DENSE_TRY(check_mat(&d.dy, false));
    const int64_t dt = d.dy.dtype;
    if (!is_half(dt) || !is_fp8(d.g_dtype))
        return CONV_I8_ERR_DTYPE;
    const int64_t M = p->M = d.dy.rows, N = p->N = d.dy.cols;
    if (d.activation < DENSE_ACT_NONE || d.activation > DENSE_ACT_SILU)
        return CONV_I8_ERR_PARAM;
    if (d.dy.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    if (d.activation != DENSE_ACT_NONE) {
        if (d.preact.dtype == DENSE_NONE)
            return CONV_I8_ERR_NULL;
        DENSE_TRY(check_mat(&d.preact, false));
        if (d.preact.dtype != dt)
            return CONV_I8_ERR_DTYPE;
        if (d.preact.rows != M || d.preact.cols != N)
            return CONV_I8_ERR_DIMS;
        if (d.preact.col_stride != 1)
            return CONV_I8_ERR_STRIDES;
    }
    p->want_dx = d.dx.dtype != DENSE_NONE;
    p->want_dw = d.dw.dtype != DENSE_NONE;
    p->want_db = d.dbias.dtype != DENSE_NONE;
    p->K = p->want_dx ? d.dx.cols : p->want_dw ? d.dw.cols : 0;
    auto operand = [&](dense_mat_t *q, dense_mat_t *scale, int64_t inner, bool *tiles) {
        if (q->dtype != DENSE_E4M3)
            return q->dtype == DENSE_NONE ? CONV_I8_ERR_NULL : CONV_I8_ERR_DTYPE;
        DENSE_TRY(check_fp8(q, false));
        if (q->rows != p->K)
            return CONV_I8_ERR_CHANNELS;
        if (q->cols != inner)
            return CONV_I8_ERR_DIMS;
        return check_scales(scale, p->K, inner, false, tiles);
    };
    if (p->want_dx) {
        DENSE_TRY(check_mat(&d.dx, true));
        if (d.dx.dtype != dt)
            return CONV_I8_ERR_DTYPE;
        if (d.dx.rows != M)
            return CONV_I8_ERR_OUT_DIMS;
        DENSE_TRY(operand(&d.wt, &d.wt_scale, N, &p->wt_tiles));
    }
    if (p->want_dw) {
        DENSE_TRY(check_mat(&d.dw, true));
        if (d.dw.dtype != dt)
            return CONV_I8_ERR_DTYPE;
        if (d.dw.rows != N || d.dw.cols != p->K)
            return CONV_I8_ERR_OUT_DIMS;
        DENSE_TRY(operand(&d.xt, &d.xt_scale, M, &p->xt_tiles));
    }
    DENSE_TRY(check_vec(&d.dbias, N));
    if (p->want_db && d.dbias.dtype != dt)
        return CONV_I8_ERR_DTYPE;
    p->want_dx = p->want_dx && M > 0 && p->K > 0;
    p->want_dw = p->want_dw && N > 0 && p->K > 0;
    p->want_db = p->want_db && N > 0;
    p->pass = M > 0 && N > 0 && (p->want_dx || p->want_dw || p->want_db);

    // g as the products read it: rows of whole 16-byte chunks, zeros in the last one
    auto quantised = [&](int64_t dim, int64_t inner, Operand *o, int64_t *bytes, int64_t *scale_bytes) {
        o->es = 1;
        o->dim = dim;
        o->inner = inner;
        o->ld = round_up(inner, 16);
        *bytes = round_up(dim * o->ld, kWsAlign);
        *scale_bytes = round_up(dim * ceil_div(inner, kBlock), kWsAlign);
        return check_reach(*o);
    };
    Forced forced;
    DENSE_TRY(forced_tile(&forced));
    p->wb.es = p->xb.es = 1;  // both are copied by one launch, also where one is absent
    double apart = 0.0;
    if (p->want_dx) {
        DENSE_TRY(quantised(M, N, &p->ga, &p->g_bytes, &p->gs_bytes));
        DENSE_TRY(plan_bytes(d.wt, &p->wb));
        apart += plan_gemm(M, p->K, N, 1, forced, &p->dx, kCostF8);
        if (!grid_fits(p->dx, M))
            return CONV_I8_ERR_UNSUPPORTED;
        p->part_bytes = p->dx.part_bytes;
    }
    if (p->want_dw) {
        DENSE_TRY(quantised(N, M, &p->gt, &p->gt_bytes, &p->gts_bytes));
        DENSE_TRY(plan_bytes(d.xt, &p->xb));
        apart += plan_gemm(N, p->K, M, 1, forced, &p->dw, kCostF8);
        // apart: a launch more, and the bias gradient's
        if (p->want_dx && !forced.on && pair_cost(M, N, p->K, 1, kCostF8) < apart + 4.0) {
            set_plan(M, p->K, N, 1, kPairTile, 1, &p->dx);
            set_plan(N, p->K, M, 1, kPairTile, 1, &p->dw);
            p->part_bytes = 0;
        }
        if (!grid_fits(p->dw, N))
            return CONV_I8_ERR_UNSUPPORTED;
        if (p->dw.part_bytes > p->part_bytes)
            p->part_bytes = p->dw.part_bytes;  // the two products run one after the other
    }
    if (p->want_db) {
        p->sum_ld = round_up(N, 32);
        p->sum_bytes = round_up(ceil_div(M, kBlock) * p->sum_ld * 4, kWsAlign);
    }
    if (!launch_fits(ceil_div(M, kBlock) * ceil_div(N, kBlock) + pack_wgs(p->wb) + pack_wgs(p->xb), kTileThreads))
        return CONV_I8_ERR_UNSUPPORTED;
    p->ws_bytes = p->g_bytes + p->gs_bytes + p->gt_bytes + p->gts_bytes + p->sum_bytes + p->wb.pack_bytes + p->xb.pack_bytes +
                  p->part_bytes;
    return CONV_I8_OK;
}

template <typename T>
void launch_pass(int64_t act, dim3 grid, const QuantArgs &a, const PackArgs &pack, hipStream_t s)
{
    switch (act) {
    case DENSE_ACT_RELU: hipLaunchKernelGGL((quantize_tile_kernel<T, DENSE_ACT_RELU>), grid, dim3(kTileThreads), 0, s, a, pack); break;
    case DENSE_ACT_GELU: hipLaunchKernelGGL((quantize_tile_kernel<T, DENSE_ACT_GELU>), grid, dim3(kTileThreads), 0, s, a, pack); break;
    case DENSE_ACT_GELU_TANH: hipLaunchKernelGGL((quantize_tile_kernel<T, DENSE_ACT_GELU_TANH>), grid, dim3(kTileThreads), 0, s, a, pack); break;
    case DENSE_ACT_SILU: hipLaunchKernelGGL((quantize_tile_kernel<T, DENSE_ACT_SILU>), grid, dim3(kTileThreads), 0, s, a, pack); break;
    default: hipLaunchKernelGGL((quantize_tile_kernel<T, DENSE_ACT_NONE>), grid, dim3(kTileThreads), 0, s, a, pack); break;
    }
}

conv_i8_status_t run_backward(const BackwardF8Plan &p, void *ws, hipStream_t stream)
{
    const dense_linear_fp8_backward_t &d = p.d;
    uint8_t *gq = (uint8_t *)ws, *gs = gq + p.g_bytes, *gtq = gs + p.gs_bytes, *gts = gtq + p.gt_bytes;
    uint8_t *sums = gts + p.gts_bytes, *pw = sums + p.sum_bytes, *px = pw + p.wb.pack_bytes, *part = px + p.xb.pack_bytes;
    if (p.pass) {
        QuantArgs a;
        memset(&a, 0, sizeof a);
        a.x = d.dy.ptr;
        a.ldx = d.dy.row_stride;
        a.z = d.activation != DENSE_ACT_NONE ? d.preact.ptr : nullptr;
        a.ldz = d.preact.row_stride;
        a.M = (int)p.M;
        a.K = (int)p.N;
        a.strips = (int)ceil_div(p.N, kBlock);
        a.e5 = d.g_dtype == DENSE_E5M2;
        if (p.want_dx) {
            a.q = gq;
            a.scale = gs;
            a.ldq = p.ga.ld;
            a.q_cols = (int)p.ga.ld;
            a.lds = ceil_div(p.N, kBlock);
        }
        if (p.want_dw) {
            a.qt = gtq;
            a.scale_t = gts;
            a.ldqt = p.gt.ld;
            a.qt_cols = (int)p.gt.ld;
            a.ldst = ceil_div(p.M, kBlock);
        }
        a.colsum = p.want_db ? (float *)sums : nullptr;
        a.sum_ld = p.sum_ld;
        a.blocks = (int)(a.strips * ceil_div(p.M, kBlock));
        PackArgs pack;
        const dim3 grid((unsigned)(a.blocks + pack_jobs(p.wb, pw, p.xb, px, &pack, kTileThreads)));
        if (d.dy.dtype == DENSE_BF16)
            launch_pass<bf16>(d.activation, grid, a, pack, stream);
        else
            launch_pass<f16>(d.activation, grid, a, pack, stream);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    } else if (!launch_pack(p.wb, pw, p.xb, px, stream)) {
        return CONV_I8_ERR_HIP;
    }
    ColSumArgs c;
    memset(&c, 0, sizeof c);
    if (p.want_db) {
        c.part = (const float *)sums;
        c.ld = p.sum_ld;
        c.rows = (int)ceil_div(p.M, kBlock);  // none: zeros
        c.cols = c.split = c.valid = p.N;
        c.out0 = const_cast<void *>(d.dbias.ptr);
        c.dt = (int)d.dy.dtype;
    }
    Epilogue e;
    memset(&e, 0, sizeof e);
    e.out_dt = (int)d.dy.dtype;
    GemmArgs dx, dw;
    if (p.want_dx) {
        e.out = const_cast<void *>(d.dx.ptr);
        e.ldo = d.dx.row_stride;
        dx = gemm_args(p.ga, gq, p.wb, p.wb.packed ? pw : p.wb.src, p.M, p.K, p.N, p.dx, part, e);
        set_scales(&dx, gs, ceil_div(p.N, kBlock), d.wt_scale.ptr, d.wt_scale.row_stride, p.wt_tiles, p.N);
    }
    if (p.want_dw) {
        e.out = const_cast<void *>(d.dw.ptr);
        e.ldo = d.dw.row_stride;
        dw = gemm_args(p.gt, gtq, p.xb, p.xb.packed ? px : p.xb.src, p.N, p.K, p.M, p.dw, part, e);
        set_scales(&dw, gts, ceil_div(p.M, kBlock), d.xt_scale.ptr, d.xt_scale.row_stride, p.xt_tiles, p.M);
    }
    if (p.pair()) {
        const PairArgs both = {dx, dw, c};
        const bool ok = d.g_dtype == DENSE_E4M3 ? launch_gemm_pair_f8e4(both, stream) : launch_gemm_pair_f8e5(both, stream);
        return ok ? CONV_I8_OK : CONV_I8_ERR_HIP;
    }
    if (p.want_db) {
        hipLaunchKernelGGL(colsum_kernel<>, colsum_grid(p.N), dim3(32 * kSumGroups), 0, stream, c);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    if (p.want_dx && !run_gemm(d.g_dtype, p.ga, p.wb, p.dx, dx, stream))
        return CONV_I8_ERR_HIP;
    if (p.want_dw && !run_gemm(d.g_dtype, p.gt, p.xb, p.dw, dw, stream))
        return CONV_I8_ERR_HIP;
    return CONV_I8_OK;
}

conv_i8_status_t answer(const char *text, char *buf, size_t len)
{
    if (strlen(text) + 1 > len)
        return CONV_I8_ERR_PARAM;
    memcpy(buf, text, strlen(text) + 1);
    return CONV_I8_OK;
}

}  // namespace
}  // namespace dense

using namespace dense;

extern "C" {

conv_i8_status_t dense_quantize(const dense_quantize_t *args, void *stream)
{
    QuantPlan p;
    DENSE_TRY(analyze(args, &p));
    if (p.d.x.rows == 0 || p.d.x.cols == 0)
        return CONV_I8_OK;
    run_quantize(p, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? CONV_I8_OK : CONV_I8_ERR_HIP;
}

conv_i8_status_t dense_dequantize(const dense_dequantize_t *args, void *stream)
{
    dense_dequantize_t d;
    bool tiles = false;
    DENSE_TRY(analyze(args, &d, &tiles));
    if (d.q.rows == 0 || d.q.cols == 0)
        return CONV_I8_OK;
    run_dequantize(d.q, d.scale, tiles, d.x.dtype, const_cast<void *>(d.x.ptr), d.x.row_stride, (int)d.x.cols, (hipStream_t)stream);
    return hipGetLastError() == hipSuccess ? CONV_I8_OK : CONV_I8_ERR_HIP;
}

conv_i8_status_t dense_linear_fp8_workspace_size(const dense_linear_fp8_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    LinearF8Plan p;
    DENSE_TRY(analyze(args, &p));
    *bytes = (size_t)p.ws_bytes;
    return CONV_I8_OK;
}

conv_i8_status_t dense_linear_fp8(const dense_linear_fp8_t *args, void *workspace, size_t bytes, void *stream)
{
    LinearF8Plan p;
    DENSE_TRY(analyze(args, &p));
    if (p.M == 0 || p.N == 0)
        return CONV_I8_OK;
    DENSE_TRY(check_workspace(workspace, bytes, p.ws_bytes));
    return run_linear(p, workspace, (hipStream_t)stream);
}

conv_i8_status_t dense_linear_fp8_plan(const dense_linear_fp8_t *args, char *buf, size_t len)
{
    if (!buf)
        return CONV_I8_ERR_NULL;
    LinearF8Plan p;
    DENSE_TRY(analyze(args, &p));
    char text[256];
    if (p.M == 0 || p.N == 0) {
        snprintf(text, sizeof text, "kernel=none");
    } else if (p.skinny) {
        snprintf(text, sizeof text, "kernel=skinny waves=%d", p.waves);
    } else {
        char t[200];
        describe(p.gemm, p.a, p.b, t, sizeof t);
        snprintf(text, sizeof text, "kernel=%s %s", p.wide ? "gemm_bf16" : "gemm", t);
    }
    return answer(text, buf, len);
}

conv_i8_status_t dense_linear_fp8_backward_workspace_size(const dense_linear_fp8_backward_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    BackwardF8Plan p;
    DENSE_TRY(analyze(args, &p));
    *bytes = (size_t)p.ws_bytes;
    return CONV_I8_OK;
}

conv_i8_status_t dense_linear_fp8_backward(const dense_linear_fp8_backward_t *args, void *workspace, size_t bytes,
                                           void *stream)
{
    BackwardF8Plan p;
    DENSE_TRY(analyze(args, &p));
    DENSE_TRY(check_workspace(workspace, bytes, p.ws_bytes));
    return run_backward(p, workspace, (hipStream_t)stream);
}

conv_i8_status_t dense_linear_fp8_backward_plan(const dense_linear_fp8_backward_t *args, char *buf, size_t len)
{
    if (!buf)
        return CONV_I8_ERR_NULL;
    BackwardF8Plan p;
    DENSE_TRY(analyze(args, &p));
    char text[512], dx[200] = "none", dw[200] = "none";
    if (p.want_dx)
        describe(p.dx, p.ga, p.wb, dx, sizeof dx);
    if (p.want_dw)
        describe(p.dw, p.gt, p.xb, dw, sizeof dw);
    snprintf(text, sizeof text, "launches=%s dx: %s; dw: %s", p.pair() ? "paired" : "apart", dx, dw);
    return answer(text, buf, len);
}

}  // extern "C"
