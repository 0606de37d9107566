// The dense layer's C entries: argument checks, the choice of kernel and the
// launches.
#include "gemm_plan.hpp"
#include "skinny_kernel.hpp"

namespace dense {
namespace {

// ---- linear ----------------------------------------------------------------

// Largest M the kernel for a few rows takes, and largest N: its workgroups have
// up to 1024 threads for 16 columns each, and a launch fewer than 2^32.
constexpr int64_t kSkinnyRows = 32, kSkinnyCols = (int64_t)1 << 25;

struct LinearPlan {
    dense_linear_t d;
    int64_t M, N, K;
    bool skinny = false;
    int waves = 4;
    bool aligned = false;
    Operand a, b;
    GemmPlan gemm;
    int64_t ws_bytes = 0;
};

conv_i8_status_t analyze(const dense_linear_t *args, LinearPlan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_linear_t &d = p->d;
    DENSE_TRY(check_mat(&d.x, false));
    DENSE_TRY(check_mat(&d.w, false));
    DENSE_TRY(check_mat(&d.y, true));
    const int64_t dt = d.x.dtype;
    if (dt == DENSE_FP32 || d.w.dtype != dt)
        return CONV_I8_ERR_DTYPE;
    if (!is_float(d.y.dtype) || (dt != DENSE_INT8 && d.y.dtype != DENSE_FP32 && d.y.dtype != dt))
        return CONV_I8_ERR_DTYPE;
    p->M = d.x.rows;
    p->K = d.x.cols;
    p->N = d.w.rows;
    if (d.w.cols != p->K)
        return CONV_I8_ERR_CHANNELS;
    if (d.y.rows != p->M || d.y.cols != p->N)
        return CONV_I8_ERR_OUT_DIMS;
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
    DENSE_TRY(check_vec(&d.x_scale, p->M));
    DENSE_TRY(check_vec(&d.w_scale, p->N));
    for (const dense_vec_t *s : {&d.x_scale, &d.w_scale})
        if (s->dtype != DENSE_NONE && (s->dtype != DENSE_FP32 || dt != DENSE_INT8))
            return CONV_I8_ERR_DTYPE;
    if (d.activation < DENSE_ACT_NONE || d.activation > DENSE_ACT_SILU)
        return CONV_I8_ERR_PARAM;
    if (dt == DENSE_INT8 && p->K > CONV_I8_MAX_REDUCTION)
        return CONV_I8_ERR_RANGE;

    if (p->M == 0 || p->N == 0)
        return CONV_I8_OK;
    Forced forced;
    DENSE_TRY(forced_tile(&forced));
    const int es = (int)size_of(dt);
    const bool x_rows = d.x.col_stride == 1 || p->K <= 1, w_rows = d.w.col_stride == 1 || p->K <= 1;
    p->skinny = p->M <= kSkinnyRows && p->N <= kSkinnyCols && x_rows && w_rows && !forced.on;
    if (p->skinny) {
        p->aligned = (((uintptr_t)d.x.ptr | (uintptr_t)d.w.ptr) & 15) == 0 && p->K * es % 16 == 0 &&
                     (p->M <= 1 || d.x.row_stride * es % 16 == 0) && (p->N <= 1 || d.w.row_stride * es % 16 == 0);
        // load offsets are 31-bit: 32 rows from a workgroup's first
        if (p->M > 1 && d.x.row_stride * es > kMaxRowBytes)
            p->aligned = false;
        if (p->N > 1 && d.w.row_stride * es > kMaxRowBytes)
            p->aligned = false;
        // blocks of 128 bytes of the inner dimension for every wave, or fewer waves
        p->waves = !p->aligned ? 8 : p->K * es < 16 * 128 ? 4 : p->M <= 16 ? 16 : 8;
        return CONV_I8_OK;
    }
    p->a.src = d.x.ptr;
    p->a.rs = d.x.row_stride;
    p->a.cs = d.x.col_stride;
    p->a.dim = p->M;
    p->b.src = d.w.ptr;
    p->b.rs = d.w.row_stride;
    p->b.cs = d.w.col_stride;
    p->b.dim = p->N;
    p->a.inner = p->b.inner = p->K;
    p->a.es = p->b.es = es;
    plan_operand(&p->a, true, false);
    plan_operand(&p->b, true, es == 2);
    DENSE_TRY(check_reach(p->a));
    DENSE_TRY(check_reach(p->b));
    plan_gemm(p->M, p->N, p->K, es, forced, &p->gemm);
    if (!grid_fits(p->gemm, p->M))
        return CONV_I8_ERR_UNSUPPORTED;
    if (!launch_fits(pack_wgs(p->a) + pack_wgs(p->b), 256))
        return CONV_I8_ERR_UNSUPPORTED;
    p->ws_bytes = p->a.pack_bytes + p->b.pack_bytes + p->gemm.part_bytes;
    return CONV_I8_OK;
}

Epilogue epilogue_of(const dense_linear_t &d)
{
    Epilogue e;
    memset(&e, 0, sizeof e);
    e.out = const_cast<void *>(d.y.ptr);
    e.ldo = d.y.row_stride;
    e.residual = d.residual.ptr;
    e.ldr = d.residual.row_stride;
    e.preact = const_cast<void *>(d.preact.ptr);
    e.ldp = d.preact.row_stride;
    e.bias = d.bias.ptr;
    e.bias_dt = (int)d.bias.dtype;
    e.x_scale = (const float *)d.x_scale.ptr;
    e.w_scale = (const float *)d.w_scale.ptr;
    e.out_dt = (int)d.y.dtype;
    e.act = (int)d.activation;
    return e;
}

template <typename T>
bool launch_skinny(const SkinnyArgs &s, const LinearPlan &p, hipStream_t stream)
{
    const dim3 one((unsigned)ceil_div(s.N, 16)), two((unsigned)ceil_div(s.N, 32));
    if (!p.aligned) {
        if (p.M <= 16)
            hipLaunchKernelGGL((skinny_unaligned_kernel<T, 1, 8, 4>), one, dim3(512), 0, stream, s);
        else
            hipLaunchKernelGGL((skinny_unaligned_kernel<T, 2, 8, 2>), one, dim3(512), 0, stream, s);
    } else if (p.M <= 4) {
        if (p.waves == 4)
            hipLaunchKernelGGL((skinny_kernel<T, 1, 1, 4, 4, false>), one, dim3(256), 0, stream, s);
        else
            hipLaunchKernelGGL((skinny_kernel<T, 1, 1, 16, 2, false>), one, dim3(1024), 0, stream, s);
    } else if (p.M <= 16) {
        if (p.waves == 4)
            hipLaunchKernelGGL((skinny_kernel<T, 1, 1, 4, 4, true>), one, dim3(256), 0, stream, s);
        else
            hipLaunchKernelGGL((skinny_kernel<T, 1, 1, 16, 2, true>), one, dim3(1024), 0, stream, s);
    } else {
        if (p.waves == 4)
            hipLaunchKernelGGL((skinny_kernel<T, 2, 2, 4, 2, true>), two, dim3(256), 0, stream, s);
        else
            hipLaunchKernelGGL((skinny_kernel<T, 2, 2, 8, 2, true>), two, dim3(512), 0, stream, s);
    }
    return hipGetLastError() == hipSuccess;
}

conv_i8_status_t run_linear(const LinearPlan &p, void *ws, hipStream_t stream)
{
    const Epilogue epi = epilogue_of(p.d);
    if (p.skinny) {
        SkinnyArgs s;
        memset(&s, 0, sizeof s);
        const int64_t es = size_of(p.d.x.dtype);
        s.x = (const uint8_t *)p.d.x.ptr;
        s.w = (const uint8_t *)p.d.w.ptr;
        s.ldx = p.d.x.row_stride * es;
        s.ldw = p.d.w.row_stride * es;
        s.M = (int)p.M;
        s.N = (int)p.N;
        s.kbytes = p.K * es;
        s.epi = epi;
        const bool ok = p.d.x.dtype == DENSE_BF16 ? launch_skinny<bf16>(s, p, stream)
                      : p.d.x.dtype == DENSE_FP16 ? launch_skinny<f16>(s, p, stream)
                                                  : launch_skinny<int8_t>(s, p, stream);
        return ok ? CONV_I8_OK : CONV_I8_ERR_HIP;
    }
    uint8_t *pa = (uint8_t *)ws, *pb = pa + p.a.pack_bytes, *part = pb + p.b.pack_bytes;
    if (!launch_pack(p.a, pa, p.b, pb, stream))
        return CONV_I8_ERR_HIP;
    const GemmArgs g = gemm_args(p.a, p.a.packed ? pa : p.a.src, p.b, p.b.packed ? pb : p.b.src, p.M, p.N, p.K, p.gemm,
                                 part, epi);
    return run_gemm(p.d.x.dtype, p.a, p.b, p.gemm, g, stream) ? CONV_I8_OK : CONV_I8_ERR_HIP;
}

// ---- linear_backward -------------------------------------------------------

struct BackwardPlan {
    dense_linear_backward_t d;
    int64_t M, N, K;
    bool want_dx, want_dw, want_db;
    bool pass;                 // the pass over dy (and z) that writes g and the column sums
    bool write_g;
    bool wide = false;         // g as two terms: every product twice, joined like a split
    int64_t ldg = 0;           // elements
    int64_t g_bytes = 0;
    int row_blocks = 0, rows = 0;
    int64_t sum_ld = 0, sum_bytes = 0;
    Operand ga, wb;            // dx = g w: g in rows form, w in columns form over n
    Operand gt, xb;            // dw = g^T x: both in columns form over m
    GemmPlan dx, dw;
    int64_t part_bytes = 0, ws_bytes = 0;

    // Both products go out in one launch.
    bool pair() const
    {
        return !wide && want_dx && want_dw && dx.tile == kPairTile && dw.tile == kPairTile && dx.splits == 1 && dw.splits == 1 &&
               launch_fits((int64_t)dx.tiles_m * dx.tiles_n + (int64_t)dw.tiles_m * dw.tiles_n + ceil_div(N, 8), 256);
    }
};

conv_i8_status_t analyze(const dense_linear_backward_t *args, BackwardPlan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_linear_backward_t &d = p->d;
    const bool wide = d.activation & DENSE_WIDE_G;
    d.activation &= ~(int64_t)DENSE_WIDE_G;
    DENSE_TRY(check_mat(&d.dy, false));
    DENSE_TRY(check_mat(&d.x, false));
    DENSE_TRY(check_mat(&d.w, false));
    const int64_t dt = d.dy.dtype;
    if (!is_half(dt) || d.x.dtype != dt || d.w.dtype != dt)
        return CONV_I8_ERR_DTYPE;
    p->M = d.dy.rows;
    p->N = d.dy.cols;
    p->K = d.x.cols;
    if (d.w.cols != p->K)
        return CONV_I8_ERR_CHANNELS;
    if (d.x.rows != p->M || d.w.rows != p->N)
        return CONV_I8_ERR_DIMS;
    if (d.activation < DENSE_ACT_NONE || d.activation > DENSE_ACT_SILU)
        return CONV_I8_ERR_PARAM;
    const bool act = d.activation != DENSE_ACT_NONE;
    if (act) {
        if (d.preact.dtype == DENSE_NONE)
            return CONV_I8_ERR_NULL;
        DENSE_TRY(check_mat(&d.preact, false));
        if (d.preact.dtype != dt)
            return CONV_I8_ERR_DTYPE;
        if (d.preact.rows != p->M || d.preact.cols != p->N)
            return CONV_I8_ERR_DIMS;
        if (d.preact.col_stride != 1)
            return CONV_I8_ERR_STRIDES;
    }
    if (d.dy.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    p->want_dx = d.dx.dtype != DENSE_NONE;
    p->want_dw = d.dw.dtype != DENSE_NONE;
    p->want_db = d.dbias.dtype != DENSE_NONE;
    if (p->want_dx) {
        DENSE_TRY(check_mat(&d.dx, true));
        if (d.dx.dtype != dt)
            return CONV_I8_ERR_DTYPE;
        if (d.dx.rows != p->M || d.dx.cols != p->K)
            return CONV_I8_ERR_OUT_DIMS;
    }
    if (p->want_dw) {
        DENSE_TRY(check_mat(&d.dw, true));
        if (d.dw.dtype != dt)
            return CONV_I8_ERR_DTYPE;
        if (d.dw.rows != p->N || d.dw.cols != p->K)
            return CONV_I8_ERR_OUT_DIMS;
    }
    DENSE_TRY(check_vec(&d.dbias, p->N));
    if (p->want_db && d.dbias.dtype != dt)
        return CONV_I8_ERR_DTYPE;
    p->want_dx = p->want_dx && p->M > 0 && p->K > 0;
    p->want_dw = p->want_dw && p->N > 0 && p->K > 0;
    p->want_db = p->want_db && p->N > 0;

    // g: dy itself where there is no slope to apply, its rows are aligned and within a
    // tile's reach and, for dw, which reads it in columns form, none repeats or overlaps another
    const bool dy_ok = ((uintptr_t)d.dy.ptr & 15) == 0 && p->N % 8 == 0 &&
                       (p->M <= 1 || (d.dy.row_stride % 8 == 0 && (!p->want_dw || d.dy.row_stride >= p->N) &&
                                      d.dy.row_stride * 2 <= kMaxRowBytes));
    const bool any = p->M > 0 && p->N > 0;
    p->write_g = any && (p->want_dx || p->want_dw) && (act || !dy_ok);
    p->pass = any && (p->write_g || p->want_db);
    p->ldg = p->write_g ? round_up(p->N, 8) : p->M <= 1 ? round_up(p->N, 8) : d.dy.row_stride;
    p->g_bytes = p->write_g ? round_up(p->M * p->ldg * 2, kWsAlign) : 0;
    p->wide = wide && act && p->write_g;  // without a slope g is dy, of one term
    if (p->pass || p->want_db) {
        // about two thousand workgroups of 512 columns, at least 16 rows each
        const int64_t strips = ceil_div(p->N > 0 ? p->N : 1, 512);
        int64_t blocks = ceil_div(2048, strips);
        if (blocks > ceil_div(p->M, 16))
            blocks = ceil_div(p->M, 16);
        if (blocks < 1)
            blocks = 1;
        p->rows = (int)ceil_div(p->M > 0 ? p->M : 1, blocks);
        p->row_blocks = (int)ceil_div(p->M, p->rows);
        p->sum_ld = round_up(p->N, 32);
        p->sum_bytes = p->want_db ? round_up(p->row_blocks * p->sum_ld * 4, kWsAlign) : 0;
    }
    Operand g;
    g.es = 2;
    g.ld = p->ldg * 2;
    p->ga = g;
    p->ga.dim = p->M;
    p->ga.inner = p->N;
    p->gt = g;
    p->gt.cols = true;
    p->gt.dim = p->N;
    p->gt.inner = p->M;
    Forced forced;
    DENSE_TRY(forced_tile(&forced));
    double apart = 0.0;
    if (p->want_dx) {
        p->wb.src = d.w.ptr;
        p->wb.rs = d.w.col_stride;
        p->wb.cs = d.w.row_stride;
        p->wb.dim = p->K;
        p->wb.inner = p->N;
        plan_operand(&p->wb, false, true);
        DENSE_TRY(check_reach(p->ga));
        DENSE_TRY(check_reach(p->wb));
        apart += plan_gemm(p->M, p->K, p->N, 2, forced, &p->dx);
        if (p->wide)
            two_terms(p->M, &p->dx);
        if (!grid_fits(p->dx, p->M))
            return CONV_I8_ERR_UNSUPPORTED;
        p->part_bytes = p->dx.part_bytes;
    }
    if (p->want_dw) {
        p->xb.src = d.x.ptr;
        p->xb.rs = d.x.col_stride;
        p->xb.cs = d.x.row_stride;
        p->xb.dim = p->K;
        p->xb.inner = p->M;
        plan_operand(&p->xb, false, true);
        DENSE_TRY(check_reach(p->gt));
        DENSE_TRY(check_reach(p->xb));
        apart += plan_gemm(p->N, p->K, p->M, 2, forced, &p->dw);
        // apart: a launch more, and the bias gradient's (320x400x7312: 26 us apart, 21 paired)
        if (p->wide)
            two_terms(p->N, &p->dw);
        if (!p->wide && p->want_dx && !forced.on && pair_cost(p->M, p->N, p->K) < apart + 4.0) {
            set_plan(p->M, p->K, p->N, 2, kPairTile, 1, &p->dx);
            set_plan(p->N, p->K, p->M, 2, kPairTile, 1, &p->dw);
            p->part_bytes = 0;
        }
        if (!grid_fits(p->dw, p->N))
            return CONV_I8_ERR_UNSUPPORTED;
        if (p->dw.part_bytes > p->part_bytes)
            p->part_bytes = p->dw.part_bytes;  // the two products run one after the other
    }
    if (!launch_fits(ceil_div(p->N, 512) * p->row_blocks + pack_wgs(p->wb) + pack_wgs(p->xb), 256))
        return CONV_I8_ERR_UNSUPPORTED;
    p->ws_bytes = (p->wide ? 2 : 1) * p->g_bytes + p->sum_bytes + p->wb.pack_bytes + p->xb.pack_bytes + p->part_bytes;
    return CONV_I8_OK;
}

template <typename T, int ACT>
void launch_prepare_act(dim3 grid, const ActGradArgs &a, const PackArgs &pack, hipStream_t stream)
{
    if (ACT != DENSE_ACT_NONE && a.g2)
        hipLaunchKernelGGL((act_grad_kernel<T, ACT, ACT != DENSE_ACT_NONE>), grid, dim3(256), 0, stream, a, pack);
    else
        hipLaunchKernelGGL((act_grad_kernel<T, ACT, false>), grid, dim3(256), 0, stream, a, pack);
}

template <typename T>
void launch_prepare(int64_t act, dim3 grid, const ActGradArgs &a, const PackArgs &pack, hipStream_t stream)
{
    switch (act) {
    case DENSE_ACT_RELU: launch_prepare_act<T, DENSE_ACT_RELU>(grid, a, pack, stream); break;
    case DENSE_ACT_GELU: launch_prepare_act<T, DENSE_ACT_GELU>(grid, a, pack, stream); break;
    case DENSE_ACT_GELU_TANH: launch_prepare_act<T, DENSE_ACT_GELU_TANH>(grid, a, pack, stream); break;
    case DENSE_ACT_SILU: launch_prepare_act<T, DENSE_ACT_SILU>(grid, a, pack, stream); break;
    default: launch_prepare_act<T, DENSE_ACT_NONE>(grid, a, pack, stream); break;
    }
}

conv_i8_status_t run_backward(const BackwardPlan &p, void *ws, hipStream_t stream)
{
    const dense_linear_backward_t &d = p.d;
    const int64_t dt = d.dy.dtype;
    uint8_t *g = (uint8_t *)ws, *g2 = g + (p.wide ? p.g_bytes : 0), *sums = g2 + p.g_bytes, *pw = sums + p.sum_bytes, *px = pw + p.wb.pack_bytes;
    uint8_t *part = px + p.xb.pack_bytes;
    if (p.pass) {
        ActGradArgs a;
        memset(&a, 0, sizeof a);
        a.dy = d.dy.ptr;
        a.z = d.activation != DENSE_ACT_NONE ? d.preact.ptr : nullptr;
        a.ldy = d.dy.row_stride;
        a.ldz = d.preact.row_stride;
        a.M = (int)p.M;
        a.N = (int)p.N;
        a.rows = p.rows;
        a.g = p.write_g ? g : nullptr;
        a.g2 = p.wide ? g2 : nullptr;
        a.ldg = p.ldg;
        a.colsum = p.want_db ? (float *)sums : nullptr;
        a.sum_ld = p.sum_ld;
        a.strips = (int)ceil_div(p.N, 512);
        a.blocks = a.strips * p.row_blocks;
        PackArgs pack;
        const int64_t wgs = a.blocks + pack_jobs(p.wb, pw, p.xb, px, &pack);
        const dim3 grid((unsigned)wgs);
        if (dt == DENSE_BF16)
            launch_prepare<bf16>(d.activation, grid, a, pack, stream);
        else
            launch_prepare<f16>(d.activation, grid, a, pack, stream);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    ColSumArgs c;
    memset(&c, 0, sizeof c);
    if (p.want_db) {
        c.part = (const float *)sums;
        c.ld = p.sum_ld;
        c.rows = p.row_blocks;  // none: zeros
        c.cols = c.split = c.valid = p.N;
        c.out0 = const_cast<void *>(d.dbias.ptr);
        c.dt = (int)dt;
    }
    if (!p.pass && !launch_pack(p.wb, pw, p.xb, px, stream))
        return CONV_I8_ERR_HIP;
    const void *gp = p.write_g ? (const void *)g : d.dy.ptr;
    Epilogue e;
    memset(&e, 0, sizeof e);
    e.out_dt = (int)dt;
    GemmArgs dx, dw;
    if (p.want_dx) {
        e.out = const_cast<void *>(d.dx.ptr);
        e.ldo = d.dx.row_stride;
        dx = gemm_args(p.ga, gp, p.wb, p.wb.packed ? pw : p.wb.src, p.M, p.K, p.N, p.dx, part, e);
    }
    if (p.want_dw) {
        e.out = const_cast<void *>(d.dw.ptr);
        e.ldo = d.dw.row_stride;
        dw = gemm_args(p.gt, gp, p.xb, p.xb.packed ? px : p.xb.src, p.N, p.K, p.M, p.dw, part, e);
    }
    if (p.pair()) {
        const PairArgs both = {dx, dw, c};
        const bool ok = dt == DENSE_BF16 ? launch_gemm_pair_bf16(both, stream) : launch_gemm_pair_f16(both, stream);
        return ok ? CONV_I8_OK : CONV_I8_ERR_HIP;
    }
    if (p.want_db) {
        hipLaunchKernelGGL(colsum_kernel<>, colsum_grid(p.N), dim3(32 * kSumGroups), 0, stream, c);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    if (p.want_dx && !run_gemm(dt, p.ga, p.wb, p.dx, dx, stream, g2))
        return CONV_I8_ERR_HIP;
    if (p.want_dw && !run_gemm(dt, p.gt, p.xb, p.dw, dw, stream, g2))
        return CONV_I8_ERR_HIP;
    return CONV_I8_OK;
}

}  // namespace
}  // namespace dense

using namespace dense;

extern "C" {

conv_i8_status_t dense_linear_workspace_size(const dense_linear_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    LinearPlan p;
    DENSE_TRY(analyze(args, &p));
    *bytes = (size_t)p.ws_bytes;
    return CONV_I8_OK;
}

conv_i8_status_t dense_linear(const dense_linear_t *args, void *workspace, size_t bytes, void *stream)
{
    LinearPlan p;
    DENSE_TRY(analyze(args, &p));
    if (p.M == 0 || p.N == 0)
        return CONV_I8_OK;
    DENSE_TRY(check_workspace(workspace, bytes, p.ws_bytes));
    return run_linear(p, workspace, (hipStream_t)stream);
}

conv_i8_status_t dense_linear_plan(const dense_linear_t *args, char *buf, size_t len)
{
    if (!buf)
        return CONV_I8_ERR_NULL;
    LinearPlan p;
    DENSE_TRY(analyze(args, &p));
    char text[256];
    if (p.M == 0 || p.N == 0)
        snprintf(text, sizeof text, "kernel=none");
    else if (p.skinny)
        snprintf(text, sizeof text, "kernel=skinny waves=%d aligned=%d", p.waves, (int)p.aligned);
    else {
        char t[200];
        describe(p.gemm, p.a, p.b, t, sizeof t);
        snprintf(text, sizeof text, "kernel=gemm %s", t);
    }
    if (strlen(text) + 1 > len)
        return CONV_I8_ERR_PARAM;
    memcpy(buf, text, strlen(text) + 1);
    return CONV_I8_OK;
}

conv_i8_status_t dense_linear_backward_workspace_size(const dense_linear_backward_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    BackwardPlan p;
    DENSE_TRY(analyze(args, &p));
    *bytes = (size_t)p.ws_bytes;
    return CONV_I8_OK;
}

conv_i8_status_t dense_linear_backward(const dense_linear_backward_t *args, void *workspace, size_t bytes,
                                       void *stream)
{
    BackwardPlan p;
    DENSE_TRY(analyze(args, &p));
    DENSE_TRY(check_workspace(workspace, bytes, p.ws_bytes));
    return run_backward(p, workspace, (hipStream_t)stream);
}

conv_i8_status_t dense_linear_backward_plan(const dense_linear_backward_t *args, char *buf, size_t len)
{
    if (!buf)
        return CONV_I8_ERR_NULL;
    BackwardPlan p;
    DENSE_TRY(analyze(args, &p));
    char text[512], dx[200] = "none", dw[200] = "none";
    if (p.want_dx)
        describe(p.dx, p.ga, p.wb, dx, sizeof dx);
    if (p.want_dw)
        describe(p.dw, p.gt, p.xb, dw, sizeof dw);
    snprintf(text, sizeof text, "g=%s launches=%s dx: %s; dw: %s", p.wide ? "written_wide" : p.write_g ? "written" : "dy",
             p.pair() ? "paired" : "apart", dx, dw);
    if (strlen(text) + 1 > len)
        return CONV_I8_ERR_PARAM;
    memcpy(buf, text, strlen(text) + 1);
    return CONV_I8_OK;
}

}  // extern "C"
