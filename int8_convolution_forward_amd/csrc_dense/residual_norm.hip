// C entries of the norm fused with a residual connection, and of its gradients:
// argument checks, the choice of kernel, the launches.
#include <string.h>

#include "host_common.hpp"
#include "residual_norm_launch.hpp"

namespace dense {
namespace {

constexpr int64_t kWsAlign = 256;
constexpr int64_t kMaxGridY = 65535;

// The sums over workgroups: blockIdx.y 0 dweight, 1 dbias, 2 dpost_weight, 3 + g row g of dgate.
struct ResNormSumArgs {
    const float *part;
    int64_t part_ld;
    int wgs, chunks, D, dt;
    void *out[3], *dgate;             // null: not wanted
    int64_t lddg;
};

__global__ __launch_bounds__(32 * kSumGroups) void residual_norm_sums_kernel(const ResNormSumArgs a)
{
    __shared__ float red[kSumGroups][33];
    const int job = blockIdx.y;
    ColSumArgs c;
    c.ld = 4 * a.part_ld;
    c.cols = c.split = c.valid = a.D;
    c.out1 = nullptr;
    c.dt = a.dt;
    if (job < 3) {
        c.part = a.part + job * a.part_ld;
        c.rows = a.wgs;
        c.out0 = a.out[job];
    } else {
        const int g = job - 3;
        c.part = a.part + ((int64_t)g * a.chunks * 4 + 3) * a.part_ld;
        c.rows = a.chunks;
        c.out0 = (char *)a.dgate + g * a.lddg * (a.dt == DENSE_FP32 ? 4 : 2);
    }
    if (c.out0)
        column_sums<32>(c, blockIdx.x, red);
}

// Present, [M, D] of type dt, rows contiguous
conv_i8_status_t check_rows(dense_mat_t *m, int64_t M, int64_t D, int64_t dt, bool output)
{
    DENSE_TRY(check_mat(m, output));
    if (m->dtype != dt)
        return CONV_I8_ERR_DTYPE;
    if (m->rows != M || m->cols != D)
        return output ? CONV_I8_ERR_OUT_DIMS : CONV_I8_ERR_DIMS;
    return m->col_stride == 1 ? CONV_I8_OK : CONV_I8_ERR_STRIDES;
}

conv_i8_status_t check_like(dense_vec_t *v, int64_t n, int64_t dt)
{
    DENSE_TRY(check_vec(v, n));
    return v->dtype == DENSE_NONE || v->dtype == dt ? CONV_I8_OK : CONV_I8_ERR_DTYPE;
}

// A gate of G rows for M: M is a multiple of G
conv_i8_status_t check_gate(dense_mat_t *g, int64_t M, int64_t D, int64_t dt, bool output)
{
    DENSE_TRY(check_rows(g, g->rows, D, dt, output));
    if (g->rows < 1 ? M > 0 || g->rows < 0 : M % g->rows != 0)
        return CONV_I8_ERR_DIMS;
    return CONV_I8_OK;
}

conv_i8_status_t analyze(const dense_residual_norm_t *args, dense_residual_norm_t *d)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    *d = *args;
    DENSE_TRY(check_mat(&d->x, false));
    const int64_t dt = d->x.dtype, M = d->x.rows, D = d->x.cols;
    if (!is_float(dt))
        return CONV_I8_ERR_DTYPE;
    if (D < 1)
        return CONV_I8_ERR_DIMS;
    if (d->x.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    if (d->h.dtype == DENSE_NONE) {
        if (d->gate.dtype != DENSE_NONE || d->post_weight.dtype != DENSE_NONE || d->r.dtype != DENSE_NONE)
            return CONV_I8_ERR_PARAM;
    } else {
        DENSE_TRY(check_rows(&d->h, M, D, dt, false));
        if (d->r.dtype == DENSE_NONE)
            return CONV_I8_ERR_NULL;
        DENSE_TRY(check_rows(&d->r, M, D, dt, true));
        if (d->gate.dtype != DENSE_NONE)
            DENSE_TRY(check_gate(&d->gate, M, D, dt, false));
    }
    const bool q8 = d->y.dtype == DENSE_E4M3;
    if (q8) {
        DENSE_TRY(check_mat_of(&d->y, true, 1));
        if (d->y.rows != M || d->y.cols != D)
            return CONV_I8_ERR_OUT_DIMS;
        DENSE_TRY(check_scales(&d->y_scale, M, D, true, nullptr));
    } else {
        if (d->y_scale.dtype != DENSE_NONE)
            return CONV_I8_ERR_PARAM;
        DENSE_TRY(check_rows(&d->y, M, D, dt, true));
    }
    DENSE_TRY(check_like(&d->post_weight, D, dt));
    DENSE_TRY(check_like(&d->weight, D, dt));
    DENSE_TRY(check_like(&d->bias, D, dt));
    for (dense_vec_t *v : {&d->mean, &d->rstd, &d->post_mean, &d->post_rstd})
        DENSE_TRY(check_like(v, M, DENSE_FP32));
    if (d->post_weight.dtype == DENSE_NONE && (d->post_mean.dtype != DENSE_NONE || d->post_rstd.dtype != DENSE_NONE))
        return CONV_I8_ERR_PARAM;
    if (!(d->eps >= 0.0) || d->alpha != d->alpha || (d->kind != DENSE_LAYER_NORM && d->kind != DENSE_RMS_NORM))
        return CONV_I8_ERR_PARAM;
    return CONV_I8_OK;
}

struct BackPlan {
    dense_residual_norm_backward_t d;
    int64_t M, D;
    bool sums;
    int groups = 1, chunks = 1, wgs = 0;
    int64_t part_ld = 0, part_bytes = 0, ws_bytes = 0;
    bool any() const { return !back_in_registers(D); }
    // Rows of the gate whose gradients residual_norm_sums_kernel writes: a workgroup that takes
    // all rows of one has written it.
    int64_t gate_sums() const { return d.dgate.dtype != DENSE_NONE && (chunks > 1 || M == 0) ? groups : 0; }
};

conv_i8_status_t analyze(const dense_residual_norm_backward_t *args, BackPlan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_residual_norm_backward_t &d = p->d;
    DENSE_TRY(check_mat(&d.r, false));
    const int64_t dt = d.r.dtype, M = p->M = d.r.rows, D = p->D = d.r.cols;
    if (!is_float(dt))
        return CONV_I8_ERR_DTYPE;
    if (D < 1)
        return CONV_I8_ERR_DIMS;
    if (d.r.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    DENSE_TRY(check_rows(&d.dy, M, D, dt, false));
    if (d.dr.dtype != DENSE_NONE)
        DENSE_TRY(check_rows(&d.dr, M, D, dt, false));
    else
        d.dr.ptr = nullptr;
    DENSE_TRY(check_rows(&d.dx, M, D, dt, true));
    const bool gate = d.gate.dtype != DENSE_NONE, post = d.post_weight.dtype != DENSE_NONE;
    if (d.dh.dtype == DENSE_NONE) {
        if (gate || post || d.dgate.dtype != DENSE_NONE || d.dpost_weight.dtype != DENSE_NONE)
            return CONV_I8_ERR_PARAM;
        d.h.ptr = nullptr;
    } else {
        DENSE_TRY(check_rows(&d.dh, M, D, dt, true));
        if (gate || post) {
            if (d.h.dtype == DENSE_NONE)
                return CONV_I8_ERR_NULL;
            DENSE_TRY(check_rows(&d.h, M, D, dt, false));
        }
    }
    if (gate)
        DENSE_TRY(check_gate(&d.gate, M, D, dt, false));
    if (d.dgate.dtype != DENSE_NONE) {
        if (!gate)
            return CONV_I8_ERR_PARAM;
        DENSE_TRY(check_rows(&d.dgate, d.gate.rows, D, dt, true));
    }
    DENSE_TRY(check_like(&d.weight, D, dt));
    DENSE_TRY(check_like(&d.post_weight, D, dt));
    for (dense_vec_t *v : {&d.dweight, &d.dbias, &d.dpost_weight})
        DENSE_TRY(check_like(v, D, dt));
    if (!post && d.dpost_weight.dtype != DENSE_NONE)
        return CONV_I8_ERR_PARAM;
    if (d.kind != DENSE_LAYER_NORM && d.kind != DENSE_RMS_NORM)
        return CONV_I8_ERR_PARAM;
    if (d.alpha != d.alpha)
        return CONV_I8_ERR_PARAM;
    const bool rms = d.kind == DENSE_RMS_NORM;
    if (d.rstd.dtype == DENSE_NONE || (post && d.post_rstd.dtype == DENSE_NONE) ||
        (!rms && (d.mean.dtype == DENSE_NONE || (post && d.post_mean.dtype == DENSE_NONE))))
        return CONV_I8_ERR_NULL;
    for (dense_vec_t *v : {&d.mean, &d.rstd, &d.post_mean, &d.post_rstd})
        DENSE_TRY(check_like(v, M, DENSE_FP32));

    const bool dgate = d.dgate.dtype != DENSE_NONE;
    p->sums = dgate || d.dweight.dtype != DENSE_NONE || d.dbias.dtype != DENSE_NONE || d.dpost_weight.dtype != DENSE_NONE;
    p->part_ld = round_up(D, 8);
    p->groups = gate ? (int)d.gate.rows : 1;
    // Workgroups: one or two on a CU, but two rows at least for each of their groups of
    // threads; more leave more partial sums.  One takes part of the rows of a row of the gate or
    // those of several.
    const int threads = norm_threads(back_threads(D)), rpw = threads / back_threads(D);
    const int64_t most = threads <= 256 ? 2 * kCUs : kCUs, rows = p->any() ? 64 : 2 * rpw;
    const int64_t want = ceil_div(M, rows) < most ? ceil_div(M, rows) : most;
    if (M > 0) {
        p->chunks = want >= 2 * p->groups ? (int)(want / p->groups) : 1;
        p->wgs = p->chunks > 1 || want > p->groups ? p->groups * p->chunks : (int)want;
    }
    p->part_bytes = p->sums && p->wgs ? round_up((int64_t)p->wgs * 4 * p->part_ld * 4, kWsAlign) : 0;
    // residual_norm_columns_kernel takes fewer threads
    if (p->sums && (3 + p->gate_sums() > kMaxGridY || !launch_fits(ceil_div(D, 32) * (3 + p->gate_sums()), 32 * kSumGroups)))
        return CONV_I8_ERR_UNSUPPORTED;
    p->ws_bytes = p->part_bytes + (p->sums && p->any() ? round_up(M * 8, kWsAlign) : 0);
    return CONV_I8_OK;
}

}  // namespace
}  // namespace dense

using namespace dense;

extern "C" {

conv_i8_status_t dense_residual_norm(const dense_residual_norm_t *args, void *stream)
{
    dense_residual_norm_t d;
    DENSE_TRY(analyze(args, &d));
    if (d.x.rows == 0)
        return CONV_I8_OK;
    ResNormArgs a;
    memset(&a, 0, sizeof a);
    a.x = d.x.ptr;
    a.ldx = d.x.row_stride;
    a.M = (int)d.x.rows;
    a.D = (int)d.x.cols;
    a.d = (float)a.D;
    a.gate_rows = 1;
    if (d.h.dtype != DENSE_NONE) {
        a.h = d.h.ptr;
        a.ldh = d.h.row_stride;
        a.r = const_cast<void *>(d.r.ptr);
        a.ldr = d.r.row_stride;
        a.post_weight = d.post_weight.ptr;
        if (d.gate.dtype != DENSE_NONE) {
            a.gate = d.gate.ptr;
            a.ldg = d.gate.row_stride;
            a.gate_rows = (int)(d.x.rows / d.gate.rows);
        }
    }
    a.weight = d.weight.ptr;
    a.bias = d.bias.ptr;
    a.y = const_cast<void *>(d.y.ptr);
    a.ldy = d.y.row_stride;
    const bool q8 = d.y.dtype == DENSE_E4M3;
    if (q8) {
        a.y_scale = (uint8_t *)const_cast<void *>(d.y_scale.ptr);
        a.ldys = d.y_scale.row_stride;
    }
    a.alpha = (float)d.alpha;
    a.eps = (float)d.eps;
    a.mean = (float *)const_cast<void *>(d.mean.ptr);
    a.rstd = (float *)const_cast<void *>(d.rstd.ptr);
    a.post_mean = (float *)const_cast<void *>(d.post_mean.ptr);
    a.post_rstd = (float *)const_cast<void *>(d.post_rstd.ptr);
    const bool rms = d.kind == DENSE_RMS_NORM;
    hipStream_t s = (hipStream_t)stream;
    if (d.x.dtype == DENSE_BF16)
        launch_residual_norm_bf16(a, rms, q8, s);
    else if (d.x.dtype == DENSE_FP16)
        launch_residual_norm_f16(a, rms, q8, s);
    else
        launch_residual_norm_f32(a, rms, q8, s);
    return hipGetLastError() == hipSuccess ? CONV_I8_OK : CONV_I8_ERR_HIP;
}

conv_i8_status_t dense_residual_norm_backward_workspace_size(const dense_residual_norm_backward_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    BackPlan p;
    DENSE_TRY(analyze(args, &p));
    *bytes = (size_t)p.ws_bytes;
    return CONV_I8_OK;
}

conv_i8_status_t dense_residual_norm_backward(const dense_residual_norm_backward_t *args, void *workspace, size_t bytes,
                                              void *stream)
{
    BackPlan p;
    DENSE_TRY(analyze(args, &p));
    if (p.ws_bytes > 0) {
        if (bytes < (size_t)p.ws_bytes || ((uintptr_t)workspace & (kWsAlign - 1)) != 0)
            return CONV_I8_ERR_WORKSPACE;
        if (!workspace)
            return CONV_I8_ERR_NULL;
    }
    const dense_residual_norm_backward_t &d = p.d;
    ResNormBackArgs a;
    memset(&a, 0, sizeof a);
    a.dr = d.dr.ptr;
    a.lddr = d.dr.row_stride;
    a.dy = d.dy.ptr;
    a.lddy = d.dy.row_stride;
    a.r = d.r.ptr;
    a.ldr = d.r.row_stride;
    a.h = d.h.ptr;
    a.ldh = d.h.row_stride;
    a.weight = d.weight.ptr;
    a.post_weight = d.post_weight.ptr;
    a.mean = (const float *)d.mean.ptr;
    a.rstd = (const float *)d.rstd.ptr;
    a.post_mean = (const float *)d.post_mean.ptr;
    a.post_rstd = (const float *)d.post_rstd.ptr;
    a.dx = const_cast<void *>(d.dx.ptr);
    a.lddx = d.dx.row_stride;
    if (d.dh.dtype != DENSE_NONE) {
        a.dh = const_cast<void *>(d.dh.ptr);
        a.lddh = d.dh.row_stride;
    }
    if (d.gate.dtype != DENSE_NONE) {
        a.gate = d.gate.ptr;
        a.ldg = d.gate.row_stride;
    }
    if (d.dgate.dtype != DENSE_NONE) {
        a.dgate = const_cast<void *>(d.dgate.ptr);
        a.lddg = d.dgate.row_stride;
    }
    a.M = (int)p.M;
    a.D = (int)p.D;
    a.d = (float)a.D;
    a.inv_d = 1.0f / a.d;
    a.alpha = (float)d.alpha;
    a.groups = p.groups;
    a.chunks = p.chunks;
    a.gate_rows = p.M > 0 ? (int)(p.M / p.groups) : 1;
    a.part = p.sums ? (float *)workspace : nullptr;
    a.part_ld = p.part_ld;
    a.row_sums = p.sums && p.any() ? (float2 *)((char *)workspace + p.part_bytes) : nullptr;
    hipStream_t s = (hipStream_t)stream;
    const bool post = d.post_weight.dtype != DENSE_NONE;
    if (p.M > 0) {
        const bool rms = d.kind == DENSE_RMS_NORM;
        if (d.r.dtype == DENSE_BF16)
            launch_residual_norm_backward_bf16(a, rms, post, p.wgs, s);
        else if (d.r.dtype == DENSE_FP16)
            launch_residual_norm_backward_f16(a, rms, post, p.wgs, s);
        else
            launch_residual_norm_backward_f32(a, rms, post, p.wgs, s);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    if (p.sums) {
        ResNormSumArgs c;
        memset(&c, 0, sizeof c);
        c.part = a.part;
        c.part_ld = p.part_ld;
        c.wgs = p.wgs;  // none: zeros
        c.chunks = p.M > 0 ? p.chunks : 0;
        c.D = a.D;
        c.dt = (int)d.r.dtype;
        c.out[0] = const_cast<void *>(d.dweight.ptr);
        c.out[1] = const_cast<void *>(d.dbias.ptr);
        c.out[2] = const_cast<void *>(d.dpost_weight.ptr);
        c.dgate = a.dgate;
        c.lddg = a.lddg;
        const dim3 grid((unsigned)ceil_div(p.D, 32), (unsigned)(3 + p.gate_sums()));
        hipLaunchKernelGGL(residual_norm_sums_kernel, grid, dim3(32 * kSumGroups), 0, s, c);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    return CONV_I8_OK;
}

}  // extern "C"
