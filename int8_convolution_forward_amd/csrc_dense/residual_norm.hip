// C entries of the norm fused with a residual connection, and of its gradients:
// argument checks, the choice of kernel, the launches.
#include <string.h>

#include "host_common.hpp"
#include "residual_norm_kernel.hpp"

namespace dense {
namespace {

constexpr int64_t kWsAlign = 256;
// Longest rows that stay in registers, forward and backward.
constexpr int64_t kRow = 16384, kBackRow = 8192;

template <typename T> struct As { typedef T type; };
template <bool B> struct Flag { static constexpr bool value = B; };

// f(As<type>, Flag<RMS>)
template <typename F>
void by_type(int64_t dt, bool rms, F f)
{
    auto with = [&](auto t) { rms ? f(t, Flag<true>{}) : f(t, Flag<false>{}); };
    if (dt == DENSE_BF16)
        with(As<bf16>{});
    else if (dt == DENSE_FP16)
        with(As<f16>{});
    else
        with(As<float>{});
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

inline unsigned capped(int64_t wgs, int threads)
{
    const int64_t most = threads <= 256 ? 1 << 21 : 1 << 16;
    return (unsigned)(wgs < most ? wgs : most);
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

template <typename T, bool RMS, bool Q8, int P, int V>
void launch_rows(const ResNormArgs &a, hipStream_t s)
{
    constexpr int rows = norm_threads(P) / P;
    constexpr bool hold = P <= 512;
    int64_t wgs = ceil_div(a.M, rows);
    if (hold && wgs > 1024)
        wgs = P > 256 || wgs <= 2048 ? 1024 : ceil_div(wgs, 2);
    const dim3 grid(capped(wgs, norm_threads(P))), block(norm_threads(P));
    if (a.D % 8 == 0)
        hipLaunchKernelGGL((residual_norm_kernel<T, P, V, hold, false, RMS, Q8>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((residual_norm_kernel<T, P, V, hold, true, RMS, Q8>), grid, block, 0, s, a);
}

template <typename T, bool RMS, bool Q8>
void launch(const ResNormArgs &a, hipStream_t s)
{
    const int D = a.D;
    // a wave per row while that gives each CU a few waves, else a workgroup per row
    const bool few = a.M < 4 * kCUs;
    if (D < 8)
        hipLaunchKernelGGL((residual_norm_any_kernel<T, 64, RMS, Q8>), dim3(capped(a.M, 64)), dim3(64), 0, s, a);
    else if (D > kRow)
        hipLaunchKernelGGL((residual_norm_any_kernel<T, 1024, RMS, Q8>), dim3(capped(a.M, 1024)), dim3(1024), 0, s, a);
    else if (D <= 512)
        launch_rows<T, RMS, Q8, 64, 1>(a, s);
    else if (D <= 1024 && !few)
        launch_rows<T, RMS, Q8, 64, 2>(a, s);
    else if (D <= 2048)
        launch_rows<T, RMS, Q8, 256, 1>(a, s);
    else if (D <= 4096)
        launch_rows<T, RMS, Q8, 512, 1>(a, s);
    else if (D <= 8192)
        launch_rows<T, RMS, Q8, 512, 2>(a, s);
    else
        launch_rows<T, RMS, Q8, 1024, 2>(a, s);
}

struct BackPlan {
    dense_residual_norm_backward_t d;
    int64_t M, D;
    bool sums;
    int groups = 1, chunks = 1, each = 1, wgs = 0;
    int64_t part_ld = 0, part_bytes = 0, ws_bytes = 0;
    bool any() const { return D < 8 || D > kBackRow; }
};

constexpr int back_threads(int64_t D) { return D <= 1024 ? 64 : D <= 2048 ? 256 : 512; }

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
    // Workgroups: one or two on a CU, but four rows at least for each of their groups of
    // threads; more leave more partial sums.  One takes part of the rows of a row of the gate or
    // those of several.
    const int threads = norm_threads(back_threads(D)), rpw = threads / back_threads(D);
    const int64_t most = threads <= 256 ? 2 * kCUs : kCUs, rows = p->any() ? 64 : 4 * rpw;
    const int64_t want = ceil_div(M, rows) < most ? ceil_div(M, rows) : most;
    if (M > 0) {
        if (want >= 2 * p->groups)
            p->chunks = (int)(want / p->groups);
        else
            p->each = (int)ceil_div(p->groups, want);
        p->wgs = (int)(p->chunks > 1 ? (int64_t)p->groups * p->chunks : ceil_div(p->groups, p->each));
    }
    p->part_bytes = p->sums && p->wgs ? round_up((int64_t)p->wgs * 4 * p->part_ld * 4, kWsAlign) : 0;
    p->ws_bytes = p->part_bytes + (p->sums && p->any() ? round_up(M * 8, kWsAlign) : 0);
    return CONV_I8_OK;
}

template <typename T, bool RMS, bool POST, int P, int V, int AHEAD>
void launch_back_rows(const ResNormBackArgs &a, int wgs, hipStream_t s)
{
    const dim3 grid((unsigned)wgs), block(norm_threads(P));
    if (a.D % 8 == 0)
        hipLaunchKernelGGL((residual_norm_backward_kernel<T, P, V, AHEAD, false, RMS, POST>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((residual_norm_backward_kernel<T, P, V, AHEAD, true, RMS, POST>), grid, block, 0, s, a);
}

template <typename T, bool RMS, bool POST>
void launch_back(const ResNormBackArgs &a, const BackPlan &p, hipStream_t s)
{
    if (p.any()) {
        if (p.D < 8)
            hipLaunchKernelGGL((residual_norm_backward_any_kernel<T, 64, RMS, POST>), dim3(capped(a.M, 64)), dim3(64), 0, s, a);
        else
            hipLaunchKernelGGL((residual_norm_backward_any_kernel<T, 1024, RMS, POST>), dim3(capped(a.M, 1024)), dim3(1024), 0, s, a);
        if (p.sums)
            hipLaunchKernelGGL((residual_norm_columns_kernel<T, RMS, POST>), dim3((unsigned)ceil_div(p.D, 2048), (unsigned)p.wgs),
                               dim3(256), 0, s, a);
    } else if (p.D <= 512) {
        launch_back_rows<T, RMS, POST, 64, 1, 1>(a, p.wgs, s);
    } else if (p.D <= 1024) {
        launch_back_rows<T, RMS, POST, 64, 2, (sizeof(T) == 2)>(a, p.wgs, s);
    } else if (p.D <= 2048) {
        launch_back_rows<T, RMS, POST, 256, 1, 1>(a, p.wgs, s);
    } else if (p.D <= 4096) {
        launch_back_rows<T, RMS, POST, 512, 1, 1>(a, p.wgs, s);
    } else {
        launch_back_rows<T, RMS, POST, 512, 2, 0>(a, p.wgs, s);
    }
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
    by_type(d.x.dtype, d.kind == DENSE_RMS_NORM, [&](auto t, auto rms) {
        typedef typename decltype(t)::type T;
        constexpr bool RMS = decltype(rms)::value;
        q8 ? launch<T, RMS, true>(a, (hipStream_t)stream) : launch<T, RMS, false>(a, (hipStream_t)stream);
    });
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
    a.alpha = (float)d.alpha;
    a.groups = p.groups;
    a.chunks = p.chunks;
    a.each = p.each;
    a.gate_rows = p.M > 0 ? (int)(p.M / p.groups) : 1;
    a.part = p.sums ? (float *)workspace : nullptr;
    a.part_ld = p.part_ld;
    a.row_sums = p.sums && p.any() ? (float2 *)((char *)workspace + p.part_bytes) : nullptr;
    hipStream_t s = (hipStream_t)stream;
    const bool post = d.post_weight.dtype != DENSE_NONE;
    if (p.M > 0) {
        by_type(d.r.dtype, d.kind == DENSE_RMS_NORM, [&](auto t, auto rms) {
            typedef typename decltype(t)::type T;
            constexpr bool RMS = decltype(rms)::value;
            post ? launch_back<T, RMS, true>(a, p, s) : launch_back<T, RMS, false>(a, p, s);
        });
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
        // a workgroup that takes all rows of a row of the gate has written it
        const bool gates = a.dgate && (p.chunks > 1 || p.M == 0);
        const dim3 grid((unsigned)ceil_div(p.D, 32), (unsigned)(3 + (gates ? p.groups : 0)));
        hipLaunchKernelGGL(residual_norm_sums_kernel, grid, dim3(32 * kSumGroups), 0, s, c);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    return CONV_I8_OK;
}

}  // extern "C"
