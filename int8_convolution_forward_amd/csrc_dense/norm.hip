// Layer norm's C entries: argument checks, the choice of kernel, the launches.
#include <string.h>

#include "colsum.hpp"
#include "host_common.hpp"
#include "norm_kernel.hpp"

namespace dense {
namespace {

constexpr int64_t kWsAlign = 256;
// Longest row that stays in registers, forward and backward.
constexpr int64_t kNormRow = 65536;
constexpr int64_t kBackRow = 16384;
// Longer rows are read again for each step; rows of fewer than eight columns have kernels of their own.
inline bool back_in_registers(int64_t D) { return D >= 8 && D <= kBackRow; }

conv_i8_status_t check_stat(dense_vec_t *v, int64_t n)
{
    DENSE_TRY(check_vec(v, n));
    return v->dtype == DENSE_NONE || v->dtype == DENSE_FP32 ? CONV_I8_OK : CONV_I8_ERR_DTYPE;
}

conv_i8_status_t analyze(const dense_layer_norm_t *args, dense_layer_norm_t *d)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    *d = *args;
    DENSE_TRY(check_mat(&d->x, false));
    DENSE_TRY(check_mat(&d->y, true));
    const int64_t dt = d->x.dtype, M = d->x.rows, D = d->x.cols;
    if (!is_float(dt) || (d->y.dtype != dt && d->y.dtype != DENSE_INT8))
        return CONV_I8_ERR_DTYPE;
    if (D < 1)
        return CONV_I8_ERR_DIMS;
    if (d->y.rows != M || d->y.cols != D)
        return CONV_I8_ERR_OUT_DIMS;
    if (d->x.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    DENSE_TRY(check_vec(&d->weight, D));
    DENSE_TRY(check_vec(&d->bias, D));
    for (const dense_vec_t *v : {&d->weight, &d->bias})
        if (v->dtype != DENSE_NONE && v->dtype != dt)
            return CONV_I8_ERR_DTYPE;
    DENSE_TRY(check_stat(&d->mean, M));
    DENSE_TRY(check_stat(&d->rstd, M));
    DENSE_TRY(check_stat(&d->scale, M));
    if ((d->scale.dtype != DENSE_NONE) != (d->y.dtype == DENSE_INT8))
        return CONV_I8_ERR_PARAM;
    if (!(d->eps >= 0.0))
        return CONV_I8_ERR_PARAM;
    return CONV_I8_OK;
}

// A launch has fewer than 2^32 threads: past so many workgroups they walk over rows.
inline unsigned capped(int64_t wgs, int threads)
{
    const int64_t most = threads <= 256 ? 1 << 21 : 1 << 16;
    return (unsigned)(wgs < most ? wgs : most);
}

// Two rows for each thread group once there are more than 1024 workgroups: the
// second one's loads overlap the first one's work, and the card still balances
// itself.  Over 180 shapes from 2048 x 64 to 200000 x 256 that is 1 % faster than
// one row in the mean, more for large ones (16384 x 4096 BF16 as int8 50.0 us, one
// row 54.2; 16384 x 8192 FP32 196 and 215), less below 10 us (10000 x 1024 BF16 9.6
// and 8.7; 2048 x 4096 BF16 9.3 and 8.7).
// Wide groups (512 threads) hold fewer workgroups on a CU and take more rows
// (4096 x 16384: four rows 55.4 us, two 59.3, one 74.4).
template <typename T, int P, int V, bool Q8>
void launch_one(const NormArgs &a, hipStream_t s)
{
    constexpr int rows = norm_threads(P) / P;
    constexpr bool hold = P <= 512;
    int64_t wgs = ceil_div(a.M, rows);
    if (hold && wgs > 1024)
        wgs = P > 256 || wgs <= 2048 ? 1024 : ceil_div(wgs, 2);
    const dim3 grid(capped(wgs, norm_threads(P))), block(norm_threads(P));
    if (a.D % 8 == 0)
        hipLaunchKernelGGL((norm_kernel<T, P, V, hold, false, Q8>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((norm_kernel<T, P, V, hold, true, Q8>), grid, block, 0, s, a);
}

template <typename T, bool Q8>
void launch_norm(const NormArgs &a, hipStream_t s)
{
    const int D = a.D;
    // a wave per row while that gives each CU a few waves, else a workgroup per row
    const bool few = a.M < 4 * kCUs;
    if (D <= kNarrow)
        hipLaunchKernelGGL((norm_narrow_kernel<T, Q8>), dim3(capped(ceil_div(a.M, 256), 256)), dim3(256), 0, s, a);
    else if (D > kNormRow)
        hipLaunchKernelGGL((norm_long_kernel<T, Q8>), dim3(capped(a.M, 1024)), dim3(1024), 0, s, a);
    else if (D <= 512)
        launch_one<T, 64, 1, Q8>(a, s);
    else if (D <= 1024 && !few)
        launch_one<T, 64, 2, Q8>(a, s);
    else if (D <= 2048)
        few ? launch_one<T, 256, 1, Q8>(a, s) : launch_one<T, 64, 4, Q8>(a, s);
    else if (D <= 4096)
        launch_one<T, 256, 2, Q8>(a, s);
    else if (D <= 8192)
        Q8 ? launch_one<T, 512, 2, Q8>(a, s) : launch_one<T, 256, 4, Q8>(a, s);
    else if (D <= 16384)
        launch_one<T, 512, 4, Q8>(a, s);
    else if (D <= 32768)
        launch_one<T, 1024, 4, Q8>(a, s);
    else
        launch_one<T, 1024, 8, Q8>(a, s);
}

struct BackPlan {
    dense_layer_norm_backward_t d;
    int64_t M, D;
    bool sums;
    bool once = false;   // norm_backward_once_kernel
    int wgs = 0;         // workgroups that walk the rows, or row blocks of a long row's sums
    int64_t part_ld = 0, ws_bytes = 0;
};

constexpr int back_threads(int64_t D) { return D <= 1024 ? 64 : D <= 2048 ? 256 : D <= 8192 ? 512 : 1024; }

conv_i8_status_t analyze(const dense_layer_norm_backward_t *args, BackPlan *p)
{
    if (!args)
        return CONV_I8_ERR_NULL;
    p->d = *args;
    dense_layer_norm_backward_t &d = p->d;
    DENSE_TRY(check_mat(&d.dy, false));
    DENSE_TRY(check_mat(&d.x, false));
    DENSE_TRY(check_mat(&d.dx, true));
    const int64_t dt = d.x.dtype;
    p->M = d.x.rows;
    p->D = d.x.cols;
    if (!is_float(dt) || d.dy.dtype != dt || d.dx.dtype != dt)
        return CONV_I8_ERR_DTYPE;
    if (p->D < 1 || d.dy.rows != p->M || d.dy.cols != p->D)
        return CONV_I8_ERR_DIMS;
    if (d.dx.rows != p->M || d.dx.cols != p->D)
        return CONV_I8_ERR_OUT_DIMS;
    if (d.x.col_stride != 1 || d.dy.col_stride != 1)
        return CONV_I8_ERR_STRIDES;
    DENSE_TRY(check_vec(&d.weight, p->D));
    DENSE_TRY(check_vec(&d.dweight, p->D));
    DENSE_TRY(check_vec(&d.dbias, p->D));
    for (const dense_vec_t *v : {&d.weight, &d.dweight, &d.dbias})
        if (v->dtype != DENSE_NONE && v->dtype != dt)
            return CONV_I8_ERR_DTYPE;
    if (d.mean.dtype == DENSE_NONE || d.rstd.dtype == DENSE_NONE)
        return CONV_I8_ERR_NULL;
    DENSE_TRY(check_stat(&d.mean, p->M));
    DENSE_TRY(check_stat(&d.rstd, p->M));
    if ((d.dweight.dtype == DENSE_NONE) != (d.dbias.dtype == DENSE_NONE))
        return CONV_I8_ERR_PARAM;
    p->sums = d.dweight.dtype != DENSE_NONE;
    p->part_ld = round_up(p->D, 8);
    if (p->D <= kNarrow) {
        // four rows a thread before there are more than two workgroups on a CU
        const int64_t want = ceil_div(p->M, 4 * 256);
        p->wgs = (int)(want < 2 * kCUs ? want : 2 * kCUs);
    } else if (!back_in_registers(p->D)) {
        const int64_t blocks = p->M < 64 ? p->M : 64;
        p->wgs = (int)(p->M > 0 ? ceil_div(p->M, ceil_div(p->M, blocks)) : 0);
    } else {
        // eight waves or more on a CU, and at least four rows for each group of threads: more
        // workgroups leave more partial sums (16384 x 4096 BF16: 256 workgroups of 512 threads
        // 74.0 us, 512 of 256 76.2, 512 of 512 75.9)
        const int threads = norm_threads(back_threads(p->D));
        const int rows = threads / back_threads(p->D), most = threads <= 256 ? 2 * kCUs : kCUs;
        const int64_t want = ceil_div(p->M, 4 * rows);
        p->wgs = (int)(want < most ? want : most);
    }
    p->once = p->sums && p->M > 0 && p->M <= once_rows(p->D) && back_in_registers(p->D);
    p->ws_bytes = p->sums && !p->once ? round_up((int64_t)p->wgs * 2 * p->part_ld * 4, kWsAlign) : 0;
    return CONV_I8_OK;
}

template <typename T, int P, int V, int AHEAD>
void launch_back_one(const NormBackArgs &a, int wgs, hipStream_t s)
{
    const dim3 block(norm_threads(P));
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)wgs), block, 0, s, a); };
    if (a.dweight) {
        const int cols = (int)ceil_div(a.D, kOnceCols);
        const dim3 grid((unsigned)(cols + ceil_div(a.M, norm_threads(P) / P)));
        if (a.D % 8 == 0)
            hipLaunchKernelGGL((norm_backward_once_kernel<T, P, V, false>), grid, block, 0, s, a, cols);
        else
            hipLaunchKernelGGL((norm_backward_once_kernel<T, P, V, true>), grid, block, 0, s, a, cols);
    } else if (a.D % 8 == 0) {
        a.part ? launch(norm_backward_kernel<T, P, V, AHEAD, false, true>)
               : launch(norm_backward_kernel<T, P, V, AHEAD, false, false>);
    } else {
        a.part ? launch(norm_backward_kernel<T, P, V, AHEAD, true, true>)
               : launch(norm_backward_kernel<T, P, V, AHEAD, true, false>);
    }
}

template <typename T>
void launch_back(const NormBackArgs &a, int wgs, hipStream_t s)
{
    const int D = a.D;
    if (D <= kNarrow) {
        hipLaunchKernelGGL(norm_backward_narrow_kernel<T>, dim3((unsigned)wgs), dim3(256), 0, s, a);
    } else if (!back_in_registers(D)) {
        hipLaunchKernelGGL(norm_backward_long_kernel<T>, dim3(capped(a.M, 1024)), dim3(1024), 0, s, a);
        if (a.part)
            hipLaunchKernelGGL(norm_backward_sums_kernel<T>, dim3((unsigned)ceil_div(D, 2048), (unsigned)wgs), dim3(256),
                               0, s, a, (int)ceil_div(a.M, wgs));
    } else if (D <= 512) {
        launch_back_one<T, 64, 1, 1>(a, wgs, s);
    } else if (D <= 1024) {
        launch_back_one<T, 64, 2, 1>(a, wgs, s);
    } else if (D <= 2048) {
        launch_back_one<T, 256, 1, 1>(a, wgs, s);
    } else if (D <= 4096) {
        launch_back_one<T, 512, 1, 1>(a, wgs, s);
    } else if (D <= 8192) {
        launch_back_one<T, 512, 2, 1>(a, wgs, s);
    } else {
        launch_back_one<T, 1024, 2, 0>(a, wgs, s);
    }
}

}  // namespace
}  // namespace dense

using namespace dense;

extern "C" {

conv_i8_status_t dense_layer_norm(const dense_layer_norm_t *args, void *stream)
{
    dense_layer_norm_t d;
    DENSE_TRY(analyze(args, &d));
    if (d.x.rows == 0)
        return CONV_I8_OK;
    NormArgs a;
    memset(&a, 0, sizeof a);
    a.x = d.x.ptr;
    a.weight = d.weight.ptr;
    a.bias = d.bias.ptr;
    a.y = const_cast<void *>(d.y.ptr);
    a.ldx = d.x.row_stride;
    a.ldy = d.y.row_stride;
    a.M = (int)d.x.rows;
    a.D = (int)d.x.cols;
    a.eps = (float)d.eps;
    a.d = (float)a.D;
    a.mean = (float *)const_cast<void *>(d.mean.ptr);
    a.rstd = (float *)const_cast<void *>(d.rstd.ptr);
    a.scale = (float *)const_cast<void *>(d.scale.ptr);
    const bool q8 = d.y.dtype == DENSE_INT8;
    hipStream_t s = (hipStream_t)stream;
    if (d.x.dtype == DENSE_BF16)
        q8 ? launch_norm<bf16, true>(a, s) : launch_norm<bf16, false>(a, s);
    else if (d.x.dtype == DENSE_FP16)
        q8 ? launch_norm<f16, true>(a, s) : launch_norm<f16, false>(a, s);
    else
        q8 ? launch_norm<float, true>(a, s) : launch_norm<float, false>(a, s);
    return hipGetLastError() == hipSuccess ? CONV_I8_OK : CONV_I8_ERR_HIP;
}

conv_i8_status_t dense_layer_norm_backward_workspace_size(const dense_layer_norm_backward_t *args, size_t *bytes)
{
    if (!bytes)
        return CONV_I8_ERR_NULL;
    BackPlan p;
    DENSE_TRY(analyze(args, &p));
    *bytes = (size_t)p.ws_bytes;
    return CONV_I8_OK;
}

conv_i8_status_t dense_layer_norm_backward(const dense_layer_norm_backward_t *args, void *workspace, size_t bytes,
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
    NormBackArgs a;
    memset(&a, 0, sizeof a);
    a.dy = p.d.dy.ptr;
    a.x = p.d.x.ptr;
    a.weight = p.d.weight.ptr;
    a.mean = (const float *)p.d.mean.ptr;
    a.rstd = (const float *)p.d.rstd.ptr;
    a.dx = const_cast<void *>(p.d.dx.ptr);
    a.lddy = p.d.dy.row_stride;
    a.ldx = p.d.x.row_stride;
    a.lddx = p.d.dx.row_stride;
    a.M = (int)p.M;
    a.D = (int)p.D;
    a.d = (float)a.D;
    a.part = p.sums && !p.once ? (float *)workspace : nullptr;
    a.part_ld = p.part_ld;
    if (p.once) {
        a.dweight = const_cast<void *>(p.d.dweight.ptr);
        a.dbias = const_cast<void *>(p.d.dbias.ptr);
    }
    hipStream_t s = (hipStream_t)stream;
    const int64_t dt = p.d.x.dtype;
    if (p.M > 0) {
        if (dt == DENSE_BF16)
            launch_back<bf16>(a, p.wgs, s);
        else if (dt == DENSE_FP16)
            launch_back<f16>(a, p.wgs, s);
        else
            launch_back<float>(a, p.wgs, s);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    if (p.sums && !p.once) {
        ColSumArgs c;
        memset(&c, 0, sizeof c);
        c.part = a.part;
        c.ld = 2 * p.part_ld;
        c.rows = p.M > 0 ? p.wgs : 0;  // none: zeros
        c.cols = 2 * p.part_ld;
        c.split = p.part_ld;
        c.valid = p.D;
        c.out0 = const_cast<void *>(p.d.dweight.ptr);
        c.out1 = const_cast<void *>(p.d.dbias.ptr);
        c.dt = (int)dt;
        hipLaunchKernelGGL(colsum_kernel<>, colsum_grid(c.cols), dim3(32 * kSumGroups), 0, s, c);
        if (hipGetLastError() != hipSuccess)
            return CONV_I8_ERR_HIP;
    }
    return CONV_I8_OK;
}

}  // extern "C"
