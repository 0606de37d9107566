// The launches of the norm fused with a residual connection, one source file per
// element type.
#pragma once

#include "host_common.hpp"
#include "residual_norm_kernel.hpp"

namespace dense {

// Longest rows that stay in registers, forward and backward.
constexpr int64_t kRow = 16384, kBackRow = 8192;
inline bool back_in_registers(int64_t D) { return D >= 8 && D <= kBackRow; }
// Threads that share a row of the gradients' kernel (us, BF16, both norms and a gate for all rows: 16384x1024
// by 64 threads 58, by 256 72; 16384x2048 by 256 86, by 512 127; 16384x4096 by 256 187, by 512 152).
constexpr int back_threads(int64_t D) { return D <= 1024 ? 64 : D <= 2048 ? 256 : 512; }

void launch_residual_norm_bf16(const ResNormArgs &a, bool rms, bool q8, hipStream_t s);
void launch_residual_norm_backward_bf16(const ResNormBackArgs &a, bool rms, bool post, int wgs, hipStream_t s);
void launch_residual_norm_f16(const ResNormArgs &a, bool rms, bool q8, hipStream_t s);
void launch_residual_norm_backward_f16(const ResNormBackArgs &a, bool rms, bool post, int wgs, hipStream_t s);
void launch_residual_norm_f32(const ResNormArgs &a, bool rms, bool q8, hipStream_t s);
void launch_residual_norm_backward_f32(const ResNormBackArgs &a, bool rms, bool post, int wgs, hipStream_t s);

inline unsigned capped(int64_t wgs, int threads)
{
    const int64_t most = threads <= 256 ? 1 << 21 : 1 << 16;
    return (unsigned)(wgs < most ? wgs : most);
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

// Two rows or more for each thread group, as layer norm's kernel takes them.  16384 x
// 4096 BF16 with both norms and a gate: 108 to 118 us with 256 threads for a row, by where its
// memory lies (537 MB, 4.6 to 5.0 TB/s), 132 with 512, which wait twice as long at its four reductions.
template <typename T, bool RMS, bool Q8>
void launch(const ResNormArgs &a, hipStream_t s)
{
    const int D = a.D;
    // a wave per row while that gives each CU two waves, else a workgroup per row (us, BF16, rms, r and y:
    // 256x1024 3.3 and 3.1, 900x1024 3.6 and 4.6, 16384x1024 24.0 and 29.8)
    const bool few = a.M < 2 * kCUs;
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
        launch_rows<T, RMS, Q8, 256, 2>(a, s);
    else if (D <= 8192)
        launch_rows<T, RMS, Q8, 512, 2>(a, s);
    else
        launch_rows<T, RMS, Q8, 1024, 2>(a, s);
}

template <typename T>
void launch_residual_norm(const ResNormArgs &a, bool rms, bool q8, hipStream_t s)
{
    if (rms)
        q8 ? launch<T, true, true>(a, s) : launch<T, true, false>(a, s);
    else
        q8 ? launch<T, false, true>(a, s) : launch<T, false, false>(a, s);
}

template <typename T, bool RMS, bool POST, int P, int V, bool AHEAD, int OCC>
void launch_back_rows(const ResNormBackArgs &a, int wgs, hipStream_t s)
{
    const dim3 grid((unsigned)wgs), block(norm_threads(P));
    if (a.D % 8 == 0)
        hipLaunchKernelGGL((residual_norm_backward_kernel<T, P, V, AHEAD, OCC, false, RMS, POST>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((residual_norm_backward_kernel<T, P, V, AHEAD, OCC, true, RMS, POST>), grid, block, 0, s, a);
}

template <typename T, bool RMS, bool POST>
void launch_back(const ResNormBackArgs &a, int wgs, hipStream_t s)
{
    if (!back_in_registers(a.D)) {
        if (a.D < 8)
            hipLaunchKernelGGL((residual_norm_backward_any_kernel<T, 64, RMS, POST>), dim3(capped(a.M, 64)), dim3(64), 0, s, a);
        else
            hipLaunchKernelGGL((residual_norm_backward_any_kernel<T, 1024, RMS, POST>), dim3(capped(a.M, 1024)), dim3(1024), 0, s, a);
        if (a.row_sums)
            hipLaunchKernelGGL((residual_norm_columns_kernel<T, RMS, POST>), dim3((unsigned)ceil_div(a.D, 2048), (unsigned)wgs),
                               dim3(256), 0, s, a);
    } else if (a.D <= 512) {
        launch_back_rows<T, RMS, POST, 64, 1, true, 2>(a, wgs, s);
    } else if (a.D <= 1024) {
        launch_back_rows<T, RMS, POST, 64, 2, true, 1>(a, wgs, s);
    } else if (a.D <= 2048) {
        launch_back_rows<T, RMS, POST, 256, 1, true, 2>(a, wgs, s);
    } else if (a.D <= 4096) {
        launch_back_rows<T, RMS, POST, 512, 1, true, 2>(a, wgs, s);
    } else {
        // FP32 with a norm of h spills 30 (rms) to 86 registers (4096x8192: 207 us as rms, 251 as layer norm, 805 MB)
        launch_back_rows<T, RMS, POST, 512, 2, (sizeof(T) == 2 && !POST), 2>(a, wgs, s);
    }
}

template <typename T>
void launch_residual_norm_backward(const ResNormBackArgs &a, bool rms, bool post, int wgs, hipStream_t s)
{
    if (rms)
        post ? launch_back<T, true, true>(a, wgs, s) : launch_back<T, true, false>(a, wgs, s);
    else
        post ? launch_back<T, false, true>(a, wgs, s) : launch_back<T, false, false>(a, wgs, s);
}

}  // namespace dense
