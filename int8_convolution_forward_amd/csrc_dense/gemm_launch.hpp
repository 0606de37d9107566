// The tiles of the product kernel and its launch, one source file per element
// type.
#pragma once

#include "gemm_kernel.hpp"

namespace dense {

struct Tile {
    int tm, tn;
    int occ;          // workgroups per CU
    bool deep;        // for at most one workgroup per CU
    const char *name;
};

constexpr int kTiles = 4;
// 128x128d: five ring slots and a CU to itself, for products of few workgroups
// (2048^3 BF16: 19.9 us, with two slots and two workgroups a CU 25.1).
constexpr Tile kTile[kTiles] = {
    {256, 256, 1, false, "256x256"},
    {128, 128, 2, false, "128x128"},
    {64, 64, 3, false, "64x64"},
    {128, 128, 1, true, "128x128d"},
};

// One launch of tile `tile` with the operands in rows or columns form (INT8:
// rows only); false if the combination does not exist or the launch failed.
bool launch_gemm_bf16(int tile, bool a_cols, bool b_cols, const GemmArgs &g, int splits, hipStream_t stream);
bool launch_gemm_f16(int tile, bool a_cols, bool b_cols, const GemmArgs &g, int splits, hipStream_t stream);
bool launch_gemm_f8e4(int tile, const GemmArgs &g, int splits, hipStream_t stream);  // the first operand's type
bool launch_gemm_f8e5(int tile, const GemmArgs &g, int splits, hipStream_t stream);
bool launch_gemm_i8(int tile, bool a_cols, bool b_cols, const GemmArgs &g, int splits, hipStream_t stream);

// Both gradients' products with tile kPairTile, unsplit, and the bias gradient's
// last step, in one launch.
constexpr int kPairTile = 2;
bool launch_gemm_pair_bf16(const PairArgs &p, hipStream_t stream);
bool launch_gemm_pair_f16(const PairArgs &p, hipStream_t stream);

template <typename T>
bool launch_gemm_pair(const PairArgs &p, hipStream_t stream)
{
    const int sums = (int)(p.sum.cols + 256 / kSumGroups - 1) / (256 / kSumGroups);
    const dim3 grid((unsigned)(p.dx.tiles + p.dw.tiles + sums)), block(256);
    hipLaunchKernelGGL((gemm_pair_kernel<T, 64, 64, 2, 2, 3, 3, 4, 3>), grid, block, 0, stream, p);
    return hipGetLastError() == hipSuccess;
}

bool launch_gemm_pair_f8e4(const PairArgs &p, hipStream_t stream);
bool launch_gemm_pair_f8e5(const PairArgs &p, hipStream_t stream);

template <typename T>
bool launch_gemm_pair_f8(const PairArgs &p, hipStream_t stream)
{
    const int sums = (int)(p.sum.cols + 256 / kSumGroups - 1) / (256 / kSumGroups);
    const dim3 grid((unsigned)(p.dx.tiles + p.dw.tiles + sums)), block(256);
    hipLaunchKernelGGL((gemm_pair_f8_kernel<T, 64, 64, 2, 2, 3, 3, 4, 3>), grid, block, 0, stream, p);
    return hipGetLastError() == hipSuccess;
}

template <typename T, bool ASTR, bool BSTR>
bool launch_gemm_form(int tile, const GemmArgs &g, int splits, hipStream_t stream)
{
    const dim3 grid((unsigned)g.tiles, (unsigned)splits), block(256);
    switch (tile) {
    case 0: hipLaunchKernelGGL((gemm_kernel<T, 256, 256, 2, 2, 3, 2, 7, 1, ASTR, BSTR>), grid, block, 0, stream, g); break;
    case 1: hipLaunchKernelGGL((gemm_kernel<T, 128, 128, 2, 2, 2, 2, 6, 2, ASTR, BSTR>), grid, block, 0, stream, g); break;
    case 2: hipLaunchKernelGGL((gemm_kernel<T, 64, 64, 2, 2, 3, 3, 4, 3, ASTR, BSTR>), grid, block, 0, stream, g); break;
    case 3: hipLaunchKernelGGL((gemm_kernel<T, 128, 128, 2, 2, 5, 5, 6, 1, ASTR, BSTR>), grid, block, 0, stream, g); break;
    default: return false;
    }
    return hipGetLastError() == hipSuccess;
}

template <typename T>
bool launch_gemm(int tile, bool a_cols, bool b_cols, const GemmArgs &g, int splits, hipStream_t stream)
{
    if constexpr (sizeof(T) == 2) {
        if (a_cols && b_cols)
            return launch_gemm_form<T, true, true>(tile, g, splits, stream);
        if (!a_cols && b_cols)
            return launch_gemm_form<T, false, true>(tile, g, splits, stream);
    }
    if (a_cols || b_cols)
        return false;
    return launch_gemm_form<T, false, false>(tile, g, splits, stream);
}

}  // namespace dense
