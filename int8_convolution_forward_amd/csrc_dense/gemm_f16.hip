// The product kernel's instances for one element type.
#include "gemm_launch.hpp"

namespace dense {

bool launch_gemm_f16(int tile, bool a_cols, bool b_cols, const GemmArgs &g, int splits, hipStream_t stream)
{
    return launch_gemm<f16>(tile, a_cols, b_cols, g, splits, stream);
}

bool launch_gemm_pair_f16(const PairArgs &p, hipStream_t stream) { return launch_gemm_pair<f16>(p, stream); }

}  // namespace dense
