// The product kernel's instances for one element type.
#include "gemm_launch.hpp"

namespace dense {

bool launch_gemm_bf16(int tile, bool a_cols, bool b_cols, const GemmArgs &g, int splits, hipStream_t stream)
{
    return launch_gemm<bf16>(tile, a_cols, b_cols, g, splits, stream);
}

bool launch_gemm_pair_bf16(const PairArgs &p, hipStream_t stream) { return launch_gemm_pair<bf16>(p, stream); }

}  // namespace dense
