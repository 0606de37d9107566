// The product kernel's instances for 8-bit floating point: the first operand e4m3
// or e5m2, the second e4m3, both in rows form.
#include "gemm_launch.hpp"

namespace dense {

bool launch_gemm_f8e4(int tile, const GemmArgs &g, int splits, hipStream_t stream)
{
    return launch_gemm_form<f8e4, false, false>(tile, g, splits, stream);
}

bool launch_gemm_f8e5(int tile, const GemmArgs &g, int splits, hipStream_t stream)
{
    return launch_gemm_form<f8e5, false, false>(tile, g, splits, stream);
}

bool launch_gemm_pair_f8e4(const PairArgs &p, hipStream_t stream) { return launch_gemm_pair_f8<f8e4>(p, stream); }
bool launch_gemm_pair_f8e5(const PairArgs &p, hipStream_t stream) { return launch_gemm_pair_f8<f8e5>(p, stream); }

}  // namespace dense
