// The instances of the norm fused with a residual connection for one element type.
#include "residual_norm_launch.hpp"

namespace dense {

void launch_residual_norm_bf16(const ResNormArgs &a, bool rms, bool q8, hipStream_t s)
{
    launch_residual_norm<bf16>(a, rms, q8, s);
}

void launch_residual_norm_backward_bf16(const ResNormBackArgs &a, bool rms, bool post, int wgs, hipStream_t s)
{
    launch_residual_norm_backward<bf16>(a, rms, post, wgs, s);
}

}  // namespace dense
