// The instances of the norm fused with a residual connection for one element type.
#include "residual_norm_launch.hpp"

namespace dense {

void launch_residual_norm_f32(const ResNormArgs &a, bool rms, bool q8, hipStream_t s)
{
    launch_residual_norm<float>(a, rms, q8, s);
}

void launch_residual_norm_backward_f32(const ResNormBackArgs &a, bool rms, bool post, int wgs, hipStream_t s)
{
    launch_residual_norm_backward<float>(a, rms, post, wgs, s);
}

}  // namespace dense
