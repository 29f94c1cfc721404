// Instantiates the adapters' forward pass over tiles.
#include "conv2d.h"
#include "adapter_pass.cuh"

namespace sgb {
namespace ad {

int launch_pass_fwd(const PassParams& p, int32_t base_dtype, int32_t out_dtype, bool vec, cudaStream_t stream)
{
    return vec ? start_pass_by_types<false, true>(p, base_dtype, out_dtype, stream) : start_pass_by_types<false, false>(p, base_dtype, out_dtype, stream);
}

}  // namespace ad
}  // namespace sgb
