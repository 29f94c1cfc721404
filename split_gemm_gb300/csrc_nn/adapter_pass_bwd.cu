// Instantiates the adapters' backward pass over tiles.
#include "conv2d.h"
#include "adapter_pass.cuh"

namespace sgb {
namespace ad {

int launch_pass_bwd(const PassParams& p, int32_t base_dtype, int32_t out_dtype, bool vec, bool halved, cudaStream_t stream)
{
    return start_pass<true>(p, base_dtype, out_dtype, vec, halved, stream);
}

}  // namespace ad
}  // namespace sgb
