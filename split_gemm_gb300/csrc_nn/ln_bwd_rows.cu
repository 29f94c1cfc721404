// Instantiates the backward kernels that hold their row in registers.
#include "ln_rows.cuh"

namespace sgb {
namespace ln {

template <typename TX, typename TY, int VEC, int E, int G>
void start_bwd(const BwdParams& p, int grid, cudaStream_t stream)
{
    bwd_rows<TX, TY, VEC, E, G><<<static_cast<unsigned>(grid), block_threads(G), 0, stream>>>(
        static_cast<const TY*>(p.dy), static_cast<const TX*>(p.x), static_cast<TX*>(p.dx), p);
}

template <typename TX, typename TY, int VEC>
bool bwd_by_shape(const BwdParams& p, int grid, cudaStream_t stream)
{
    const RowShape s = row_shape(p.cols);
    switch (s.threads * 100 + s.elems) {
        case 808: start_bwd<TX, TY, VEC, 8, 8>(p, grid, stream); return true;
        case 1608: start_bwd<TX, TY, VEC, 8, 16>(p, grid, stream); return true;
        case 3208: start_bwd<TX, TY, VEC, 8, 32>(p, grid, stream); return true;
        case 3216: start_bwd<TX, TY, VEC, 16, 32>(p, grid, stream); return true;
        case 12808: start_bwd<TX, TY, VEC, 8, 128>(p, grid, stream); return true;
        case 25608: start_bwd<TX, TY, VEC, 8, 256>(p, grid, stream); return true;
        case 25616: start_bwd<TX, TY, VEC, 16, 256>(p, grid, stream); return true;
        case 51216: start_bwd<TX, TY, VEC, 16, 512>(p, grid, stream); return true;
        default: return false;
    }
}

template <typename TX, typename TY>
bool launch_bwd_rows(const BwdParams& p, bool vec, int grid, cudaStream_t stream)
{
    return vec ? bwd_by_shape<TX, TY, 16 / sizeof(TX)>(p, grid, stream) : bwd_by_shape<TX, TY, 1>(p, grid, stream);
}

#define SGB_BWD(TX, TY) template bool launch_bwd_rows<TX, TY>(const BwdParams&, bool, int, cudaStream_t);
SGB_BWD(float, float)
SGB_BWD(float, __nv_bfloat16)
SGB_BWD(__nv_bfloat16, float)
SGB_BWD(__nv_bfloat16, __nv_bfloat16)

}  // namespace ln
}  // namespace sgb
