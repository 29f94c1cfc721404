// Instantiates the forward kernels that hold their row in registers.
#include "ln_rows.cuh"

namespace sgb {
namespace ln {

template <typename TX, typename TY, int VEC, int E, int G>
void start_fwd(const FwdParams& p, cudaStream_t stream)
{
    constexpr int T = block_threads(G), R = T / G;
    const int64_t rows = std::is_same_v<TY, void> ? p.padded_rows : p.rows;
    const int64_t blocks = mx::cdiv<int64_t>(rows, R), most = SMS * fwd_resident({G, E});
    fwd_rows<TX, TY, VEC, E, G><<<static_cast<unsigned>(blocks < most ? blocks : most), T, 0, stream>>>(
        static_cast<const TX*>(p.x), static_cast<TY*>(p.y), p);
}

template <typename TX, typename TY, int VEC>
bool fwd_by_shape(const FwdParams& p, cudaStream_t stream)
{
    // a quantised row needs the 128 columns of a scale tile in one vector of its group, single elements a whole warp
    constexpr bool MX = std::is_same_v<TY, void>;
    constexpr int LEAST = !MX ? 8 : VEC == 8 ? 16 : 32;
    const RowShape s = row_shape(p.cols);
    switch (s.threads * 100 + s.elems) {
        case 808: if constexpr (LEAST <= 8) { start_fwd<TX, TY, VEC, 8, 8>(p, stream); return true; } [[fallthrough]];
        case 1608: if constexpr (LEAST <= 16) { start_fwd<TX, TY, VEC, 8, 16>(p, stream); return true; } [[fallthrough]];
        case 3208: start_fwd<TX, TY, VEC, 8, 32>(p, stream); return true;
        case 3216: start_fwd<TX, TY, VEC, 16, 32>(p, stream); return true;
        case 12808: start_fwd<TX, TY, VEC, 8, 128>(p, stream); return true;
        case 25608: start_fwd<TX, TY, VEC, 8, 256>(p, stream); return true;
        case 25616: start_fwd<TX, TY, VEC, 16, 256>(p, stream); return true;
        case 51216: start_fwd<TX, TY, VEC, 16, 512>(p, stream); return true;
        case 102416: start_fwd<TX, TY, VEC, 16, 1024>(p, stream); return true;
        default: return false;
    }
}

template <typename TX, typename TY>
bool launch_fwd_rows(const FwdParams& p, bool vec, cudaStream_t stream)
{
    return vec ? fwd_by_shape<TX, TY, 16 / sizeof(TX)>(p, stream) : fwd_by_shape<TX, TY, 1>(p, stream);
}

#define SGB_FWD(TX, TY) template bool launch_fwd_rows<TX, TY>(const FwdParams&, bool, cudaStream_t);
SGB_FWD(float, float)
SGB_FWD(float, __nv_bfloat16)
SGB_FWD(__nv_bfloat16, float)
SGB_FWD(__nv_bfloat16, __nv_bfloat16)
SGB_FWD(float, void)
SGB_FWD(__nv_bfloat16, void)

}  // namespace ln
}  // namespace sgb
