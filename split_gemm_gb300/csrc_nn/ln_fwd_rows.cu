// Instantiates the forward kernels that hold their row in registers.
#include "conv2d.h"
#include "ln_rows.cuh"

namespace sgb {
namespace ln {

template <typename TX, typename TY, int VEC, int E, int G, int MOST, bool WHOLE>
int start_fwd_as(const FwdParams& p, RowShape s, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    constexpr int V = VEC == 1 ? 8 : VEC;
    constexpr int per_thread = VEC > 1 ? Ring<TX, V, E / V, ring_depth(RowShape{G ? G : MOST, E, MOST}, sizeof(TX), 0), WHOLE>::THREAD_BYTES : 0;
    const auto kernel = fwd_rows<TX, TY, VEC, E, G, MOST, WHOLE>;
    if (!mx::allow_smem(kernel, per_thread * MOST, done)) return CONV2D_ERR_CUDA;
    const int64_t grid = row_blocks(std::is_same_v<TY, void> ? p.padded_rows : p.rows, s, fwd_resident(s));
    const int threads = block_threads(s);
    return mx::launch(kernel, grid, threads, per_thread * threads, stream, 1, static_cast<const TX*>(p.x), static_cast<TY*>(p.y), p) == cudaSuccess
               ? CONV2D_OK
               : CONV2D_ERR_CUDA;
}

template <typename TX, typename TY, int VEC, int E, int G, int MOST>
int start_fwd(const FwdParams& p, RowShape s, cudaStream_t stream)
{
    if (G) s = RowShape{G, E, MOST};
    if constexpr (VEC > 1)
        if (p.span == p.cols) return start_fwd_as<TX, TY, VEC, E, G, MOST, true>(p, s, stream);
    return start_fwd_as<TX, TY, VEC, E, G, MOST, false>(p, s, stream);
}

template <typename TX, typename TY, int VEC>
int fwd_by_shape(const FwdParams& p, cudaStream_t stream)
{
    // a quantised row needs a block's 32 columns in one vector of its group, and its group over whole scale tiles
    constexpr bool MX = std::is_same_v<TY, void>;
    constexpr int LEAST = !MX ? 4 : VEC > 1 ? 16 : 32;
    constexpr bool B16 = sizeof(TX) == 2;  // shapes of many elements to a thread are for 16-bit rows
    RowShape s = fwd_shape(p.rows, p.span, sizeof(TX), VEC > 1 && p.span == p.cols);
    if (s.threads == 0) return CONV2D_ERR_UNSUPPORTED;
    if (s.threads < LEAST) s = RowShape{LEAST, 8, 256};
    if constexpr (LEAST <= 4 && B16)
        if (s.threads == 4) return start_fwd<TX, TY, VEC, 16, 4, 256>(p, s, stream);
    if constexpr (LEAST <= 8 && B16)
        if (s.threads == 8 && s.elems == 16) return start_fwd<TX, TY, VEC, 16, 8, 256>(p, s, stream);
    if constexpr (LEAST <= 8)
        if (s.threads == 8) return start_fwd<TX, TY, VEC, 8, 8, 256>(p, s, stream);
    if constexpr (LEAST <= 16 && B16)
        if (s.threads == 16 && s.elems == 16) return start_fwd<TX, TY, VEC, 16, 16, 256>(p, s, stream);
    if constexpr (LEAST <= 16)
        if (s.threads == 16) return start_fwd<TX, TY, VEC, 8, 16, 256>(p, s, stream);
    if constexpr (B16 && VEC > 1)
        if (s.threads == 32 && s.elems == 32 && s.most == 256) return start_fwd_as<TX, TY, VEC, 32, 32, 256, true>(p, s, stream);
    if (s.threads == 32 && s.most == 256)
        return s.elems == 8 ? start_fwd<TX, TY, VEC, 8, 32, 256>(p, s, stream) : start_fwd<TX, TY, VEC, 16, 32, 256>(p, s, stream);
    if (s.elems == 8) return start_fwd<TX, TY, VEC, 8, 0, 256>(p, s, stream);
    if (s.elems == 16 && s.most == 256) return start_fwd<TX, TY, VEC, 16, 0, 256>(p, s, stream);
    if (s.elems == 16 && s.most == 384) return start_fwd_as<TX, TY, VEC, 16, 0, 384, false>(p, s, stream);
    if (s.elems == 16) return start_fwd_as<TX, TY, VEC, 16, 0, 512, false>(p, s, stream);
    return start_fwd<TX, TY, VEC, 32, 0, 512>(p, s, stream);
}

template <typename TX, typename TY>
int launch_fwd_rows(const FwdParams& p, bool vec, cudaStream_t stream)
{
    return vec ? fwd_by_shape<TX, TY, 16 / sizeof(TX)>(p, stream) : fwd_by_shape<TX, TY, 1>(p, stream);
}

#define SGB_FWD(TX, TY) template int launch_fwd_rows<TX, TY>(const FwdParams&, bool, cudaStream_t);
SGB_FWD(float, float)
SGB_FWD(float, __nv_bfloat16)
SGB_FWD(__nv_bfloat16, float)
SGB_FWD(__nv_bfloat16, __nv_bfloat16)
SGB_FWD(float, void)
SGB_FWD(__nv_bfloat16, void)

}  // namespace ln
}  // namespace sgb
