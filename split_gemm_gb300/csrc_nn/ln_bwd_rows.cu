// Instantiates the backward kernels that hold their row in registers.
#include "conv2d.h"
#include "ln_rows.cuh"

namespace sgb {
namespace ln {

template <typename TX, typename TY, int VEC, int E, int G, int MOST, bool SUMS, bool WHOLE>
int start_bwd_as(const BwdParams& p, RowShape s, int grid, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    constexpr int DEPTH = ring_depth(RowShape{G ? G : MOST, E, MOST}, sizeof(TX), sizeof(TY)), V = VEC == 1 ? 8 : VEC;
    constexpr int ring = VEC > 1 ? Ring<TX, V, E / V, DEPTH, WHOLE>::THREAD_BYTES + Ring<TY, V, E / V, DEPTH, WHOLE>::THREAD_BYTES : 0;
    constexpr int join = G ? 2 * E * 4 : 0;  // a block's sums by row and column
    constexpr int per_thread = ring > join ? ring : join;
    const auto kernel = bwd_rows<TX, TY, VEC, E, G, MOST, SUMS, WHOLE>;
    if (!mx::allow_smem(kernel, per_thread * MOST, done)) return CONV2D_ERR_CUDA;
    const int threads = block_threads(s);
    return mx::launch(kernel, grid, threads, per_thread * threads, stream, 1, static_cast<const TY*>(p.dy), static_cast<const TX*>(p.x),
                      static_cast<TX*>(p.dx), p) == cudaSuccess
               ? CONV2D_OK
               : CONV2D_ERR_CUDA;
}

template <typename TX, typename TY, int VEC, int E, int G, int MOST, bool SUMS>
int start_bwd(const BwdParams& p, RowShape s, int grid, cudaStream_t stream)
{
    if constexpr (VEC > 1)
        if (p.span == p.cols) return start_bwd_as<TX, TY, VEC, E, G, MOST, SUMS, true>(p, s, grid, stream);
    return start_bwd_as<TX, TY, VEC, E, G, MOST, SUMS, false>(p, s, grid, stream);
}

template <typename TX, typename TY, int VEC>
int bwd_by_shape(const BwdParams& p, int grid, cudaStream_t stream)
{
    constexpr bool B16 = sizeof(TX) == 2;  // shapes of many elements to a thread are for 16-bit rows
    const RowShape s = bwd_shape(p.rows, p.span, sizeof(TX), p.span == p.cols);
    if (s.threads == 0) return CONV2D_ERR_UNSUPPORTED;
    if constexpr (B16) {
        if (s.threads == 4) return start_bwd<TX, TY, VEC, 16, 4, 256, true>(p, s, grid, stream);
        if (s.threads == 8 && s.elems == 16) return start_bwd<TX, TY, VEC, 16, 8, 256, true>(p, s, grid, stream);
        if (s.threads == 16 && s.elems == 16) return start_bwd<TX, TY, VEC, 16, 16, 256, true>(p, s, grid, stream);
    }
    if (s.threads == 8) return start_bwd<TX, TY, VEC, 8, 8, 256, true>(p, s, grid, stream);
    if (s.threads == 16) return start_bwd<TX, TY, VEC, 8, 16, 256, true>(p, s, grid, stream);
    if (s.threads == 32)
        return s.elems == 8 ? start_bwd<TX, TY, VEC, 8, 32, 256, true>(p, s, grid, stream) : start_bwd<TX, TY, VEC, 16, 32, 256, true>(p, s, grid, stream);
    if (s.elems == 8) return start_bwd<TX, TY, VEC, 8, 0, 256, true>(p, s, grid, stream);
    if (s.elems == 16)
        return s.most == 256 ? start_bwd<TX, TY, VEC, 16, 0, 256, true>(p, s, grid, stream) : start_bwd<TX, TY, VEC, 16, 0, 512, true>(p, s, grid, stream);
    // No registers are left for the sums: dx alone, in blocks of its own number.
    return start_bwd<TX, TY, VEC, 32, 0, 512, false>(p, s, static_cast<int>(row_blocks(p.rows, s, bwd_resident(s))), stream);
}

template <typename TX, typename TY>
int launch_bwd_rows(const BwdParams& p, bool vec, int grid, cudaStream_t stream)
{
    return vec ? bwd_by_shape<TX, TY, 16 / sizeof(TX)>(p, grid, stream) : bwd_by_shape<TX, TY, 1>(p, grid, stream);
}

#define SGB_BWD(TX, TY) template int launch_bwd_rows<TX, TY>(const BwdParams&, bool, int, cudaStream_t);
SGB_BWD(float, float)
SGB_BWD(float, __nv_bfloat16)
SGB_BWD(__nv_bfloat16, float)
SGB_BWD(__nv_bfloat16, __nv_bfloat16)

}  // namespace ln
}  // namespace sgb
