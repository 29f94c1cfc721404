// The product of two microscaled 4-bit matrices: host side and kernels.
#include "mxfp4.h"

#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>

#include "mx_pair.cuh"

namespace sgb {
namespace mx {

std::once_flag encode_once;
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled = nullptr;

bool load_encoder()
{
    std::call_once(encode_once, [] {
        cudaDriverEntryPointQueryResult q{};
        void* fn = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode_tiled = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return encode_tiled != nullptr;
}

// Map of an operand's data: boxes of 128 bytes (256 elements) x box_rows rows, 128-byte swizzle; what lies
// beyond the matrix reads as zero.
bool encode(CUtensorMap* map, const void* data, int64_t rows, int64_t blocks, int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(blocks * 16), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(blocks * 16)};
    const cuuint32_t box[2] = {T_STAGE_BYTES_ROW, static_cast<cuuint32_t>(box_rows)}, steps[2] = {1, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dims, strides, box, steps,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Device status word of this library's product kernels, and what mxfp4_matmul_status last took out of it: read and cleared in
// one step, so that no report falls between the two.
__device__ uint32_t product_status, taken_status;

__global__ void take_status() { taken_status = atomicExch(&product_status, 0u); }

std::mutex asking;  // taken_status is one question's at a time

struct Operand {
    const void* data;
    const void* scales;
    int64_t rows;
};

// How the sum of `tiles` tiles is split: over clusters of 1, 2, 4 or 8 CTAs, of which the SMs hold 152, 76, 36 and 15 at
// once (one CTA to an SM).  A wave costs some 3 us of start and end, 0.7 us more where partial tiles are joined, and each stage its
// bytes at 55 bytes a clock, what an SM takes from L2.
struct Split {
    int splits;
    double us;
};

Split best_split(int64_t tiles, int stages, int bn)
{
    constexpr int held[4] = {152, 76, 36, 15};
    Split best{1, 1e30};
    for (int i = 0; i < 4; ++i) {
        const int s = 1 << i;
        if (s > stages) break;
        const double us = static_cast<double>(cdiv<int64_t>(tiles, held[i])) *
                          (3.0 + (s > 1 ? 0.7 : 0.0) + cdiv(stages, s) * (128.0 + bn + 16.0) * 128.0 / (55.0 * 1900.0));
        if (us < best.us) best = {s, us};
    }
    return best;
}

template <int BN, bool SWAP, typename T>
int launch_tile(const Operand& P, const Operand& Q, TileParams& k, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    using C = TileConfig<BN, SWAP>;
    CUtensorMap tm_p, tm_q;
    if (!encode(&tm_p, P.data, P.rows, k.blocks, T_ROWS) || !encode(&tm_q, Q.data, Q.rows, k.blocks, BN)) return CONV2D_ERR_CUDA;
    if (!allow_smem(tile_kernel<BN, SWAP, T>, C::SMEM, done)) return CONV2D_ERR_CUDA;
    k.q_tiles = cdiv(k.q_rows, BN);
    const int64_t tiles = cdiv<int64_t>(k.p_rows, T_ROWS) * k.q_tiles;
    k.splits = best_split(tiles, k.stages, BN).splits;
    if (tiles * k.splits > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    return launch(tile_kernel<BN, SWAP, T>, tiles * k.splits, T_THREADS, C::SMEM, stream, k.splits, tm_p, tm_q, k) == cudaSuccess ? CONV2D_OK
                                                                                                                           : CONV2D_ERR_CUDA;
}

// Map of an operand's scales: tiles of 128 words, `tiles` of them to a row of tiles; boxes of 2 x box_rows tiles.
bool encode_scales(CUtensorMap* map, const void* scales, int64_t rows, int btiles, int box_rows)
{
    const cuuint64_t dims[3] = {TILE_BYTES / 4, static_cast<cuuint64_t>(btiles), static_cast<cuuint64_t>(cdiv<int64_t>(rows, TILE_ROWS))};
    const cuuint64_t strides[2] = {TILE_BYTES, static_cast<cuuint64_t>(btiles) * TILE_BYTES};
    const cuuint32_t box[3] = {TILE_BYTES / 4, 2, static_cast<cuuint32_t>(box_rows)}, steps[3] = {1, 1, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(scales), dims, strides, box, steps,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of y [m][n] for stores of 32 rows x 128 bytes.
bool encode_y(CUtensorMap* map, void* y, int64_t m, int64_t n, int elem)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(n * elem)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), 32}, steps[2] = {1, 1};
    return encode_tiled(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims, strides, box,
                        steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
int launch_pair(const Operand& a, const Operand& b, const TileParams& k, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    PairParams p{};
    p.bias = k.bias;
    p.y = k.y;
    p.status = k.status;
    p.ldy = k.ldy;
    p.m = static_cast<int>(a.rows);
    p.n = static_cast<int>(b.rows);
    p.stages = k.stages;
    p.m_tiles = cdiv(p.m, W_TILE);
    p.n_tiles = cdiv(p.n, W_TILE);
    p.relu = k.relu;
    p.tma_store = b.rows * sizeof(T) % 16 == 0;
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    if (tiles > INT32_MAX - SMS) return CONV2D_ERR_UNSUPPORTED;
    CUtensorMap tm_a, tm_b, tm_sa, tm_sb, tm_y{};
    if (!encode(&tm_a, a.data, a.rows, k.blocks, W_ROWS) || !encode(&tm_b, b.data, b.rows, k.blocks, W_ROWS) ||
        !encode_scales(&tm_sa, a.scales, a.rows, k.btiles, 1) || !encode_scales(&tm_sb, b.scales, b.rows, k.btiles, 2) ||
        (p.tma_store && !encode_y(&tm_y, k.y, a.rows, b.rows, sizeof(T))))
        return CONV2D_ERR_CUDA;
    if (!allow_smem(pair_kernel<T>, W_SMEM, done)) return CONV2D_ERR_CUDA;
    const int64_t grid = 2 * (tiles < SMS / 2 ? tiles : SMS / 2);
    return launch(pair_kernel<T>, grid, W_THREADS, W_SMEM, stream, 2, tm_a, tm_b, tm_sa, tm_sb, tm_y, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

template <typename T>
int product(const Operand& a, const Operand& b, TileParams& k, cudaStream_t stream)
{
    // Up to 128 rows of y: the weight's rows in the accumulator's lanes, y's rows in
    // its columns, as few as cover them.
    const bool swap = a.rows <= 128;
    // 256 x 256 tiles where they fill half of the SM pairs (bf16 y; 32 tiles, 512 x 4096 x 4096: pairs 10.4 us, single CTAs 9.6;
    // 40 tiles, 1280 x 2048 x 1024: 6.9 and 10.9; 64 tiles, 1024 x 4096 x 4096: 10.7 and 18.5).
    if (!swap && cdiv<int64_t>(a.rows, W_TILE) * cdiv<int64_t>(b.rows, W_TILE) * 4 >= SMS) return launch_pair<T>(a, b, k, stream);
    const Operand &P = swap ? b : a, &Q = swap ? a : b;
    k.p_scales = static_cast<const uint8_t*>(P.scales);
    k.q_scales = static_cast<const uint8_t*>(Q.scales);
    k.p_rows = static_cast<int>(P.rows);
    k.q_rows = static_cast<int>(Q.rows);
    int bn = Q.rows <= 16 ? 16 : Q.rows <= 32 ? 32 : Q.rows <= 64 ? 64 : 128;
    if (bn == 128) {  // narrower tiles where more SMs are worth more than reading P twice
        const int64_t p_tiles = cdiv<int64_t>(P.rows, T_ROWS);
        if (best_split(p_tiles * cdiv<int64_t>(Q.rows, 64), k.stages, 64).us < best_split(p_tiles * cdiv<int64_t>(Q.rows, 128), k.stages, 128).us) bn = 64;
    }
    if (swap) {
        switch (bn) {
            case 16: return launch_tile<16, true, T>(P, Q, k, stream);
            case 32: return launch_tile<32, true, T>(P, Q, k, stream);
            case 64: return launch_tile<64, true, T>(P, Q, k, stream);
            default: return launch_tile<128, true, T>(P, Q, k, stream);
        }
    }
    switch (bn) {
        case 16: return launch_tile<16, false, T>(P, Q, k, stream);
        case 32: return launch_tile<32, false, T>(P, Q, k, stream);
        case 64: return launch_tile<64, false, T>(P, Q, k, stream);
        default: return launch_tile<128, false, T>(P, Q, k, stream);
    }
}

}  // namespace mx
}  // namespace sgb

using namespace sgb;

extern "C" int mxfp4_matmul(const mxfp4_matmul_params* params, const void* a_data_dev, const void* a_scales_dev,
                            const void* b_data_dev, const void* b_scales_dev, const float* bias_dev, void* y_dev,
                            const conv2d_epilogue* epi, conv2d_stream_t stream)
{
    constexpr int64_t most = (int64_t(1) << 31) - 1;
    if (!params || params->m < 0 || params->n < 0 || params->k < 1) return CONV2D_ERR_INVALID;
    if (params->m > most || params->n > most || params->k > most) return CONV2D_ERR_UNSUPPORTED;
    const int act = epi ? epi->activation : CONV2D_ACT_NONE, out = epi ? epi->out_dtype : CONV2D_OUT_F32;
    if ((act != CONV2D_ACT_NONE && act != CONV2D_ACT_RELU) || (out != CONV2D_OUT_F32 && out != CONV2D_OUT_BF16))
        return CONV2D_ERR_INVALID;
    if (params->m == 0 || params->n == 0) return CONV2D_OK;
    if (!a_data_dev || !a_scales_dev || !b_data_dev || !b_scales_dev || !y_dev) return CONV2D_ERR_INVALID;
    for (const void* p : {a_data_dev, a_scales_dev, b_data_dev, b_scales_dev, static_cast<const void*>(y_dev)})
        if (reinterpret_cast<uintptr_t>(p) % 16) return CONV2D_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(bias_dev) % 4) return CONV2D_ERR_ALIGNMENT;
    if (!mx::load_encoder()) return CONV2D_ERR_CUDA;
    mx::TileParams k{};
    k.blocks = static_cast<int>(mx::cdiv<int64_t>(params->k, mx::BLOCK));
    k.btiles = mx::cdiv(k.blocks, mx::TILE_BLOCKS);
    k.stages = mx::cdiv(k.blocks, mx::T_STAGE_BLOCKS);
    k.bias = bias_dev;
    k.relu = act == CONV2D_ACT_RELU;
    k.y = y_dev;
    k.ldy = params->n;
    k.vec_y = params->n % 4 == 0;
    void* status = nullptr;
    if (cudaGetSymbolAddress(&status, mx::product_status) != cudaSuccess) return CONV2D_ERR_CUDA;
    k.status = static_cast<uint32_t*>(status);
    const mx::Operand a{a_data_dev, a_scales_dev, params->m}, b{b_data_dev, b_scales_dev, params->n};
    return out == CONV2D_OUT_BF16 ? mx::product<__nv_bfloat16>(a, b, k, stream) : mx::product<float>(a, b, k, stream);
}

extern "C" int mxfp4_matmul_status(conv2d_stream_t stream)
{
    uint32_t word = 0;
    std::lock_guard<std::mutex> one(mx::asking);
    mx::take_status<<<1, 1, 0, stream>>>();
    if (cudaGetLastError() != cudaSuccess) return CONV2D_ERR_CUDA;
    if (cudaMemcpyFromSymbolAsync(&word, mx::taken_status, sizeof word, 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return CONV2D_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return CONV2D_ERR_CUDA;
    return word == 0 ? CONV2D_OK : CONV2D_ERR_TIMEOUT;
}
