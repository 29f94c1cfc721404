// The norm's gradient with x as an 8-bit checkpoint (mxint8.h).
#include "mxint8.h"

#include "ln_any.cuh"
#include "ln_bwd8_rows.cuh"

namespace sgb {
namespace ln {

// dx, one block per row, the row read twice: the form for rows of any width and alignment.
template <typename TY>
__global__ void __launch_bounds__(THREADS) bwd8_dx_any(const TY* dy, const Checkpoint x, TY* dx, const BwdParams p)
{
    __shared__ float warp_sums[THREADS / 32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TY* dyr = dy + r * p.dy_stride;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x; c < p.cols; c += THREADS) {
            const float g = mx::to_float(dyr[c]) * (p.weight ? p.weight[c] : 1.f);
            s1 += g;
            s2 = fmaf(g, (x.at(r, c) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, warp_sums) * p.inv_cols;
        s2 = block_sum(s2, warp_sums) * p.inv_cols;
        for (int c = threadIdx.x; c < p.cols; c += THREADS) {
            const float g = mx::to_float(dyr[c]) * (p.weight ? p.weight[c] : 1.f);
            const float xh = (x.at(r, c) - mean) * rstd;
            mx::from_float(dx[r * p.cols + c], rstd * (g - s1 - xh * s2));
        }
    }
}

// Partial sums of dweight and dbias where registers do not hold them: a thread keeps VEC columns and takes every p.chunks-th row; rows of dy that do
// not start at 16 bytes are taken by single elements.
template <typename TY, int VEC>
__global__ void __launch_bounds__(THREADS) bwd8_part_any(const TY* __restrict__ dy, const Checkpoint x, const BwdParams p)
{
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x) * VEC;
    if (c >= p.cols) return;
    float dw[VEC] = {}, db[VEC] = {};
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < p.rows; r += p.chunks) {
        const float mean = __ldg(p.mean + r), rstd = __ldg(p.rstd + r);
        if constexpr (VEC == 8) {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(x.data + r * (x.blocks * mx::BLOCK) + c));
            const float f = mx::scale_value(__ldg(x.scales + r * x.blocks + c / mx::BLOCK));
            float2 v[4];
            mx::unpack_int8x4(reinterpret_cast<float2(&)[2]>(v[0]), q.x);
            mx::unpack_int8x4(reinterpret_cast<float2(&)[2]>(v[2]), q.y);
            Pack<TY, 8> g;
            const TY* from = dy + r * p.dy_stride + c;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(TY)) / 2; ++i) reinterpret_cast<uint4*>(&g)[i] = __ldg(reinterpret_cast<const uint4*>(from) + i);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float gi = mx::to_float(g.v[i]);
                dw[i] = fmaf(gi, (f * (i % 2 ? v[i / 2].y : v[i / 2].x) - mean) * rstd, dw[i]);
                db[i] += gi;
            }
        } else {
            const float g = mx::to_float(dy[r * p.dy_stride + c]);
            dw[0] = fmaf(g, (x.at(r, c) - mean) * rstd, dw[0]);
            db[0] += g;
        }
    }
    float* part = p.part + 2 * static_cast<int64_t>(blockIdx.y) * p.cols;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        part[c + i] = dw[i];
        part[p.cols + c + i] = db[i];
    }
}

constexpr int64_t ANY_PART_ROWS = 32, ANY_PARTS = 128;

// Columns that a row's threads have to hold, and the shape that does; 0 threads: too wide, or dy's and dx's rows start differently within 16 bytes.
int64_t span8(const layer_norm_params* p) { return p->cols + ((p->cols | p->y_stride) % 8 ? 7 : 0); }

RowShape shape8(const layer_norm_params* p)
{
    if ((p->y_stride - p->cols) % 8) return RowShape{0, 0, 0};
    return bwd_shape(p->rows, span8(p), p->y_dtype == CONV2D_OUT_BF16 ? 2 : 4, span8(p) == p->cols);
}

bool sums_in_rows8(RowShape s) { return s.elems == 8 || s.elems == 16; }

int64_t bwd8_parts(const layer_norm_params* p)
{
    const RowShape s = shape8(p);
    if (s.threads && sums_in_rows8(s)) {
        const int64_t rows = bwd_blocks(p->rows, s), any = mx::cdiv(p->rows, ANY_PART_ROWS);  // the workspace does for either way
        return rows > any || rows > ANY_PARTS ? rows : any < ANY_PARTS ? any : ANY_PARTS;
    }
    const int64_t n = mx::cdiv(p->rows, ANY_PART_ROWS);
    return n < ANY_PARTS ? n : ANY_PARTS;
}

int check8(const layer_norm_params* p)
{
    constexpr int64_t most_rows = (int64_t(1) << 31) - 32, most_cols = int64_t(1) << 30;
    if (!p || p->rows < 0 || p->cols < 1) return CONV2D_ERR_INVALID;
    if (p->rows > most_rows || p->cols > most_cols) return CONV2D_ERR_UNSUPPORTED;
    if ((p->y_dtype != CONV2D_OUT_F32 && p->y_dtype != CONV2D_OUT_BF16) || p->y_stride < p->cols) return CONV2D_ERR_INVALID;
    return CONV2D_OK;
}

template <typename TY, int E, int G, int MOST, bool SUMS, bool WHOLE>
int start8(const BwdParams& p, const Checkpoint& x, RowShape s, int64_t grid, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    constexpr int ring = depth8<TY, E, G, MOST, WHOLE>() * RING8<TY, E, WHOLE>, join = G ? 2 * E * 4 : 0;
    constexpr int per_thread = ring > join ? ring : join;
    const auto kernel = bwd8_rows<TY, E, G, MOST, SUMS, WHOLE>;
    if (!mx::allow_smem(kernel, per_thread * MOST, done)) return CONV2D_ERR_CUDA;
    const int threads = block_threads(s);
    return mx::launch(kernel, grid, threads, per_thread * threads, stream, 1, static_cast<const TY*>(p.dy), x, static_cast<TY*>(p.dx), p) == cudaSuccess
               ? CONV2D_OK
               : CONV2D_ERR_CUDA;
}

template <typename TY, int E, int G, int MOST, bool SUMS>
int start8(const BwdParams& p, const Checkpoint& x, RowShape s, int64_t grid, cudaStream_t stream)
{
    return p.span == p.cols ? start8<TY, E, G, MOST, SUMS, true>(p, x, s, grid, stream) : start8<TY, E, G, MOST, SUMS, false>(p, x, s, grid, stream);
}

template <typename TY>
int rows8(const BwdParams& p, const Checkpoint& x, RowShape s, cudaStream_t stream)
{
    const int64_t grid = p.chunks;
    if constexpr (sizeof(TY) == 2) {
        if (s.threads == 4) return start8<TY, 16, 4, 256, true>(p, x, s, grid, stream);
        if (s.threads == 8 && s.elems == 16) return start8<TY, 16, 8, 256, true>(p, x, s, grid, stream);
        if (s.threads == 16 && s.elems == 16) return start8<TY, 16, 16, 256, true>(p, x, s, grid, stream);
    }
    if (s.threads == 8) return start8<TY, 8, 8, 256, true>(p, x, s, grid, stream);
    if (s.threads == 16) return start8<TY, 8, 16, 256, true>(p, x, s, grid, stream);
    if (s.threads == 32) return s.elems == 8 ? start8<TY, 8, 32, 256, true>(p, x, s, grid, stream) : start8<TY, 16, 32, 256, true>(p, x, s, grid, stream);
    if (s.elems == 8) return start8<TY, 8, 0, 256, true>(p, x, s, grid, stream);
    if (s.elems == 16) return s.most == 256 ? start8<TY, 16, 0, 256, true>(p, x, s, grid, stream) : start8<TY, 16, 0, 512, true>(p, x, s, grid, stream);
    // No registers are left for the sums: dx alone, in blocks of its own number.
    return start8<TY, 32, 0, 512, false>(p, x, s, row_blocks(p.rows, s, bwd_resident(s)), stream);
}

// Rows that lie in vectors, each alike to dy's and dx's, by the kernels that hold them; others are read again for each pass.
template <typename TY>
int bwd8(BwdParams& k, const Checkpoint& x, const layer_norm_params* params, cudaStream_t stream)
{
    const TY* dy = static_cast<const TY*>(k.dy);
    const RowShape s = shape8(params);
    const bool starts = reinterpret_cast<uintptr_t>(k.dy) % 16 == 0 && reinterpret_cast<uintptr_t>(k.dx) % 16 == 0;
    const bool held = s.threads && starts;
    k.span = static_cast<int>(span8(params));
    if (held && sums_in_rows8(s)) {
        k.chunks = static_cast<int>(bwd_blocks(k.rows, s));
        return rows8<TY>(k, x, s, stream);
    }
    k.chunks = static_cast<int>(mx::cdiv(k.rows, ANY_PART_ROWS) < ANY_PARTS ? mx::cdiv(k.rows, ANY_PART_ROWS) : ANY_PARTS);
    if (k.part) {  // first, as dx may take dy's place
        const bool vec = starts && (k.cols | k.dy_stride) % 8 == 0;
        const dim3 parts(static_cast<unsigned>(mx::cdiv<int64_t>(k.cols, THREADS * (vec ? 8 : 1))), static_cast<unsigned>(k.chunks));
        if (vec)
            bwd8_part_any<TY, 8><<<parts, THREADS, 0, stream>>>(dy, x, k);
        else
            bwd8_part_any<TY, 1><<<parts, THREADS, 0, stream>>>(dy, x, k);
    }
    if (held) {
        if (int rc = rows8<TY>(k, x, s, stream)) return rc;
    } else {
        const unsigned grid = static_cast<unsigned>(k.rows < 65536 ? k.rows : 65536);
        bwd8_dx_any<<<grid, THREADS, 0, stream>>>(dy, x, static_cast<TY*>(k.dx), k);
    }
    return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

}  // namespace ln
}  // namespace sgb

using namespace sgb;

extern "C" size_t mxint8_layer_norm_bwd_workspace_bytes(const layer_norm_params* params)
{
    if (ln::check8(params)) return 0;
    return static_cast<size_t>(ln::bwd8_parts(params)) * 2 * static_cast<size_t>(params->cols) * sizeof(float);
}

extern "C" int mxint8_layer_norm_bwd(const layer_norm_params* params, const void* dy_dev, const void* data_dev, const void* scales_dev,
                                     const float* mean_dev, const float* rstd_dev, const float* weight_dev, void* dx_dev,
                                     float* dweight_dev, float* dbias_dev, void* workspace_dev, size_t workspace_bytes,
                                     conv2d_stream_t stream)
{
    if (int rc = ln::check8(params)) return rc;
    const bool sums = dweight_dev || dbias_dev;
    if (params->rows > 0 && (!dy_dev || !data_dev || !scales_dev || !mean_dev || !rstd_dev || !dx_dev)) return CONV2D_ERR_INVALID;
    const auto aligned = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    const size_t sy = params->y_dtype == CONV2D_OUT_BF16 ? 2 : 4;
    if (!aligned(data_dev, 16) || !aligned(dx_dev, sy) || !aligned(dy_dev, sy) || !aligned(mean_dev, 4) || !aligned(rstd_dev, 4) ||
        !aligned(weight_dev, 4) || !aligned(dweight_dev, 4) || !aligned(dbias_dev, 4) || !aligned(workspace_dev, 16))
        return CONV2D_ERR_ALIGNMENT;
    const size_t need = mxint8_layer_norm_bwd_workspace_bytes(params);
    if (sums && need && (!workspace_dev || workspace_bytes < need)) return CONV2D_ERR_WORKSPACE;
    ln::BwdParams k{};
    k.rows = params->rows;
    k.dy_stride = params->y_stride;
    k.cols = static_cast<int>(params->cols);
    k.inv_cols = 1.f / static_cast<float>(params->cols);
    k.mean = mean_dev;
    k.rstd = rstd_dev;
    k.weight = weight_dev;
    k.dweight = dweight_dev;
    k.dbias = dbias_dev;
    k.dy = dy_dev;
    k.dx = dx_dev;
    k.part = sums ? static_cast<float*>(workspace_dev) : nullptr;
    const ln::Checkpoint x{static_cast<const uint8_t*>(data_dev), static_cast<const uint8_t*>(scales_dev),
                           mx::cdiv<int64_t>(params->cols, mx::BLOCK)};
    int rc = CONV2D_OK;
    if (params->rows > 0) rc = params->y_dtype == CONV2D_OUT_BF16 ? ln::bwd8<__nv_bfloat16>(k, x, params, stream) : ln::bwd8<float>(k, x, params, stream);
    if (rc || !sums) return rc;
    return ln::join_parts(k, stream);
}
