// Low-rank adapters: the C entry points and the rules by which kernels are chosen.
#include "adapter.h"

#include <atomic>
#include <mutex>

#include "adapter_params.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ad {

__device__ uint32_t adapter_word, adapter_taken;  // as the product's status words

__global__ void take_adapter_status() { adapter_taken = atomicExch(&adapter_word, 0u); }

std::mutex asking;

constexpr int64_t MOST_COLS = int64_t(1) << 30;

size_t size_of(int32_t t) { return t == CONV2D_OUT_BF16 ? 2 : 4; }

bool vectors(const void* p, int64_t stride, size_t elem) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * elem % 16 == 0; }

// Whether every row that the pass touches is whole 16-byte vectors.
bool in_vectors(const PassParams& p, int32_t base, int32_t out)
{
    return (p.rank | p.from | p.to) % 8 == 0 && vectors(p.in, p.in_stride, 2) && vectors(p.w1, 8, 2) && vectors(p.w2, 8, 2) && vectors(p.mid, 8, 4) &&
           vectors(p.base, p.base ? p.base_stride : 8, size_of(base)) && vectors(p.out, p.out ? p.out_stride : 8, size_of(out));
}

// dh's bytes in the workspace, to whole vectors.
size_t dh_bytes(int64_t rows, int64_t rank) { return (static_cast<size_t>(rows) * static_cast<size_t>(rank) * 4 + 15) / 16 * 16; }

// Two parts of a gradient to a piece, to whole vectors.
size_t part_bytes(const adapter_bwd_params& q, int64_t cols, int tiles_each)
{
    const int64_t pieces = sum_pieces(PlanLayout(q.rows, q.adapters), tiles_each);
    return (2 * static_cast<size_t>(pieces) * q.rank * static_cast<size_t>(cols) * 4 + 15) / 16 * 16;
}

SumCut cut_sums(const adapter_bwd_params& q) { return cut_sums(q.rows, q.adapters, static_cast<int>(q.rank), q.cols, q.outs); }

size_t bwd_bytes(const adapter_bwd_params& q, const SumCut& each)
{
    return dh_bytes(q.rows, q.rank) + part_bytes(q, q.cols, each.da) + part_bytes(q, q.outs, each.db);
}

bool status_word(uint32_t** word)
{
    void* at = nullptr;
    if (cudaGetSymbolAddress(&at, adapter_word) != cudaSuccess) return false;
    *word = static_cast<uint32_t*>(at);
    return true;
}

bool dtype_ok(int32_t t) { return t == CONV2D_OUT_F32 || t == CONV2D_OUT_BF16; }
bool aligned(const void* p, int32_t t) { return reinterpret_cast<uintptr_t>(p) % (t == CONV2D_OUT_BF16 ? 2 : 4) == 0; }

int check(int64_t rows, int64_t cols, int64_t outs, int64_t rank, int64_t adapters)
{
    if (rows < 0 || cols < 1 || outs < 1 || rank < 1 || adapters < 1) return CONV2D_ERR_INVALID;
    if (rows > MOST_ROWS || cols > MOST_COLS || outs > MOST_COLS || rank > MOST_RANK || adapters > MOST_ADAPTERS) return CONV2D_ERR_UNSUPPORTED;
    return CONV2D_OK;
}

}  // namespace ad
}  // namespace sgb

using namespace sgb;

extern "C" int adapter_fwd(const adapter_fwd_params* params, const void* plan_dev, const void* y_dev, const void* x_dev,
                           const void* a_dev, const void* b_dev, const float* scale_dev, void* out_dev, float* h_dev,
                           conv2d_stream_t stream)
{
    if (!params) return CONV2D_ERR_INVALID;
    const adapter_fwd_params& q = *params;
    if (int rc = ad::check(q.rows, q.cols, q.outs, q.rank, q.adapters)) return rc;
    if (!ad::dtype_ok(q.y_dtype) || !ad::dtype_ok(q.out_dtype) || (q.activation != CONV2D_ACT_NONE && q.activation != CONV2D_ACT_RELU) ||
        q.x_stride < q.cols || q.y_stride < q.outs || q.out_stride < q.outs)
        return CONV2D_ERR_INVALID;
    if (q.rows == 0) return CONV2D_OK;
    if (!plan_dev || !y_dev || !x_dev || !a_dev || !b_dev || !out_dev) return CONV2D_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(plan_dev) % 16 || !ad::aligned(x_dev, CONV2D_OUT_BF16) || !ad::aligned(a_dev, CONV2D_OUT_BF16) ||
        !ad::aligned(b_dev, CONV2D_OUT_BF16) || !ad::aligned(scale_dev, CONV2D_OUT_F32) || !ad::aligned(h_dev, CONV2D_OUT_F32) ||
        !ad::aligned(y_dev, q.y_dtype) || !ad::aligned(out_dev, q.out_dtype))
        return CONV2D_ERR_ALIGNMENT;
    ad::PassParams p{};
    p.plan = ad::plan_of(plan_dev, q.rows, q.adapters);
    if (!ad::status_word(&p.status)) return CONV2D_ERR_CUDA;
    p.in = static_cast<const __nv_bfloat16*>(x_dev);
    p.w1 = static_cast<const __nv_bfloat16*>(a_dev);
    p.w2 = static_cast<const __nv_bfloat16*>(b_dev);
    p.scale = scale_dev;
    p.base = y_dev;
    p.out = out_dev;
    p.mid = h_dev;
    p.in_stride = q.x_stride;
    p.base_stride = q.y_stride;
    p.out_stride = q.out_stride;
    p.adapters = static_cast<int>(q.adapters);
    p.rank = static_cast<int>(q.rank);
    p.from = static_cast<int>(q.cols);
    p.to = static_cast<int>(q.outs);
    p.relu = q.activation == CONV2D_ACT_RELU;
    // Few rows by pieces of 8, which read an adapter's weights for each.  The same calls by pieces and by tiles, us, 4096 -> 4096: rank 16, 32 adapters, 64 rows
    // 5.2 and 17.6, 512 14.4 and 18.9, 640 16.1 and 20.5; rank 32, 8 adapters, 256 rows 8.5 and 12.4, 320 12.9 and 12.5; rank 64, 8 adapters, 160 rows 13.8 and 14.2, 256 20.5
    // and 14.6.  Narrower layers would gain from pieces for longer (1024 -> 1024, rank 64, 256 rows 6.8 and 10.0).  Ranks above 64 have no such kernel.
    if (q.rows * mx::cdiv<int64_t>(q.rank, 16) <= ad::SMALL_ROWS && q.rank <= 64)
        return ad::launch_small_fwd(p, q.y_dtype, q.out_dtype, ad::in_vectors(p, q.y_dtype, q.out_dtype), stream);
    const bool vec = ad::in_vectors(p, q.y_dtype, q.out_dtype);
    const ad::PassCut cut = ad::cut_pass(q.rows, p.adapters, p.rank, p.from, p.to, static_cast<int>(ad::size_of(q.y_dtype)), static_cast<int>(ad::size_of(q.out_dtype)), vec);
    p.splits = cut.splits;
    return ad::launch_pass_fwd(p, q.y_dtype, q.out_dtype, vec, cut.halved, stream);
}

extern "C" size_t adapter_bwd_workspace_bytes(const adapter_bwd_params* params)
{
    if (!params || ad::check(params->rows, params->cols, params->outs, params->rank, params->adapters)) return 0;
    return ad::bwd_bytes(*params, ad::cut_sums(*params));
}

extern "C" int adapter_bwd(const adapter_bwd_params* params, const void* plan_dev, const void* dy_dev, const void* x_dev,
                           const void* x_scales_dev, const float* h_dev, const void* a_dev, const void* b_dev,
                           const float* scale_dev, const void* dx0_dev, void* dx_dev, float* da_dev, float* db_dev,
                           void* workspace_dev, size_t workspace_bytes, conv2d_stream_t stream)
{
    if (!params) return CONV2D_ERR_INVALID;
    const adapter_bwd_params& q = *params;
    if (int rc = ad::check(q.rows, q.cols, q.outs, q.rank, q.adapters)) return rc;
    const bool eight = q.x_type == ADAPTER_X_MXINT8;
    if ((!eight && q.x_type != ADAPTER_X_BF16) || !ad::dtype_ok(q.dx0_dtype) || !ad::dtype_ok(q.dx_dtype) || q.dy_stride < q.outs ||
        (dx_dev && q.dx_stride < q.cols) || (dx0_dev && q.dx0_stride < q.cols) || (!eight && da_dev && q.x_stride < q.cols))
        return CONV2D_ERR_INVALID;
    if (!ad::aligned(da_dev, CONV2D_OUT_F32) || !ad::aligned(db_dev, CONV2D_OUT_F32)) return CONV2D_ERR_ALIGNMENT;
    ad::SumCut each{1, 1};
    if (q.rows > 0) {
        if (!plan_dev || !dy_dev || !a_dev || !b_dev || (da_dev && (!x_dev || (eight && !x_scales_dev))) || (db_dev && !h_dev))
            return CONV2D_ERR_INVALID;
        if (reinterpret_cast<uintptr_t>(plan_dev) % 16 || reinterpret_cast<uintptr_t>(workspace_dev) % 16 || !ad::aligned(dy_dev, CONV2D_OUT_BF16) ||
            (eight ? reinterpret_cast<uintptr_t>(x_dev) % 16 != 0 : !ad::aligned(x_dev, CONV2D_OUT_BF16)) || !ad::aligned(h_dev, CONV2D_OUT_F32) ||
            !ad::aligned(a_dev, CONV2D_OUT_BF16) || !ad::aligned(b_dev, CONV2D_OUT_BF16) || !ad::aligned(scale_dev, CONV2D_OUT_F32) ||
            !ad::aligned(dx0_dev, q.dx0_dtype) || !ad::aligned(dx_dev, q.dx_dtype))
            return CONV2D_ERR_ALIGNMENT;
        each = ad::cut_sums(q);
        const size_t need = ad::bwd_bytes(q, each);
        if (need && (!workspace_dev || workspace_bytes < need)) return CONV2D_ERR_WORKSPACE;
    } else {
        const size_t grads = static_cast<size_t>(q.adapters) * q.rank * 4;
        if (da_dev && cudaMemsetAsync(da_dev, 0, grads * q.cols, stream) != cudaSuccess) return CONV2D_ERR_CUDA;
        if (db_dev && cudaMemsetAsync(db_dev, 0, grads * q.outs, stream) != cudaSuccess) return CONV2D_ERR_CUDA;
        return CONV2D_OK;
    }
    ad::PassParams p{};
    p.plan = ad::plan_of(plan_dev, q.rows, q.adapters);
    p.in = static_cast<const __nv_bfloat16*>(dy_dev);
    p.w1 = static_cast<const __nv_bfloat16*>(b_dev);
    p.w2 = static_cast<const __nv_bfloat16*>(a_dev);
    p.scale = scale_dev;
    p.base = dx0_dev;
    p.out = dx_dev;
    p.mid = static_cast<float*>(workspace_dev);
    p.in_stride = q.dy_stride;
    p.base_stride = q.dx0_stride;
    p.out_stride = q.dx_stride;
    p.adapters = static_cast<int>(q.adapters);
    p.rank = static_cast<int>(q.rank);
    p.from = static_cast<int>(q.outs);
    p.to = static_cast<int>(q.cols);
    if (!ad::status_word(&p.status)) return CONV2D_ERR_CUDA;
    const bool vec = ad::in_vectors(p, q.dx0_dtype, q.dx_dtype);
    const ad::PassCut cut = ad::cut_pass(q.rows, p.adapters, p.rank, p.from, p.to, dx0_dev ? static_cast<int>(ad::size_of(q.dx0_dtype)) : 0, dx_dev ? static_cast<int>(ad::size_of(q.dx_dtype)) : 0, vec);
    p.splits = cut.splits;
    p.early = da_dev || db_dev;
    if (dx_dev || da_dev)
        if (int rc = ad::launch_pass_bwd(p, q.dx0_dtype, q.dx_dtype, vec, cut.halved, stream)) return rc;
    ad::SumParams s{};
    s.plan = p.plan;
    s.status = p.status;
    s.adapters = p.adapters;
    s.rank = p.rank;
    s.beside = dx_dev || da_dev;
    uint8_t* part = static_cast<uint8_t*>(workspace_dev) + ad::dh_bytes(q.rows, q.rank);
    if (da_dev) {
        ad::SumJob& job = s.jobs[0];
        job.in = static_cast<const __nv_bfloat16*>(x_dev);
        job.data = static_cast<const uint8_t*>(x_dev);
        job.scales = static_cast<const uint8_t*>(x_scales_dev);
        job.mid = p.mid;
        job.out = da_dev;
        job.part = reinterpret_cast<float*>(part);
        job.tiles_each = each.da;
        job.in_stride = q.x_stride;
        job.blocks = mx::cdiv<int64_t>(q.cols, 32);
        job.cols = static_cast<int>(q.cols);
        job.mode = eight ? 2 : q.cols % 8 == 0 && ad::vectors(x_dev, q.x_stride, 2) ? 0 : 1;
        job.out_col = 1;
    }
    if (db_dev) {
        ad::SumJob& job = s.jobs[1];
        job.in = static_cast<const __nv_bfloat16*>(dy_dev);
        job.mid = h_dev;
        job.out = db_dev;
        job.part = reinterpret_cast<float*>(part + ad::part_bytes(q, q.cols, each.da));
        job.tiles_each = each.db;
        job.in_stride = q.dy_stride;
        job.cols = static_cast<int>(q.outs);
        job.mode = q.outs % 8 == 0 && ad::vectors(dy_dev, q.dy_stride, 2) ? 0 : 1;
        job.out_col = 0;
    }
    return ad::launch_sums(s, ad::PlanLayout(q.rows, q.adapters), stream);
}

extern "C" int adapter_status(conv2d_stream_t stream)
{
    uint32_t word = 0;
    std::lock_guard<std::mutex> one(ad::asking);
    ad::take_adapter_status<<<1, 1, 0, stream>>>();
    if (cudaGetLastError() != cudaSuccess) return CONV2D_ERR_CUDA;
    if (cudaMemcpyFromSymbolAsync(&word, ad::adapter_taken, sizeof word, 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return CONV2D_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return CONV2D_ERR_CUDA;
    return word == 0 ? CONV2D_OK : CONV2D_ERR_TIMEOUT;
}
