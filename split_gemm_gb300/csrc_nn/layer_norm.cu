// Layer normalisation: the C entry points.
#include "layer_norm.h"

#include <type_traits>

#include "ln_any.cuh"

namespace sgb {
namespace ln {

// ---------------------------------------------------------------- host
constexpr int64_t MAX_ROWS = (int64_t(1) << 31) - 1;
constexpr int64_t MAX_COLS = int64_t(1) << 30;  // column counters are ints and step past the end

bool dtype_ok(int32_t t) { return t == CONV2D_OUT_F32 || t == CONV2D_OUT_BF16; }
size_t dtype_size(int32_t t) { return t == CONV2D_OUT_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check(const layer_norm_params* p, bool y)
{
    if (!p || p->rows < 0 || p->cols < 1) return CONV2D_ERR_INVALID;
    if (p->rows > MAX_ROWS || p->cols > MAX_COLS) return CONV2D_ERR_UNSUPPORTED;
    if (!dtype_ok(p->x_dtype) || p->x_stride < p->cols || !(p->eps >= 0.f)) return CONV2D_ERR_INVALID;
    if (y && (!dtype_ok(p->y_dtype) || p->y_stride < p->cols)) return CONV2D_ERR_INVALID;
    return CONV2D_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA; }

unsigned row_grid(int64_t rows) { return static_cast<unsigned>(rows < 65536 ? rows : 65536); }

FwdParams fwd_params(const layer_norm_params* p, const float* weight, const float* bias, float* mean, float* rstd)
{
    FwdParams k{};
    k.rows = p->rows;
    k.x_stride = p->x_stride;
    k.y_stride = p->y_stride;
    k.padded_rows = mx::cdiv<int64_t>(p->rows, mx::TILE_ROWS) * mx::TILE_ROWS;
    k.cols = static_cast<int>(p->cols);
    k.eps = p->eps;
    k.inv_cols = 1.f / static_cast<float>(p->cols);
    k.weight = weight;
    k.bias = bias;
    k.mean = mean;
    k.rstd = rstd;
    return k;
}

// Calls f with null pointers of the two element types.
template <typename F>
void by_types(int32_t x, int32_t y, F&& f)
{
    float* f32 = nullptr;
    __nv_bfloat16* b16 = nullptr;
    if (x == CONV2D_OUT_BF16)
        y == CONV2D_OUT_BF16 ? f(b16, b16) : f(b16, f32);
    else
        y == CONV2D_OUT_BF16 ? f(f32, b16) : f(f32, f32);
}

// Parts that the sums over the rows are made in: one for each block of the kernel that takes them, or, for rows too wide
// for that, a multiple of 8 of some 32 rows each, at most so many.
constexpr int64_t PART_ROWS = 32, PARTS = 128;

// Columns that the threads of a row have to hold: where rows do not start at whole vectors, up to 7 elements
// stand in front of them.  A row that fits its kernel (`most` columns) only without those is read by elements instead,
// where that is the faster way.
bool whole_rows(const layer_norm_params* p) { return (p->cols | p->x_stride | p->y_stride) % 8 == 0; }

int64_t span_of(const layer_norm_params* p, int64_t most)
{
    return whole_rows(p) || (p->cols <= most && p->cols + 7 > most) ? p->cols : p->cols + 7;
}

// 16384 columns: else the kernels for any width (8192 x 16383: fp32 forward 244 us against 405, backward 476 against 778; but
// bf16 forward 317 against 209, though backward 454 against 501; bf16, 64 rows: 6.2 against 16.4 and 13.8 against 22.0).
int64_t most_columns(const layer_norm_params* p) { return p->x_dtype == CONV2D_OUT_F32 || p->rows <= SMS ? 16384 : 0; }
int64_t fwd_span(const layer_norm_params* p) { return span_of(p, most_columns(p)); }
// 8192 columns: else the sums take a kernel of their own (16384 x 8191: bf16 303 us against 386, fp32 322 against 640).
int64_t bwd_span(const layer_norm_params* p) { return span_of(p, p->cols <= 8192 ? 8192 : most_columns(p)); }

// Whether the kernels that hold rows read them in vectors, `vec` telling of their alignment to each other.
bool rows_in_vectors(const layer_norm_params* p, int64_t span, bool vec) { return vec && (span != p->cols || whole_rows(p)); }

// Whether the kernel that computes dx holds the sums over its rows as well.
bool sums_in_rows(RowShape s) { return s.elems == 8 || s.elems == 16; }

int64_t bwd_parts(const layer_norm_params* p)
{
    const int64_t span = bwd_span(p);
    const RowShape s = bwd_shape(p->rows, span, static_cast<int>(dtype_size(p->x_dtype)), span == p->cols);
    if (!sums_in_rows(s)) {
        const int64_t n = mx::cdiv(p->rows, 8 * PART_ROWS) * 8;
        return n < PARTS ? n : PARTS;
    }
    return bwd_blocks(p->rows, s);
}

// Whether rows at `p`, `stride` elements apart, lie to vectors of `vec` elements as those of x do, x starting at a
// whole one.
bool in_vectors(const void* p, int64_t stride, int64_t x_stride, size_t elem, int64_t vec)
{
    const size_t bytes = vec * elem < 16 ? vec * elem : 16;
    return (stride - x_stride) % vec == 0 && aligned(p, bytes);
}

int64_t vector_of(int32_t x_dtype) { return x_dtype == CONV2D_OUT_BF16 ? 8 : 4; }

}  // namespace ln
}  // namespace sgb

using namespace sgb;

extern "C" int layer_norm_fwd(const layer_norm_params* params, const void* x_dev, const float* weight_dev,
                              const float* bias_dev, void* y_dev, float* mean_dev, float* rstd_dev,
                              conv2d_stream_t stream)
{
    if (int rc = ln::check(params, true)) return rc;
    if (params->rows == 0) return CONV2D_OK;
    if (!x_dev || !y_dev) return CONV2D_ERR_INVALID;
    if (!ln::aligned(x_dev, ln::dtype_size(params->x_dtype)) || !ln::aligned(y_dev, ln::dtype_size(params->y_dtype)) ||
        !ln::aligned(weight_dev, 4) || !ln::aligned(bias_dev, 4) || !ln::aligned(mean_dev, 4) || !ln::aligned(rstd_dev, 4))
        return CONV2D_ERR_ALIGNMENT;
    ln::FwdParams k = ln::fwd_params(params, weight_dev, bias_dev, mean_dev, rstd_dev);
    k.x = x_dev;
    k.y = y_dev;
    const int64_t v = ln::vector_of(params->x_dtype);
    const bool vec = ln::in_vectors(x_dev, k.x_stride, k.x_stride, ln::dtype_size(params->x_dtype), v) &&
                     ln::in_vectors(y_dev, k.y_stride, k.x_stride, ln::dtype_size(params->y_dtype), v);
    k.span = static_cast<int>(ln::fwd_span(params));
    const bool rows_vec = ln::rows_in_vectors(params, k.span, vec);
    int rc = CONV2D_OK;
    ln::by_types(params->x_dtype, params->y_dtype, [&](auto* tx, auto* ty) {
        using TX = std::remove_pointer_t<decltype(tx)>;
        using TY = std::remove_pointer_t<decltype(ty)>;
        rc = ln::launch_fwd_rows<TX, TY>(k, rows_vec, stream);
        if (rc != CONV2D_ERR_UNSUPPORTED) return;
        ln::fwd_any<<<ln::row_grid(k.rows), ln::THREADS, 0, stream>>>(static_cast<const TX*>(x_dev), static_cast<TY*>(y_dev), k);
        rc = ln::launched();
    });
    return rc;
}

extern "C" int layer_norm_mxfp4(const layer_norm_params* params, const void* x_dev, const float* weight_dev,
                                const float* bias_dev, void* data_dev, void* scales_dev, float* mean_dev,
                                float* rstd_dev, conv2d_stream_t stream)
{
    if (int rc = ln::check(params, false)) return rc;
    if (params->rows == 0) return CONV2D_OK;
    if (!x_dev || !data_dev || !scales_dev) return CONV2D_ERR_INVALID;
    if (!ln::aligned(x_dev, ln::dtype_size(params->x_dtype)) || !ln::aligned(data_dev, 16) || !ln::aligned(scales_dev, 16) ||
        !ln::aligned(weight_dev, 4) || !ln::aligned(bias_dev, 4) || !ln::aligned(mean_dev, 4) || !ln::aligned(rstd_dev, 4))
        return CONV2D_ERR_ALIGNMENT;
    ln::FwdParams k = ln::fwd_params(params, weight_dev, bias_dev, mean_dev, rstd_dev);
    k.x = x_dev;
    const int64_t v = ln::vector_of(params->x_dtype);
    const bool whole = k.cols % v == 0 && k.x_stride % v == 0;
    k.span = static_cast<int>(whole ? k.cols : ln::fwd_span(params));
    const bool vec = ln::aligned(x_dev, 16) && (whole || k.span != k.cols);
    k.data = static_cast<uint8_t*>(data_dev);
    k.scales = static_cast<uint8_t*>(scales_dev);
    int rc = CONV2D_OK;
    ln::by_types(params->x_dtype, CONV2D_OUT_F32, [&](auto* tx, auto*) {
        using TX = std::remove_pointer_t<decltype(tx)>;
        rc = ln::launch_fwd_rows<TX, void>(k, vec, stream);
        if (rc != CONV2D_ERR_UNSUPPORTED) return;
        ln::fwd_mx_any<<<ln::row_grid(k.padded_rows), ln::THREADS, 0, stream>>>(static_cast<const TX*>(x_dev), k);
        rc = ln::launched();
    });
    return rc;
}

extern "C" size_t layer_norm_bwd_workspace_bytes(const layer_norm_params* params)
{
    if (ln::check(params, true)) return 0;
    return static_cast<size_t>(ln::bwd_parts(params)) * 2 * static_cast<size_t>(params->cols) * sizeof(float);
}

extern "C" int layer_norm_bwd(const layer_norm_params* params, const void* dy_dev, const void* x_dev,
                              const float* mean_dev, const float* rstd_dev, const float* weight_dev, void* dx_dev,
                              float* dweight_dev, float* dbias_dev, void* workspace_dev, size_t workspace_bytes,
                              conv2d_stream_t stream)
{
    if (int rc = ln::check(params, true)) return rc;
    const bool sums = dweight_dev || dbias_dev;
    if (params->rows > 0 && (!dy_dev || !x_dev || !mean_dev || !rstd_dev || !dx_dev)) return CONV2D_ERR_INVALID;
    if (!ln::aligned(x_dev, ln::dtype_size(params->x_dtype)) || !ln::aligned(dx_dev, ln::dtype_size(params->x_dtype)) ||
        !ln::aligned(dy_dev, ln::dtype_size(params->y_dtype)) || !ln::aligned(mean_dev, 4) || !ln::aligned(rstd_dev, 4) ||
        !ln::aligned(weight_dev, 4) || !ln::aligned(dweight_dev, 4) || !ln::aligned(dbias_dev, 4) || !ln::aligned(workspace_dev, 16))
        return CONV2D_ERR_ALIGNMENT;
    const size_t need = layer_norm_bwd_workspace_bytes(params);
    if (sums && need && (!workspace_dev || workspace_bytes < need)) return CONV2D_ERR_WORKSPACE;
    ln::BwdParams k{};
    k.rows = params->rows;
    k.x_stride = params->x_stride;
    k.dy_stride = params->y_stride;
    k.cols = static_cast<int>(params->cols);
    k.inv_cols = 1.f / static_cast<float>(params->cols);
    k.mean = mean_dev;
    k.rstd = rstd_dev;
    k.weight = weight_dev;
    k.dweight = dweight_dev;
    k.dbias = dbias_dev;
    k.x = x_dev;
    k.dy = dy_dev;
    k.dx = dx_dev;
    k.part = sums ? static_cast<float*>(workspace_dev) : nullptr;
    k.chunks = static_cast<int>(ln::bwd_parts(params));
    const int64_t v = ln::vector_of(params->x_dtype);
    const size_t sx = ln::dtype_size(params->x_dtype);
    const bool vec = ln::in_vectors(x_dev, k.x_stride, k.x_stride, sx, v) && ln::in_vectors(dx_dev, k.cols, k.x_stride, sx, v) &&
                     ln::in_vectors(dy_dev, k.dy_stride, k.x_stride, ln::dtype_size(params->y_dtype), v);
    k.span = static_cast<int>(ln::bwd_span(params));
    const bool rows_vec = ln::rows_in_vectors(params, k.span, vec);
    int rc = CONV2D_OK;
    if (params->rows > 0)
        ln::by_types(params->x_dtype, params->y_dtype, [&](auto* tx, auto* ty) {
            using TX = std::remove_pointer_t<decltype(tx)>;
            using TY = std::remove_pointer_t<decltype(ty)>;
            rc = ln::launch_bwd_rows<TX, TY>(k, rows_vec, k.chunks, stream);
            if (rc != CONV2D_OK && rc != CONV2D_ERR_UNSUPPORTED) return;
            if (rc == CONV2D_OK && ln::sums_in_rows(ln::bwd_shape(k.rows, k.span, sizeof(TX), k.span == k.cols))) return;
            const TX* x = static_cast<const TX*>(x_dev);
            const TY* dy = static_cast<const TY*>(dy_dev);
            if (rc == CONV2D_ERR_UNSUPPORTED)
                ln::bwd_dx_any<<<ln::row_grid(k.rows), ln::THREADS, 0, stream>>>(dy, x, static_cast<TX*>(dx_dev), k);
            constexpr int VEC = 16 / sizeof(TX);
            const auto columns = [&](int vec) {  // with what may stand in front of an unaligned row
                return dim3(static_cast<unsigned>(mx::cdiv<int64_t>(int64_t(k.cols) + vec - 1, ln::THREADS * vec)), static_cast<unsigned>(k.chunks));
            };
            if (sums && vec)
                ln::bwd_part_any<TX, TY, VEC><<<columns(VEC), ln::THREADS, 0, stream>>>(dy, x, k);
            else if (sums)
                ln::bwd_part_any<TX, TY, 1><<<columns(1), ln::THREADS, 0, stream>>>(dy, x, k);
            rc = ln::launched();
        });
    if (rc) return rc;
    if (!sums) return CONV2D_OK;
    return mx::launch(ln::bwd_join, mx::cdiv(k.cols, 32), 1024, 0, stream, 1, k) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}
