// The row operators' calls on ordinary torch tensors, without Python between the arguments and the C ABI.
//
// A one-token call spends a few microseconds on the GPU; checking its arguments and allocating its results in Python took
// 11 to 23 us on a Grace core.  These functions take the usual case (dense tensors of the expected types on the current
// device, results on its current stream) and return None for everything else: the Python functions that call them then check
// one thing after another and raise what is wrong, or take the strided and streamed cases.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "adapter.h"
#include "layer_norm.h"
#include "mxfp4.h"
#include "mxint8.h"

namespace {

PyObject* g_mxfp4 = nullptr;   // the Mxfp4 type, a named tuple (data, scales, rows, cols)
PyObject* g_mxint8 = nullptr;  // the Mxint8 type, the same
PyObject* g_plan = nullptr;    // the AdapterPlan type, a named tuple (data, rows, adapters)

// The tensor, or nullptr if the object is none (a subclass goes the general way).
const at::Tensor* tensor(PyObject* o)
{
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// conv2d_out_dtype of a type, or -1.
int code_of(at::ScalarType t) { return t == at::kFloat ? CONV2D_OUT_F32 : t == at::kBFloat16 ? CONV2D_OUT_BF16 : -1; }

// Whether kernels that are started now can take the tensor: they start on the current device.
bool here(const at::Tensor& t) { return t.is_cuda() && t.get_device() == c10::cuda::current_device(); }

// A dense CUDA tensor of rows; rows, cols and its type's code are filled in.
struct Rows {
    const at::Tensor* t = nullptr;
    int64_t rows = 0, cols = 0;
    int code = -1;
    explicit Rows(PyObject* o)
    {
        const at::Tensor* x = tensor(o);
        if (!x || !here(*x) || x->dim() < 1 || !x->is_contiguous()) return;
        code = code_of(x->scalar_type());
        cols = x->size(-1);
        if (code < 0 || cols < 1) return;
        rows = x->numel() / cols;
        t = x;
    }
    explicit operator bool() const { return t != nullptr; }
};

// Device pointer of an optional dense fp32 vector of n elements beside x; false where it is something else.
bool vector(PyObject* o, int64_t n, const at::Tensor& x, const float** p)
{
    *p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor* v = tensor(o);
    if (!v || v->scalar_type() != at::kFloat || v->numel() != n || v->device() != x.device() || !v->is_contiguous()) return false;
    *p = static_cast<const float*>(v->data_ptr());
    return true;
}

// A non-negative int of a named tuple, or -1.
int64_t extent(PyObject* o)
{
    int over = 0;
    if (!PyLong_CheckExact(o)) return -1;
    const int64_t n = PyLong_AsLongLongAndOverflow(o, &over);
    return over || n < 0 ? -1 : n;
}

// A quantised matrix of the named tuple type `type`.
struct Quantised {
    const at::Tensor *data = nullptr, *scales = nullptr;
    int64_t rows = 0, cols = 0;
    explicit operator bool() const { return data != nullptr; }

protected:
    Quantised(PyObject* o, PyObject* type, at::ScalarType element, size_t (*data_bytes)(int64_t, int64_t), size_t (*scale_bytes)(int64_t, int64_t))
    {
        if (reinterpret_cast<PyObject*>(Py_TYPE(o)) != type) return;
        const at::Tensor *d = tensor(PyTuple_GET_ITEM(o, 0)), *s = tensor(PyTuple_GET_ITEM(o, 1));
        if (!d || !s) return;
        rows = extent(PyTuple_GET_ITEM(o, 2));
        cols = extent(PyTuple_GET_ITEM(o, 3));
        if (rows < 1 || cols < 1 || !here(*d) || d->device() != s->device() || d->scalar_type() != element || s->scalar_type() != at::kByte ||
            !d->is_contiguous() || !s->is_contiguous() || static_cast<size_t>(d->numel()) != data_bytes(rows, cols) ||
            static_cast<size_t>(s->numel()) != scale_bytes(rows, cols))
            return;
        data = d;
        scales = s;
    }
};

struct Mx : Quantised {
    explicit Mx(PyObject* o) : Quantised(o, g_mxfp4, at::kByte, mxfp4_data_bytes, mxfp4_scale_bytes) {}
};

struct Mx8 : Quantised {
    explicit Mx8(PyObject* o) : Quantised(o, g_mxint8, at::kChar, mxint8_data_bytes, mxint8_scale_bytes) {}
};

// A plan for `rows` rows beside `like`.
struct Plan {
    const at::Tensor* data = nullptr;
    int64_t adapters = 0;
    Plan(PyObject* o, int64_t rows, const at::Tensor& like)
    {
        if (reinterpret_cast<PyObject*>(Py_TYPE(o)) != g_plan) return;
        const at::Tensor* d = tensor(PyTuple_GET_ITEM(o, 0));
        adapters = extent(PyTuple_GET_ITEM(o, 2));
        if (!d || extent(PyTuple_GET_ITEM(o, 1)) != rows || adapters < 1 || d->device() != like.device() || d->scalar_type() != at::kInt ||
            !d->is_contiguous() || static_cast<size_t>(d->numel()) * 4 != adapter_plan_bytes(rows, adapters))
            return;
        data = d;
    }
    explicit operator bool() const { return data != nullptr; }
};

// The adapters' weights, dense bf16 of [adapters][rank][cols] and [adapters][outs][rank] beside `like`; the rank, or 0.
int64_t rank_of(const at::Tensor* a, const at::Tensor* b, int64_t adapters, int64_t cols, int64_t outs, const at::Tensor& like)
{
    if (!a || !b || a->scalar_type() != at::kBFloat16 || b->scalar_type() != at::kBFloat16 || a->device() != like.device() ||
        b->device() != like.device() || !a->is_contiguous() || !b->is_contiguous() || a->dim() != 3 || b->dim() != 3 || a->size(0) != adapters ||
        a->size(2) != cols || b->size(0) != adapters || b->size(1) != outs || a->size(1) != b->size(2))
        return 0;
    return a->size(1);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType t, const at::Tensor& like)
{
    return at::empty(shape, like.options().dtype(t).requires_grad(false));
}

conv2d_stream_t stream_of(const at::Tensor& t) { return reinterpret_cast<conv2d_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream()); }

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject* tuple_of(at::Tensor a, at::Tensor b, at::Tensor c)
{
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, wrap(std::move(a)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(b)));
    PyTuple_SET_ITEM(r, 2, wrap(std::move(c)));
    return r;
}

// (data, scales, rows, cols)
PyObject* mx_tuple(at::Tensor data, at::Tensor scales, int64_t rows, int64_t cols)
{
    PyObject* r = PyTuple_New(4);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, wrap(std::move(data)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(scales)));
    PyTuple_SET_ITEM(r, 2, PyLong_FromLongLong(rows));
    PyTuple_SET_ITEM(r, 3, PyLong_FromLongLong(cols));
    return r;
}

// Type code of an out_dtype argument (None: `other`), or -1.
int out_code(PyObject* o, int other)
{
    if (o == Py_None) return other;
    return THPDtype_Check(o) ? code_of(reinterpret_cast<THPDtype*>(o)->scalar_type) : -1;
}

at::ScalarType type_of(int code) { return code == CONV2D_OUT_BF16 ? at::kBFloat16 : at::kFloat; }

// (x, weight, bias, eps, out_dtype) -> (y, mean, rstd)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5 || !PyFloat_CheckExact(a[3])) Py_RETURN_NONE;
    const Rows x(a[0]);
    if (!x) Py_RETURN_NONE;
    const float *w, *b;
    const int code = out_code(a[4], x.code);
    if (code < 0 || !vector(a[1], x.cols, *x.t, &w) || !vector(a[2], x.cols, *x.t, &b)) Py_RETURN_NONE;
    const auto shape = x.t->sizes();
    at::Tensor y = empty(shape, type_of(code), *x.t);
    at::Tensor mean = empty(shape.slice(0, shape.size() - 1), at::kFloat, *x.t), rstd = empty(shape.slice(0, shape.size() - 1), at::kFloat, *x.t);
    const layer_norm_params p{x.rows, x.cols, x.cols, x.cols, x.code, code, static_cast<float>(PyFloat_AS_DOUBLE(a[3]))};
    if (layer_norm_fwd(&p, x.t->data_ptr(), w, b, y.data_ptr(), static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()),
                       stream_of(*x.t)))
        Py_RETURN_NONE;
    return tuple_of(std::move(y), std::move(mean), std::move(rstd));
    END_HANDLE_TH_ERRORS
}

// (dy, x, mean, rstd, weight) -> (dx, dweight, dbias)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const Rows dy(a[0]), x(a[1]);
    if (!dy || !x || dy.t->device() != x.t->device() || dy.t->sizes() != x.t->sizes() || a[2] == Py_None || a[3] == Py_None) Py_RETURN_NONE;
    const float *mean, *rstd, *w;
    if (!vector(a[2], x.rows, *x.t, &mean) || !vector(a[3], x.rows, *x.t, &rstd) || !vector(a[4], x.cols, *x.t, &w)) Py_RETURN_NONE;
    const layer_norm_params p{x.rows, x.cols, x.cols, x.cols, x.code, dy.code, 0.f};
    const int64_t need = static_cast<int64_t>(layer_norm_bwd_workspace_bytes(&p));
    at::Tensor dx = empty(x.t->sizes(), x.t->scalar_type(), *x.t);
    at::Tensor dw = empty({x.cols}, at::kFloat, *x.t), db = empty({x.cols}, at::kFloat, *x.t), ws = empty({need}, at::kByte, *x.t);
    if (layer_norm_bwd(&p, dy.t->data_ptr(), x.t->data_ptr(), mean, rstd, w, dx.data_ptr(), static_cast<float*>(dw.data_ptr()),
                       static_cast<float*>(db.data_ptr()), ws.data_ptr(), static_cast<size_t>(need), stream_of(*x.t)))
        Py_RETURN_NONE;
    return tuple_of(std::move(dx), std::move(dw), std::move(db));
    END_HANDLE_TH_ERRORS
}

// (x, weight, bias, eps) -> (data, scales, rows, cols)
PyObject* norm_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 4 || !PyFloat_CheckExact(a[3])) Py_RETURN_NONE;
    const Rows x(a[0]);
    if (!x || x.rows < 1) Py_RETURN_NONE;
    const float *w, *b;
    if (!vector(a[1], x.cols, *x.t, &w) || !vector(a[2], x.cols, *x.t, &b)) Py_RETURN_NONE;
    at::Tensor data = empty({x.rows, static_cast<int64_t>(mxfp4_data_bytes(1, x.cols))}, at::kByte, *x.t);
    at::Tensor scales = empty({static_cast<int64_t>(mxfp4_scale_bytes(x.rows, x.cols))}, at::kByte, *x.t);
    const layer_norm_params p{x.rows, x.cols, x.cols, x.cols, x.code, CONV2D_OUT_F32, static_cast<float>(PyFloat_AS_DOUBLE(a[3]))};
    if (layer_norm_mxfp4(&p, x.t->data_ptr(), w, b, data.data_ptr(), scales.data_ptr(), nullptr, nullptr, stream_of(*x.t))) Py_RETURN_NONE;
    return mx_tuple(std::move(data), std::move(scales), x.rows, x.cols);
    END_HANDLE_TH_ERRORS
}

// (x, by_rows, by_columns) -> ((data, scales, rows, cols) or None, the same of the transpose)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 3) Py_RETURN_NONE;
    const Rows x(a[0]);
    if (!x || x.rows < 1) Py_RETURN_NONE;
    at::Tensor q[4];
    void* p[4] = {};
    for (int t = 0; t < 2; ++t) {
        if (a[1 + t] != Py_True) continue;
        const int64_t r = t ? x.cols : x.rows, c = t ? x.rows : x.cols;
        q[2 * t] = empty({r, static_cast<int64_t>(mxfp4_data_bytes(1, c))}, at::kByte, *x.t);
        q[2 * t + 1] = empty({static_cast<int64_t>(mxfp4_scale_bytes(r, c))}, at::kByte, *x.t);
        p[2 * t] = q[2 * t].data_ptr();
        p[2 * t + 1] = q[2 * t + 1].data_ptr();
    }
    if (mxfp4_quantize(x.rows, x.cols, x.t->data_ptr(), x.code, x.cols, p[0], p[1], p[2], p[3], stream_of(*x.t))) Py_RETURN_NONE;
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, p[0] ? mx_tuple(std::move(q[0]), std::move(q[1]), x.rows, x.cols) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(r, 1, p[2] ? mx_tuple(std::move(q[2]), std::move(q[3]), x.cols, x.rows) : Py_NewRef(Py_None));
    return r;
    END_HANDLE_TH_ERRORS
}

// (q, out_dtype) -> y
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 2) Py_RETURN_NONE;
    const Mx q(a[0]);
    const int code = out_code(a[1], -1);
    if (!q || code < 0) Py_RETURN_NONE;
    at::Tensor y = empty({q.rows, q.cols}, type_of(code), *q.data);
    if (mxfp4_dequantize(q.rows, q.cols, q.data->data_ptr(), q.scales->data_ptr(), y.data_ptr(), code, stream_of(*q.data))) Py_RETURN_NONE;
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (a, b, bias, relu, out_dtype) -> y
PyObject* matmul(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const Mx a(v[0]), b(v[1]);
    const int code = out_code(v[4], -1);
    if (!a || !b || code < 0 || a.cols != b.cols || a.data->device() != b.data->device() || !PyBool_Check(v[3])) Py_RETURN_NONE;
    const float* bias;
    if (!vector(v[2], b.rows, *a.data, &bias)) Py_RETURN_NONE;
    at::Tensor y = empty({a.rows, b.rows}, type_of(code), *a.data);
    const mxfp4_matmul_params p{a.rows, b.rows, a.cols};
    const conv2d_epilogue epi{v[3] == Py_True ? CONV2D_ACT_RELU : CONV2D_ACT_NONE, code};
    if (mxfp4_matmul(&p, a.data->data_ptr(), a.scales->data_ptr(), b.data->data_ptr(), b.scales->data_ptr(), bias, y.data_ptr(), &epi,
                     stream_of(*a.data)))
        Py_RETURN_NONE;
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (x) -> (data, scales, rows, cols)
PyObject* quantize_int8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 1) Py_RETURN_NONE;
    const Rows x(a[0]);
    if (!x || x.rows < 1) Py_RETURN_NONE;
    const int64_t blocks = (x.cols + 31) / 32;
    at::Tensor data = empty({x.rows, 32 * blocks}, at::kChar, *x.t), scales = empty({x.rows, blocks}, at::kByte, *x.t);
    if (mxint8_quantize(x.rows, x.cols, x.t->data_ptr(), x.code, x.cols, data.data_ptr(), scales.data_ptr(), stream_of(*x.t))) Py_RETURN_NONE;
    return mx_tuple(std::move(data), std::move(scales), x.rows, x.cols);
    END_HANDLE_TH_ERRORS
}

// (q, out_dtype) -> y
PyObject* dequantize_int8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 2) Py_RETURN_NONE;
    const Mx8 q(a[0]);
    const int code = out_code(a[1], -1);
    if (!q || code < 0) Py_RETURN_NONE;
    at::Tensor y = empty({q.rows, q.cols}, type_of(code), *q.data);
    if (mxint8_dequantize(q.rows, q.cols, q.data->data_ptr(), q.scales->data_ptr(), y.data_ptr(), code, stream_of(*q.data))) Py_RETURN_NONE;
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (dy, x, mean, rstd, weight) -> (dx, dweight, dbias)
PyObject* norm_bwd_int8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5) Py_RETURN_NONE;
    const Rows dy(a[0]);
    const Mx8 x(a[1]);
    if (!dy || !x || dy.t->device() != x.data->device() || dy.rows != x.rows || dy.cols != x.cols || a[2] == Py_None || a[3] == Py_None)
        Py_RETURN_NONE;
    const float *mean, *rstd, *w;
    if (!vector(a[2], x.rows, *dy.t, &mean) || !vector(a[3], x.rows, *dy.t, &rstd) || !vector(a[4], x.cols, *dy.t, &w)) Py_RETURN_NONE;
    const layer_norm_params p{dy.rows, dy.cols, dy.cols, dy.cols, CONV2D_OUT_F32, dy.code, 0.f};
    const int64_t need = static_cast<int64_t>(mxint8_layer_norm_bwd_workspace_bytes(&p));
    at::Tensor dx = empty(dy.t->sizes(), dy.t->scalar_type(), *dy.t);
    at::Tensor dw = empty({dy.cols}, at::kFloat, *dy.t), db = empty({dy.cols}, at::kFloat, *dy.t), ws = empty({need}, at::kByte, *dy.t);
    if (mxint8_layer_norm_bwd(&p, dy.t->data_ptr(), x.data->data_ptr(), x.scales->data_ptr(), mean, rstd, w, dx.data_ptr(),
                              static_cast<float*>(dw.data_ptr()), static_cast<float*>(db.data_ptr()), ws.data_ptr(), static_cast<size_t>(need),
                              stream_of(*dy.t)))
        Py_RETURN_NONE;
    return tuple_of(std::move(dx), std::move(dw), std::move(db));
    END_HANDLE_TH_ERRORS
}

// (y, x, a, b, plan, scale, relu, out_dtype) -> (out, h)
PyObject* adapter_forward(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 8) Py_RETURN_NONE;
    const Rows y(v[0]), x(v[1]);
    if (!y || !x || x.code != CONV2D_OUT_BF16 || y.rows != x.rows || x.rows < 1 || y.t->device() != x.t->device() || !PyBool_Check(v[6]))
        Py_RETURN_NONE;
    const Plan plan(v[4], x.rows, *x.t);
    const int code = out_code(v[7], y.code);
    if (!plan || code < 0) Py_RETURN_NONE;
    const at::Tensor *a = tensor(v[2]), *b = tensor(v[3]);
    const int64_t rank = rank_of(a, b, plan.adapters, x.cols, y.cols, *x.t);
    const float* scale;
    if (rank < 1 || !vector(v[5], plan.adapters, *x.t, &scale)) Py_RETURN_NONE;
    at::Tensor out = empty(y.t->sizes(), type_of(code), *x.t), h = empty({x.rows, rank}, at::kFloat, *x.t);
    const adapter_fwd_params p{x.rows, x.cols, y.cols, rank, plan.adapters, x.cols, y.cols, y.cols, y.code, code,
                               v[6] == Py_True ? CONV2D_ACT_RELU : CONV2D_ACT_NONE};
    if (adapter_fwd(&p, plan.data->data_ptr(), y.t->data_ptr(), x.t->data_ptr(), a->data_ptr(), b->data_ptr(), scale, out.data_ptr(),
                    static_cast<float*>(h.data_ptr()), stream_of(*x.t)))
        Py_RETURN_NONE;
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, wrap(std::move(out)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(h)));
    return r;
    END_HANDLE_TH_ERRORS
}

// (dy, x, h, a, b, plan, scale, dx, out_dtype) -> (dx, da, db)
PyObject* adapter_backward(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 9) Py_RETURN_NONE;
    const Rows dy(v[0]), x16(v[1]);
    const Mx8 x8(v[1]);
    if (!dy || dy.code != CONV2D_OUT_BF16 || (!x8 && (!x16 || x16.code != CONV2D_OUT_BF16)) || dy.rows < 1) Py_RETURN_NONE;
    const int64_t cols = x8 ? x8.cols : x16.cols;
    if ((x8 ? x8.rows : x16.rows) != dy.rows || (x8 ? x8.data : x16.t)->device() != dy.t->device() || v[2] == Py_None) Py_RETURN_NONE;
    const Plan plan(v[5], dy.rows, *dy.t);
    if (!plan) Py_RETURN_NONE;
    const at::Tensor *a = tensor(v[3]), *b = tensor(v[4]), *dx0 = nullptr;
    const int64_t rank = rank_of(a, b, plan.adapters, cols, dy.cols, *dy.t);
    const float *scale, *h;
    if (rank < 1 || !vector(v[2], dy.rows * rank, *dy.t, &h) || !vector(v[6], plan.adapters, *dy.t, &scale)) Py_RETURN_NONE;
    int dx0_code = CONV2D_OUT_BF16;
    if (v[7] != Py_None) {
        const Rows base(v[7]);
        if (!base || base.rows != dy.rows || base.cols != cols || base.t->device() != dy.t->device()) Py_RETURN_NONE;
        dx0 = base.t;
        dx0_code = base.code;
    }
    const int code = out_code(v[8], dx0_code);
    if (code < 0) Py_RETURN_NONE;
    const adapter_bwd_params p{dy.rows, cols, dy.cols, rank, plan.adapters, dy.cols, cols, cols, cols, x8 ? ADAPTER_X_MXINT8 : ADAPTER_X_BF16,
                               dx0_code, code};
    const int64_t need = static_cast<int64_t>(adapter_bwd_workspace_bytes(&p));
    at::Tensor dx = dx0 ? empty(dx0->sizes(), type_of(code), *dy.t) : x8 ? empty({dy.rows, cols}, type_of(code), *dy.t) : empty(x16.t->sizes(), type_of(code), *dy.t);
    at::Tensor da = empty(a->sizes(), at::kFloat, *dy.t), db = empty(b->sizes(), at::kFloat, *dy.t), ws = empty({need}, at::kByte, *dy.t);
    if (adapter_bwd(&p, plan.data->data_ptr(), dy.t->data_ptr(), x8 ? x8.data->data_ptr() : x16.t->data_ptr(),
                    x8 ? x8.scales->data_ptr() : nullptr, h, a->data_ptr(), b->data_ptr(), scale, dx0 ? dx0->data_ptr() : nullptr, dx.data_ptr(),
                    static_cast<float*>(da.data_ptr()), static_cast<float*>(db.data_ptr()), ws.data_ptr(), static_cast<size_t>(need),
                    stream_of(*dy.t)))
        Py_RETURN_NONE;
    return tuple_of(std::move(dx), std::move(da), std::move(db));
    END_HANDLE_TH_ERRORS
}

// (Mxfp4, Mxint8, AdapterPlan): the types that these functions take.
PyObject* use(PyObject*, PyObject* const* types, Py_ssize_t n)
{
    PyObject** const known[3] = {&g_mxfp4, &g_mxint8, &g_plan};
    for (Py_ssize_t i = 0; i < n && i < 3; ++i) {
        Py_INCREF(types[i]);
        Py_XSETREF(*known[i], types[i]);
    }
    Py_RETURN_NONE;
}

#define FAST(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FAST("layer_norm_fwd", norm_fwd),
    FAST("layer_norm_bwd", norm_bwd),
    FAST("layer_norm_mxfp4", norm_mxfp4),
    FAST("quantize", quantize),
    FAST("dequantize", dequantize),
    FAST("matmul", matmul),
    FAST("quantize_int8", quantize_int8),
    FAST("dequantize_int8", dequantize_int8),
    FAST("mxint8_layer_norm_bwd", norm_bwd_int8),
    FAST("adapter_fwd", adapter_forward),
    FAST("adapter_bwd", adapter_backward),
    FAST("use", use),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
