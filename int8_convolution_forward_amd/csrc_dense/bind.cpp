// Python module of the dense entries: tensors to argument structures (operands
// whose layout has no such structure are copied by torch first), outputs
// and workspaces from torch's allocator on the current stream, the call.  It
// exists for the calls whose kernels take a few microseconds: marshalling
// through Python and ctypes took 6 to 10 us a call, this takes under 2.
//
// Every function returns its tensor(s), or an int: a status of conv_i8.h,
// kOperands where an operand is not a tensor on one GPU, or kRecorded where one
// takes part in automatic differentiation, which these calls do not record (the
// caller in Python then names it).  The entries' addresses are handed over once with bind(), so
// that the library stays the one that Python loaded.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Dtype.h>

#include <vector>

#include "dense.h"

namespace {

constexpr long kOperands = -1, kRecorded = -2;

struct Entries {
    decltype(&dense_linear) linear;
    decltype(&dense_linear_workspace_size) linear_size;
    decltype(&dense_linear_backward) linear_backward;
    decltype(&dense_linear_backward_workspace_size) linear_backward_size;
    decltype(&dense_layer_norm) norm;
    decltype(&dense_layer_norm_backward) norm_backward;
    decltype(&dense_layer_norm_backward_workspace_size) norm_backward_size;
    decltype(&dense_quantize) quantize;
    decltype(&dense_dequantize) dequantize;
    decltype(&dense_linear_fp8) linear_fp8;
    decltype(&dense_linear_fp8_workspace_size) linear_fp8_size;
    decltype(&dense_linear_fp8_backward) linear_fp8_backward;
    decltype(&dense_linear_fp8_backward_workspace_size) linear_fp8_backward_size;
    decltype(&dense_residual_norm) residual_norm;
    decltype(&dense_residual_norm_backward) residual_norm_backward;
    decltype(&dense_residual_norm_backward_workspace_size) residual_norm_backward_size;
    decltype(&dense_clip_grads) clip;
    decltype(&dense_clip_grads_workspace_size) clip_size;
} entries;

int64_t code_of(at::ScalarType t)
{
    switch (t) {
    case at::kChar: return DENSE_INT8;
    case at::kBFloat16: return DENSE_BF16;
    case at::kHalf: return DENSE_FP16;
    case at::kFloat: return DENSE_FP32;
    case at::kFloat8_e4m3fn: return DENSE_E4M3;
    case at::kFloat8_e5m2: return DENSE_E5M2;
    case at::kFloat8_e8m0fnu: return DENSE_E8M0;
    default: return 99;  // a type the entries refuse
    }
}

// A status that ends the call
struct Stop { long code; };

// Tensors of the call: each has to be on the first one's GPU, and none may
// expect its gradient to be recorded.  `copies` keeps those of operands that the
// entries do not take as they are.
struct Args {
    c10::Device device{c10::kCPU};
    const bool grad = c10::GradMode::is_enabled();
    c10::SmallVector<at::Tensor, 16> copies;  // two for each of up to eight operands: it never moves them

    const at::Tensor *keep(at::Tensor t) { return &copies.emplace_back(std::move(t)); }

    const at::Tensor *get(PyObject *o, bool needed, bool output = false)
    {
        if (o == Py_None && !needed)
            return nullptr;
        if (!THPVariable_Check(o))
            throw Stop{kOperands};
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || (device.is_cuda() && t.device() != device))
            throw Stop{kOperands};
        if ((grad && t.requires_grad()) || t._fw_grad(0).defined())
            throw Stop{kRecorded};
        device = t.device();
        if (t.is_neg()) {  // a view that stands for the negatives of what lies in memory
            if (output)
                throw Stop{CONV_I8_ERR_UNSUPPORTED};
            return keep(t.resolve_neg());
        }
        return &t;
    }
};

// The tensor as a matrix, if its leading dims merge into rows of one stride
bool as_rows(const at::Tensor &t, dense_mat_t *m)
{
    const auto sizes = t.sizes(), strides = t.strides();
    const int64_t d = t.dim();
    if (d < 1)
        throw Stop{CONV_I8_ERR_RANK};
    m->ptr = t.data_ptr();
    m->dtype = code_of(t.scalar_type());
    m->cols = sizes[d - 1];
    m->col_stride = strides[d - 1];
    m->rows = 1;
    m->row_stride = m->cols;
    bool first = true;
    for (int64_t i = d - 2; i >= 0; --i) {
        if (sizes[i] == 1)
            continue;
        if (first)
            m->row_stride = strides[i];
        else if (strides[i] != m->row_stride * m->rows && t.numel() != 0)
            return false;
        m->rows *= sizes[i];
        first = false;
    }
    return true;
}

// An output, or an operand that was made here
dense_mat_t rows_of(const at::Tensor *t)
{
    dense_mat_t m{};
    if (t && !as_rows(*t, &m))
        throw Stop{CONV_I8_ERR_STRIDES};
    return m;
}

// An operand: copied where its leading dims do not merge (a transposed batch) or
// `packed_cols` asks for a contiguous last dim that it does not have (a gradient
// expanded from one number).
dense_mat_t rows_in(Args &in, const at::Tensor *t, bool packed_cols)
{
    dense_mat_t m{};
    if (t && (!as_rows(*t, &m) || (packed_cols && m.col_stride != 1 && m.cols > 1)))
        as_rows(*in.keep(t->contiguous()), &m);
    return m;
}

dense_mat_t matrix_of(const at::Tensor *t)
{
    if (t && t->dim() != 2)
        throw Stop{CONV_I8_ERR_RANK};
    return rows_of(t);
}

// A contiguous vector, one made here or (vec_in) an operand, copied if it has a
// stride; `any_shape` for values that go with the rows
dense_vec_t vec_of(const at::Tensor *t, bool any_shape = false)
{
    dense_vec_t v{};
    if (!t)
        return v;
    if ((!any_shape && t->dim() != 1) || !t->is_contiguous())
        throw Stop{CONV_I8_ERR_STRIDES};
    v.ptr = t->data_ptr();
    v.n = t->numel();
    v.dtype = code_of(t->scalar_type());
    return v;
}

dense_vec_t vec_in(Args &in, const at::Tensor *t, bool any_shape = false)
{
    return vec_of(t && !t->is_contiguous() ? in.keep(t->contiguous()) : t, any_shape);
}

void check(long code)
{
    if (code != CONV_I8_OK)
        throw Stop{code};
}

// torch's allocator without its dispatcher
at::Tensor empty(at::IntArrayRef shape, at::ScalarType t, c10::Device d)
{
    return at::Tensor(at::detail::empty_cuda(shape, t, d, std::nullopt));
}

// Tells autograd that the caller's tensor was written: a graph that saved it
// then raises instead of using the new values
void written(const at::Tensor *t)
{
    if (t && !t->is_inference())
        t->unsafeGetTensorImpl()->bump_version();
}

// x's leading shape with another last dim
c10::SmallVector<int64_t, 6> shape_of(const at::Tensor &x, int64_t last)
{
    c10::SmallVector<int64_t, 6> s(x.sizes().begin(), x.sizes().end());
    s.back() = last;
    return s;
}

template <typename A>
void run(const A &a, conv_i8_status_t (*size)(const A *, size_t *),
         conv_i8_status_t (*entry)(const A *, void *, size_t, void *), c10::Device d)
{
    size_t n = 0;
    check(size(&a, &n));
    void *stream = c10::hip::getCurrentHIPStream(d.index()).stream();
    if (n == 0) {
        check(entry(&a, nullptr, 0, stream));
    } else {
        const at::Tensor ws = empty({(int64_t)n}, at::kByte, d);
        check(entry(&a, ws.data_ptr(), n, stream));
    }
}

// Runs f; an error of the arguments becomes an int, any C++ exception a Python one
template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const Stop &s) {
        return PyLong_FromLong(s.code);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want)
        return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

PyObject *wrap(const at::Tensor &t)
{
    if (t.defined())
        return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject *tuple(std::initializer_list<at::Tensor> ts)
{
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r)
        return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// linear(x, w, bias, activation, residual, x_scale, w_scale, out_dtype, preact, out)
PyObject *linear(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 10))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *x = in.get(o[0], true), *w = in.get(o[1], true), *bias = in.get(o[2], false);
        const at::Tensor *res = in.get(o[4], false), *xs = in.get(o[5], false), *ws = in.get(o[6], false);
        const at::Tensor *pre = in.get(o[8], false, true), *out = in.get(o[9], false, true);
        const c10::DeviceGuard guard(in.device);
        dense_linear_t a{};
        a.x = rows_in(in, x, false);
        a.w = matrix_of(w);
        a.residual = rows_in(in, res, true);
        a.preact = rows_of(pre);
        a.bias = vec_in(in, bias);
        a.x_scale = vec_in(in, xs, true);
        a.w_scale = vec_in(in, ws);
        a.activation = PyLong_AsLongLong(o[3]);
        at::Tensor y;
        if (out) {
            if (o[7] != Py_None && (!THPDtype_Check(o[7]) || ((THPDtype *)o[7])->scalar_type != out->scalar_type()))
                throw Stop{CONV_I8_ERR_DTYPE};
            y = *out;
        } else {
            at::ScalarType t = x->scalar_type() == at::kChar ? at::kBFloat16 : x->scalar_type();
            if (o[7] != Py_None) {
                if (!THPDtype_Check(o[7]))
                    throw Stop{CONV_I8_ERR_DTYPE};
                t = ((THPDtype *)o[7])->scalar_type;
            }
            y = empty(shape_of(*x, a.w.rows), t, in.device);
        }
        a.y = rows_of(&y);
        run(a, entries.linear_size, entries.linear, in.device);
        written(out);
        written(pre);
        return wrap(y);
    });
}

// linear_backward(dy, x, w, preact, activation, need_dx, need_dw, need_dbias)
PyObject *linear_backward(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 8))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *dy = in.get(o[0], true), *x = in.get(o[1], true), *w = in.get(o[2], true);
        const at::Tensor *z = in.get(o[3], false);
        const c10::DeviceGuard guard(in.device);
        dense_linear_backward_t a{};
        a.activation = PyLong_AsLongLong(o[4]);
        a.dy = rows_in(in, dy, true);
        a.x = rows_in(in, x, false);
        a.w = matrix_of(w);
        if (a.activation != DENSE_ACT_NONE)
            a.preact = rows_in(in, z, true);
        const at::ScalarType t = dy->scalar_type();
        at::Tensor dx, dw, db;
        if (o[5] == Py_True) {
            dx = empty(x->sizes(), t, in.device);
            a.dx = rows_of(&dx);
        }
        if (o[6] == Py_True) {
            dw = empty(w->sizes(), t, in.device);
            a.dw = rows_of(&dw);
        }
        if (o[7] == Py_True) {
            db = empty({a.w.rows}, t, in.device);
            a.dbias = vec_of(&db);
        }
        run(a, entries.linear_backward_size, entries.linear_backward, in.device);
        return tuple({dx, dw, db});
    });
}

// layer_norm(x, weight, bias, eps, as_int8): (y, mean, rstd) or (q, scale)
PyObject *layer_norm(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 5))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *x = in.get(o[0], true), *w = in.get(o[1], false), *b = in.get(o[2], false);
        const c10::DeviceGuard guard(in.device);
        dense_layer_norm_t a{};
        a.x = rows_in(in, x, true);
        a.weight = vec_in(in, w);
        a.bias = vec_in(in, b);
        a.eps = PyFloat_AsDouble(o[3]);
        if (PyErr_Occurred())
            return nullptr;
        const bool q8 = o[4] == Py_True;
        const auto lead = x->sizes().slice(0, x->dim() - 1);
        const at::Tensor y = empty(x->sizes(), q8 ? at::kChar : x->scalar_type(), in.device);
        const at::Tensor s0 = empty(lead, at::kFloat, in.device);
        at::Tensor s1;
        a.y = rows_of(&y);
        if (q8) {
            a.scale = vec_of(&s0, true);
        } else {
            s1 = empty(lead, at::kFloat, in.device);
            a.mean = vec_of(&s0, true);
            a.rstd = vec_of(&s1, true);
        }
        check(entries.norm(&a, c10::hip::getCurrentHIPStream(in.device.index()).stream()));
        return q8 ? tuple({y, s0}) : tuple({y, s0, s1});
    });
}

// layer_norm_backward(dy, x, weight, mean, rstd, need_params)
PyObject *layer_norm_backward(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 6))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *dy = in.get(o[0], true), *x = in.get(o[1], true), *w = in.get(o[2], false);
        const at::Tensor *mean = in.get(o[3], true), *rstd = in.get(o[4], true);
        const c10::DeviceGuard guard(in.device);
        dense_layer_norm_backward_t a{};
        a.dy = rows_in(in, dy, true);
        a.x = rows_in(in, x, true);
        a.weight = vec_in(in, w);
        a.mean = vec_in(in, mean, true);
        a.rstd = vec_in(in, rstd, true);
        const at::Tensor dx = empty(x->sizes(), x->scalar_type(), in.device);
        at::Tensor dw, db;
        a.dx = rows_of(&dx);
        if (o[5] == Py_True) {
            dw = empty({a.x.cols}, x->scalar_type(), in.device);
            db = empty({a.x.cols}, x->scalar_type(), in.device);
            a.dweight = vec_of(&dw);
            a.dbias = vec_of(&db);
        }
        run(a, entries.norm_backward_size, entries.norm_backward, in.device);
        return tuple({dx, dw, db});
    });
}

constexpr int64_t kBlock = 128;
int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// quantize(x, tiles, transposed, dtype): (q, scale) or (q, scale, qt, scale_t)
PyObject *quantize(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 4))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *x = in.get(o[0], true);
        const bool tiles = o[1] == Py_True, both = o[2] == Py_True;
        if (!THPDtype_Check(o[3]))
            throw Stop{CONV_I8_ERR_DTYPE};
        const at::ScalarType type = ((THPDtype *)o[3])->scalar_type;
        if (type != at::kFloat8_e4m3fn && type != at::kFloat8_e5m2)
            throw Stop{CONV_I8_ERR_DTYPE};
        if (x->dim() < 1)
            throw Stop{CONV_I8_ERR_RANK};
        const c10::DeviceGuard guard(in.device);
        dense_quantize_t a{};
        a.x = rows_in(in, x, true);
        const int64_t M = a.x.rows, K = a.x.cols;
        const auto e8 = at::kFloat8_e8m0fnu;
        const at::Tensor q = empty(x->sizes(), type, in.device);
        const at::Tensor s = tiles ? empty({blocks_of(M), blocks_of(K)}, e8, in.device)
                                   : empty(shape_of(*x, blocks_of(K)), e8, in.device);
        a.q = rows_of(&q);
        a.scale = rows_of(&s);
        if (!both) {
            check(entries.quantize(&a, c10::hip::getCurrentHIPStream(in.device.index()).stream()));
            return tuple({q, s});
        }
        const at::Tensor qt = empty({K, M}, type, in.device);
        const at::Tensor st = empty({tiles ? blocks_of(K) : K, blocks_of(M)}, e8, in.device);
        a.qt = rows_of(&qt);
        a.scale_t = rows_of(&st);
        check(entries.quantize(&a, c10::hip::getCurrentHIPStream(in.device.index()).stream()));
        return tuple({q, s, qt, st});
    });
}

// dequantize(q, scale, dtype)
PyObject *dequantize(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 3))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *q = in.get(o[0], true), *s = in.get(o[1], true);
        if (!THPDtype_Check(o[2]))
            throw Stop{CONV_I8_ERR_DTYPE};
        const c10::DeviceGuard guard(in.device);
        dense_dequantize_t a{};
        a.q = rows_in(in, q, true);
        a.scale = rows_in(in, s, true);
        const at::Tensor x = empty(q->sizes(), ((THPDtype *)o[2])->scalar_type, in.device);
        a.x = rows_of(&x);
        check(entries.dequantize(&a, c10::hip::getCurrentHIPStream(in.device.index()).stream()));
        return wrap(x);
    });
}

// linear_fp8(x, w, x_scale, w_scale, bias, activation, residual, out_dtype, preact, out)
PyObject *linear_fp8(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 10))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *x = in.get(o[0], true), *w = in.get(o[1], true), *xs = in.get(o[2], true), *ws = in.get(o[3], true);
        const at::Tensor *bias = in.get(o[4], false), *res = in.get(o[6], false);
        const at::Tensor *pre = in.get(o[8], false, true), *out = in.get(o[9], false, true);
        const c10::DeviceGuard guard(in.device);
        dense_linear_fp8_t a{};
        at::ScalarType t = out ? out->scalar_type() : at::kBFloat16;
        if (o[7] != Py_None) {
            if (!THPDtype_Check(o[7]) || (out && ((THPDtype *)o[7])->scalar_type != t))
                throw Stop{CONV_I8_ERR_DTYPE};
            t = ((THPDtype *)o[7])->scalar_type;
        }
        const bool packed = t == at::kFloat;  // what a 32-bit result asks of x and w
        matrix_of(w);
        matrix_of(ws);
        a.x = rows_in(in, x, packed);
        a.w = rows_in(in, w, packed);
        a.x_scale = rows_in(in, xs, true);
        a.w_scale = rows_in(in, ws, true);
        a.residual = rows_in(in, res, true);
        a.preact = rows_of(pre);
        a.bias = vec_in(in, bias);
        a.activation = PyLong_AsLongLong(o[5]);
        const at::Tensor y = out ? *out : empty(shape_of(*x, a.w.rows), t, in.device);
        a.y = rows_of(&y);
        run(a, entries.linear_fp8_size, entries.linear_fp8, in.device);
        written(out);
        written(pre);
        return wrap(y);
    });
}

// linear_fp8_backward(dy, xt, xt_scale, wt, wt_scale, preact, activation, need_dx, need_dw, need_dbias, g_dtype)
PyObject *linear_fp8_backward(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 11))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const bool dx_on = o[7] == Py_True, dw_on = o[8] == Py_True;
        const at::Tensor *dy = in.get(o[0], true), *xt = in.get(o[1], dw_on), *xts = in.get(o[2], dw_on);
        const at::Tensor *wt = in.get(o[3], dx_on), *wts = in.get(o[4], dx_on), *z = in.get(o[5], false);
        const c10::DeviceGuard guard(in.device);
        if (!THPDtype_Check(o[10]))
            throw Stop{CONV_I8_ERR_DTYPE};
        dense_linear_fp8_backward_t a{};
        a.activation = PyLong_AsLongLong(o[6]);
        a.g_dtype = code_of(((THPDtype *)o[10])->scalar_type);
        a.dy = rows_in(in, dy, true);
        if (a.activation != DENSE_ACT_NONE)
            a.preact = rows_in(in, z, true);
        const at::ScalarType t = dy->scalar_type();
        at::Tensor dx, dw, db;
        if (dw_on) {
            a.xt = matrix_of(xt);
            matrix_of(xts);
            a.xt_scale = rows_in(in, xts, true);
            dw = empty({a.dy.cols, a.xt.rows}, t, in.device);
            a.dw = rows_of(&dw);
        }
        if (dx_on) {
            a.wt = matrix_of(wt);
            matrix_of(wts);
            a.wt_scale = rows_in(in, wts, true);
            dx = empty(shape_of(*dy, a.wt.rows), t, in.device);
            a.dx = rows_of(&dx);
        }
        if (o[9] == Py_True) {
            db = empty({a.dy.cols}, t, in.device);
            a.dbias = vec_of(&db);
        }
        run(a, entries.linear_fp8_backward_size, entries.linear_fp8_backward, in.device);
        return tuple({dx, dw, db});
    });
}

// Vector i of `count` that lie one after the other in a contiguous tensor of 32-bit values
dense_vec_t part_of(const at::Tensor *t, int64_t i, int64_t count)
{
    dense_vec_t v{};
    if (!t || t->numel() % count != 0)
        throw Stop{CONV_I8_ERR_DIMS};
    v.n = t->numel() / count;
    v.ptr = (const char *)t->data_ptr() + i * v.n * (int64_t)t->element_size();
    v.dtype = code_of(t->scalar_type());
    return v;
}

// residual_norm(x, h, weight, bias, gate, post_weight, scale, kind, eps, as_fp8): (r, y, stats) or (r, q, scale)
PyObject *residual_norm(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 10))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *x = in.get(o[0], true), *h = in.get(o[1], false), *w = in.get(o[2], false), *b = in.get(o[3], false);
        const at::Tensor *gate = in.get(o[4], false), *pw = in.get(o[5], false);
        const c10::DeviceGuard guard(in.device);
        dense_residual_norm_t a{};
        a.x = rows_in(in, x, true);
        a.h = rows_in(in, h, true);
        a.gate = rows_in(in, gate, true);
        a.weight = vec_in(in, w);
        a.bias = vec_in(in, b);
        a.post_weight = vec_in(in, pw);
        a.alpha = PyFloat_AsDouble(o[6]);
        a.kind = PyLong_AsLongLong(o[7]);
        a.eps = PyFloat_AsDouble(o[8]);
        if (PyErr_Occurred())
            return nullptr;
        if (h && h->sizes() != x->sizes())
            throw Stop{CONV_I8_ERR_DIMS};
        const bool q8 = o[9] == Py_True;
        at::Tensor r = *x;
        if (h) {
            r = empty(x->sizes(), x->scalar_type(), in.device);
            a.r = rows_of(&r);
        }
        const at::Tensor y = empty(x->sizes(), q8 ? at::kFloat8_e4m3fn : x->scalar_type(), in.device);
        a.y = rows_of(&y);
        at::Tensor s;
        if (q8) {
            s = empty(shape_of(*x, blocks_of(a.x.cols)), at::kFloat8_e8m0fnu, in.device);
            a.y_scale = rows_of(&s);
        } else {
            c10::SmallVector<int64_t, 6> shape{pw ? 4 : 2};
            shape.append(x->sizes().begin(), x->sizes().end() - 1);
            s = empty(shape, at::kFloat, in.device);
            a.mean = part_of(&s, 0, shape[0]);
            a.rstd = part_of(&s, 1, shape[0]);
            if (pw) {
                a.post_mean = part_of(&s, 2, 4);
                a.post_rstd = part_of(&s, 3, 4);
            }
        }
        check(entries.residual_norm(&a, c10::hip::getCurrentHIPStream(in.device.index()).stream()));
        return tuple({r, y, s});
    });
}

// residual_norm_backward(dr, dy, r, h, stats, weight, gate, post_weight, scale, kind, need_params):
// (dx, dh, dweight, dbias, dgate, dpost_weight)
PyObject *residual_norm_backward(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 11))
        return nullptr;
    return guarded([&]() -> PyObject * {
        Args in;
        const at::Tensor *dr = in.get(o[0], false), *dy = in.get(o[1], true), *r = in.get(o[2], true), *h = in.get(o[3], false);
        const at::Tensor *stats = in.get(o[4], true), *w = in.get(o[5], false), *gate = in.get(o[6], false);
        const at::Tensor *pw = in.get(o[7], false);
        const c10::DeviceGuard guard(in.device);
        dense_residual_norm_backward_t a{};
        a.dr = rows_in(in, dr, true);
        a.dy = rows_in(in, dy, true);
        a.r = rows_in(in, r, true);
        a.h = rows_in(in, h, true);
        a.gate = rows_in(in, gate, true);
        a.weight = vec_in(in, w);
        a.post_weight = vec_in(in, pw);
        a.alpha = PyFloat_AsDouble(o[8]);
        a.kind = PyLong_AsLongLong(o[9]);
        if (PyErr_Occurred())
            return nullptr;
        if (!stats->is_contiguous())
            stats = in.keep(stats->contiguous());
        const int64_t parts = pw ? 4 : 2;
        a.mean = part_of(stats, 0, parts);
        a.rstd = part_of(stats, 1, parts);
        if (pw) {
            a.post_mean = part_of(stats, 2, parts);
            a.post_rstd = part_of(stats, 3, parts);
        }
        const at::ScalarType t = r->scalar_type();
        const at::Tensor dx = empty(r->sizes(), t, in.device);
        at::Tensor dh, dw, db, dg, dp;
        a.dx = rows_of(&dx);
        if (h) {
            dh = empty(r->sizes(), t, in.device);
            a.dh = rows_of(&dh);
        }
        if (o[10] == Py_True) {
            dw = empty({a.r.cols}, t, in.device);
            db = empty({a.r.cols}, t, in.device);
            a.dweight = vec_of(&dw);
            a.dbias = vec_of(&db);
            if (gate) {
                dg = empty(gate->sizes(), t, in.device);
                a.dgate = rows_of(&dg);
            }
            if (pw) {
                dp = empty({a.r.cols}, t, in.device);
                a.dpost_weight = vec_of(&dp);
            }
        }
        run(a, entries.residual_norm_backward_size, entries.residual_norm_backward, in.device);
        return tuple({dx, dh, dw, db, dg, dp});
    });
}

// clip_grad_norm(grads, max_norm, out or None), both sequences of tensors: the norm
PyObject *clip_grad_norm(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    if (!arity(n, 3))
        return nullptr;
    PyObject *given = PySequence_Fast(o[0], "grads: expected a sequence of tensors");
    if (!given)
        return nullptr;
    PyObject *outs = o[2] == Py_None ? nullptr : PySequence_Fast(o[2], "out: expected a sequence of tensors");
    PyObject *r = nullptr;
    if (outs || o[2] == Py_None) {
        r = guarded([&]() -> PyObject * {
            Args in;
            const Py_ssize_t count = PySequence_Fast_GET_SIZE(given);
            if (outs && PySequence_Fast_GET_SIZE(outs) != count)
                throw Stop{CONV_I8_ERR_OUT_DIMS};
            std::vector<dense_vec_t> a(count), b(count);
            std::vector<const at::Tensor *> to(count);
            auto flat = [](const at::Tensor &t) {
                if (!t.is_non_overlapping_and_dense())
                    throw Stop{CONV_I8_ERR_STRIDES};
                dense_vec_t v{};
                v.ptr = t.data_ptr();
                v.n = t.numel();
                v.dtype = code_of(t.scalar_type());
                return v;
            };
            for (Py_ssize_t i = 0; i < count; ++i) {
                const at::Tensor *g = in.get(PySequence_Fast_GET_ITEM(given, i), true, true);
                to[i] = outs ? in.get(PySequence_Fast_GET_ITEM(outs, i), true, true) : g;
                if (to[i]->sizes() != g->sizes())
                    throw Stop{CONV_I8_ERR_OUT_DIMS};
                for (int64_t d = 0; d < g->dim(); ++d)  // strides of dims of one mean nothing
                    if (g->size(d) > 1 && g->numel() > 0 && to[i]->stride(d) != g->stride(d))
                        throw Stop{CONV_I8_ERR_STRIDES};
                a[i] = flat(*g);
                b[i] = flat(*to[i]);
            }
            if (count == 0)
                throw Stop{kOperands};
            const c10::DeviceGuard guard(in.device);
            const at::Tensor norm = empty({}, at::kFloat, in.device);
            dense_clip_grads_t c{};
            c.in = a.data();
            c.out = b.data();
            c.count = count;
            c.max_norm = PyFloat_AsDouble(o[1]);
            if (PyErr_Occurred())
                return nullptr;
            c.norm = norm.data_ptr<float>();
            run(c, entries.clip_size, entries.clip, in.device);
            for (const at::Tensor *t : to)
                written(t);
            return wrap(norm);
        });
    }
    Py_DECREF(given);
    Py_XDECREF(outs);
    return r;
}

// bind(the addresses in the order of Entries)
PyObject *bind(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    void **p = (void **)&entries;
    constexpr int count = sizeof entries / sizeof(void *);
    if (!arity(n, count))
        return nullptr;
    for (int i = 0; i < count; ++i) {
        p[i] = PyLong_AsVoidPtr(o[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(linear), FAST(linear_backward), FAST(layer_norm), FAST(layer_norm_backward),
                         FAST(quantize), FAST(dequantize), FAST(linear_fp8), FAST(linear_fp8_backward), FAST(residual_norm),
                         FAST(residual_norm_backward), FAST(clip_grad_norm), FAST(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense(void) { return PyModule_Create(&module); }
