// ecc_torch.cpp -- argument marshalling of the language-model operators for
// PyTorch tensors: reads the tensors' pointers, shapes, strides and types,
// checks them, allocates outputs and scratch through PyTorch's caching
// allocator on the current stream, and calls the C ABI (include/ecc_lm.h),
// which does the rest.  A Python module of positional functions; the
// documented entry points in __init__.py give the defaults.  (The same
// marshalling in Python took 10 to 15 us a call, several times what the
// smallest kernels run.)

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <vector>

#include "ecc_lm.h"

namespace {

PyObject *g_error = nullptr; // EccError

struct Refused {}; // a Python error is set

[[noreturn]] void refuse(const char *what, int code = ECC_ERR_ARG)
{
    PyObject *e = g_error ? PyObject_CallFunction(g_error, "is", code, what) : nullptr;
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, what);
    }
    throw Refused{};
}
void check(ecc_status code, const char *what)
{
    if (code != ECC_OK)
        refuse(what, code);
}

uint32_t type_of(at::ScalarType t, const char *what)
{
    switch (t) {
    case at::kFloat:
        return ECC_F32;
    case at::kBFloat16:
        return ECC_BF16;
    case at::kHalf:
        return ECC_F16;
    case at::kFloat8_e4m3fn:
    case at::kByte: // the coders' bytes
        return ECC_E4M3;
    default:
        refuse(what);
    }
}

using Opt = const at::Tensor *; // NULL: None

Opt tensor(PyObject *o, const char *what)
{
    if (o == Py_None)
        return nullptr;
    if (!THPVariable_Check(o))
        refuse(what);
    return &THPVariable_Unpack(o);
}
const at::Tensor &first(PyObject *o, const char *what)
{
    Opt t = tensor(o, what);
    if (!t || !t->is_cuda())
        refuse(what);
    return *t;
}
std::optional<at::ScalarType> dtype(PyObject *o, const char *what)
{
    if (o == Py_None)
        return std::nullopt;
    if (!THPDtype_Check(o))
        refuse(what);
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}
double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Refused{};
    return v;
}
long integer(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Refused{};
    return v;
}

// a tensor of rows: the last dimension contiguous, the leading ones with one stride
struct Matrix {
    void *p = nullptr;
    uint64_t rows = 0, cols = 0, ld = 0;
    uint32_t type = 0;
};
Matrix matrix(const at::Tensor &t, c10::Device dev, const char *what)
{
    const auto size = t.sizes(), stride = t.strides();
    const int64_t n = (int64_t)size.size();
    if (n == 0 || t.device() != dev)
        refuse(what);
    Matrix m;
    m.cols = (uint64_t)size[n - 1];
    int64_t rows = 1, ld = size[n - 1];
    bool empty = false; // no rows: whatever the strides
    for (int64_t i = 0; i < n - 1; ++i)
        empty |= size[i] == 0;
    if (empty) {
        rows = 0;
    } else {
        if (size[n - 1] > 1 && stride[n - 1] != 1)
            refuse(what);
        for (int64_t i = n - 2; i >= 0; --i) {
            if (size[i] == 1)
                continue;
            if (rows == 1)
                ld = stride[i];
            else if (stride[i] != rows * ld)
                refuse(what);
            rows *= size[i];
        }
    }
    m.rows = (uint64_t)rows;
    m.ld = rows > 1 ? (uint64_t)ld : m.cols;
    m.type = type_of(t.scalar_type(), what);
    m.p = t.data_ptr();
    return m;
}
Matrix operand(Opt t, uint64_t rows, uint64_t cols, c10::Device dev, const char *what)
{
    if (!t)
        return {};
    const Matrix m = matrix(*t, dev, what);
    if (m.rows != rows || m.cols != cols)
        refuse(what);
    return m;
}
// pointer of a contiguous vector of n elements
void *vector(Opt t, uint64_t n, c10::Device dev, const char *what, std::optional<at::ScalarType> type = std::nullopt)
{
    if (!t)
        return nullptr;
    if ((uint64_t)t->numel() != n || !t->is_contiguous() || t->device() != dev || (type && t->scalar_type() != *type))
        refuse(what);
    return t->data_ptr();
}

at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, c10::Device dev)
{
    return at::detail::empty_cuda(size, type, dev, std::nullopt);
}
// `given`, or a new tensor
at::Tensor output(Opt given, at::IntArrayRef size, at::ScalarType type, c10::Device dev)
{
    return given ? *given : fresh(size, type, dev);
}
// (a given one is written from its first byte on, as far as it is long)
at::Tensor scratch(Opt given, size_t bytes, c10::Device dev, const char *what)
{
    if (given && (given->device() != dev || !given->is_contiguous()))
        refuse(what);
    return given ? *given : bytes ? fresh({(int64_t)bytes}, at::kByte, dev) : at::Tensor();
}
void *where(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes_of(const at::Tensor &t) { return t.defined() ? t.nbytes() : 0; }

PyObject *wrap(const at::Tensor &t)
{
    if (t.defined())
        return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <typename... T> PyObject *results(const T &...t)
{
    PyObject *o = PyTuple_New(sizeof...(t));
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(o, i++, wrap(t)), ...);
    return o;
}

// the current stream of x's device, current while the call runs
struct On {
    c10::Device dev;
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit On(const at::Tensor &x)
        : dev(x.device()), guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream())
    {
    }
};

// torch.OutOfMemoryError, as for torch's own allocations
void out_of_memory(const char *what)
{
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *cls = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (cls)
        PyErr_SetString(cls, what);
    Py_XDECREF(cls);
    Py_XDECREF(torch);
}

#define FUNCTION(name, count)                                                                                          \
    PyObject *name##_body(PyObject *const *a);                                                                         \
    PyObject *name(PyObject *, PyObject *const *a, Py_ssize_t n)                                                       \
    {                                                                                                                  \
        if (n != count) {                                                                                              \
            PyErr_SetString(PyExc_TypeError, #name ": wrong number of arguments");                                     \
            return nullptr;                                                                                            \
        }                                                                                                              \
        try {                                                                                                          \
            return name##_body(a);                                                                                     \
        } catch (const Refused &) {                                                                                    \
        } catch (const c10::OutOfMemoryError &e) {                                                                     \
            out_of_memory(e.what_without_backtrace());                                                                 \
        } catch (const std::exception &e) {                                                                            \
            PyErr_SetString(PyExc_RuntimeError, e.what());                                                             \
        }                                                                                                              \
        return nullptr;                                                                                                \
    }                                                                                                                  \
    PyObject *name##_body(PyObject *const *a)

// x, weight, bias, eps, out, out_dtype, out_scale, mean, rstd
FUNCTION(layer_norm, 9)
{
    const at::Tensor &x = first(a[0], "ecc_layer_norm: needs CUDA tensors");
    const On on(x);
    const Matrix mx = matrix(x, on.dev, "ecc_layer_norm: x");
    Opt weight = tensor(a[1], "ecc_layer_norm: weight"), bias = tensor(a[2], "ecc_layer_norm: bias");
    const at::ScalarType p_type = weight ? weight->scalar_type() : bias ? bias->scalar_type() : x.scalar_type();
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    at::Tensor out = output(tensor(a[4], "ecc_layer_norm: out"), x.sizes(),
                            dtype(a[5], "ecc_layer_norm: out_dtype").value_or(x.scalar_type()), on.dev);
    if (out.sizes() != x.sizes())
        refuse("ecc_layer_norm: out");
    const Matrix my = matrix(out, on.dev, "ecc_layer_norm: out");
    at::Tensor mean = output(tensor(a[7], "ecc_layer_norm: mean"), lead, at::kFloat, on.dev);
    at::Tensor rstd = output(tensor(a[8], "ecc_layer_norm: rstd"), lead, at::kFloat, on.dev);
    check(ecc_layer_norm(mx.p, mx.ld, mx.type, vector(weight, mx.cols, on.dev, "ecc_layer_norm: weight"),
                         vector(bias, mx.cols, on.dev, "ecc_layer_norm: bias", p_type),
                         type_of(p_type, "ecc_layer_norm: weight type"), mx.rows, mx.cols, (float)number(a[3]), my.p, my.ld,
                         my.type, (float)number(a[6]),
                         (float *)vector(&mean, mx.rows, on.dev, "ecc_layer_norm: mean", at::kFloat),
                         (float *)vector(&rstd, mx.rows, on.dev, "ecc_layer_norm: rstd", at::kFloat), on.stream),
          "ecc_layer_norm");
    return results(out, mean, rstd);
}

// dy, x, weight, mean, rstd, dx, dweight, dbias, ws
FUNCTION(layer_norm_grad, 9)
{
    const at::Tensor &dy = first(a[0], "ecc_layer_norm_grad: needs CUDA tensors");
    const On on(dy);
    const at::Tensor &x = first(a[1], "ecc_layer_norm_grad: x");
    if (x.sizes() != dy.sizes() || x.scalar_type() != dy.scalar_type())
        refuse("ecc_layer_norm_grad: x");
    const Matrix md = matrix(dy, on.dev, "ecc_layer_norm_grad: dy"), mx = matrix(x, on.dev, "ecc_layer_norm_grad: x");
    Opt weight = tensor(a[2], "ecc_layer_norm_grad: weight");
    Opt mean = tensor(a[3], "ecc_layer_norm_grad: mean"), rstd = tensor(a[4], "ecc_layer_norm_grad: rstd");
    if (!mean || !rstd)
        refuse("ecc_layer_norm_grad: mean and rstd");
    at::Tensor dx = output(tensor(a[5], "ecc_layer_norm_grad: dx"), x.sizes(), x.scalar_type(), on.dev);
    if (dx.sizes() != x.sizes() || dx.scalar_type() != x.scalar_type())
        refuse("ecc_layer_norm_grad: dx");
    const Matrix mo = matrix(dx, on.dev, "ecc_layer_norm_grad: dx");
    const int64_t cols = (int64_t)mx.cols;
    at::Tensor dw = output(tensor(a[6], "ecc_layer_norm_grad: dweight"), {cols}, at::kFloat, on.dev);
    at::Tensor db = output(tensor(a[7], "ecc_layer_norm_grad: dbias"), {cols}, at::kFloat, on.dev);
    at::Tensor ws = scratch(tensor(a[8], "ecc_layer_norm_grad: ws"), ecc_layer_norm_grad_workspace_bytes(mx.rows, mx.cols),
                            on.dev, "ecc_layer_norm_grad: ws");
    check(ecc_layer_norm_grad(
              md.p, md.ld, mx.p, mx.ld, mx.type, vector(weight, mx.cols, on.dev, "ecc_layer_norm_grad: weight"),
              weight ? type_of(weight->scalar_type(), "ecc_layer_norm_grad: weight") : mx.type,
              (const float *)vector(mean, mx.rows, on.dev, "ecc_layer_norm_grad: mean", at::kFloat),
              (const float *)vector(rstd, mx.rows, on.dev, "ecc_layer_norm_grad: rstd", at::kFloat), mx.rows, mx.cols, mo.p,
              mo.ld, (float *)vector(&dw, mx.cols, on.dev, "ecc_layer_norm_grad: dweight", at::kFloat),
              (float *)vector(&db, mx.cols, on.dev, "ecc_layer_norm_grad: dbias", at::kFloat), where(ws), bytes_of(ws),
              on.stream),
          "ecc_layer_norm_grad");
    return results(dx, dw, db);
}

uint32_t *status_word(const at::Tensor &t, c10::Device dev, const char *what)
{
    return (uint32_t *)vector(&t, 1, dev, what, at::kInt);
}

// x, w, bias, residual, act, scale, out, out_dtype, out_scale, pre, ws, status
FUNCTION(linear, 12)
{
    const at::Tensor &x = first(a[0], "ecc_linear: needs CUDA tensors");
    const On on(x);
    const Matrix mx = matrix(x, on.dev, "ecc_linear: x");
    Opt w = tensor(a[1], "ecc_linear: w");
    if (!w || w->dim() != 2)
        refuse("ecc_linear: w");
    const uint64_t N = (uint64_t)w->size(0);
    const Matrix mw = operand(w, N, mx.cols, on.dev, "ecc_linear: w");
    if (mw.type != mx.type)
        refuse("ecc_linear: x and w of different types");
    Opt bias = tensor(a[2], "ecc_linear: bias");
    at::DimVector size(x.sizes().begin(), x.sizes().end());
    size.back() = (int64_t)N;
    at::Tensor out = output(tensor(a[6], "ecc_linear: out"), size,
                            dtype(a[7], "ecc_linear: out_dtype").value_or(mx.type == ECC_E4M3 ? at::kBFloat16 : x.scalar_type()),
                            on.dev);
    at::Tensor status = output(tensor(a[11], "ecc_linear: status"), {1}, at::kInt, on.dev);
    const Matrix mo = operand(&out, mx.rows, N, on.dev, "ecc_linear: out");
    const Matrix mr = operand(tensor(a[3], "ecc_linear: residual"), mx.rows, N, on.dev, "ecc_linear: residual");
    const Matrix mp = operand(tensor(a[9], "ecc_linear: pre"), mx.rows, N, on.dev, "ecc_linear: pre");
    ecc_linear_job j{};
    j.x = mx.p;
    j.w = mw.p;
    j.bias = vector(bias, N, on.dev, "ecc_linear: bias");
    j.residual = mr.p;
    j.out = mo.p;
    j.pre = mp.p;
    j.M = mx.rows;
    j.N = N;
    j.K = mx.cols;
    j.ldx = mx.ld;
    j.ldw = mw.ld;
    j.ldres = mr.ld;
    j.ldout = mo.ld;
    j.ldpre = mp.ld;
    j.scale = (float)number(a[5]);
    j.out_scale = (float)number(a[8]);
    j.in_type = mx.type;
    j.bias_type = bias ? type_of(bias->scalar_type(), "ecc_linear: bias") : 0;
    j.res_type = mr.type;
    j.out_type = mo.type;
    j.pre_type = mp.type;
    j.act = (uint32_t)integer(a[4]);
    at::Tensor ws = scratch(tensor(a[10], "ecc_linear: ws"), ecc_linear_workspace_bytes(&j), on.dev, "ecc_linear: ws");
    check(ecc_linear(&j, where(ws), bytes_of(ws), status_word(status, on.dev, "ecc_linear: status"), on.stream), "ecc_linear");
    return results(out, status);
}

// dy, x, w, pre, act, scale, dx, dw, dbias, dw_dtype, want (bits: 1 dx, 2 dw, 4 dbias), ws, status
FUNCTION(linear_grad, 13)
{
    const at::Tensor &dy = first(a[0], "ecc_linear_grad: needs CUDA tensors");
    const On on(dy);
    const Matrix md = matrix(dy, on.dev, "ecc_linear_grad: dy");
    const at::Tensor &x = first(a[1], "ecc_linear_grad: x"), &w = first(a[2], "ecc_linear_grad: w");
    if (!x.dim())
        refuse("ecc_linear_grad: x");
    const uint64_t M = md.rows, N = md.cols, K = (uint64_t)x.size(-1);
    const Matrix mx = operand(&x, M, K, on.dev, "ecc_linear_grad: x"), mw = operand(&w, N, K, on.dev, "ecc_linear_grad: w");
    if (mx.type != md.type || mw.type != md.type)
        refuse("ecc_linear_grad: dy, x and w of different types");
    const Matrix mp = operand(tensor(a[3], "ecc_linear_grad: pre"), M, N, on.dev, "ecc_linear_grad: pre");
    const long want = integer(a[10]);
    Opt gx = tensor(a[6], "ecc_linear_grad: dx"), gw = tensor(a[7], "ecc_linear_grad: dw");
    Opt gb = tensor(a[8], "ecc_linear_grad: dbias");
    at::Tensor dx, dw, db;
    if (gx || (want & 1))
        dx = output(gx, x.sizes(), x.scalar_type(), on.dev);
    if (gw || (want & 2))
        dw = output(gw, {(int64_t)N, (int64_t)K}, dtype(a[9], "ecc_linear_grad: dw_dtype").value_or(x.scalar_type()), on.dev);
    if (gb || (want & 4))
        db = output(gb, {(int64_t)N}, at::kFloat, on.dev);
    at::Tensor status = output(tensor(a[12], "ecc_linear_grad: status"), {1}, at::kInt, on.dev);
    const Matrix mdx = operand(dx.defined() ? &dx : nullptr, M, K, on.dev, "ecc_linear_grad: dx");
    const Matrix mdw = operand(dw.defined() ? &dw : nullptr, N, K, on.dev, "ecc_linear_grad: dw");
    if (dx.defined() && mdx.type != md.type)
        refuse("ecc_linear_grad: dx");
    ecc_linear_grad_job j{};
    j.dy = md.p;
    j.x = mx.p;
    j.w = mw.p;
    j.pre = mp.p;
    j.dx = mdx.p;
    j.dw = mdw.p;
    j.dbias = (float *)vector(db.defined() ? &db : nullptr, N, on.dev, "ecc_linear_grad: dbias", at::kFloat);
    j.M = M;
    j.N = N;
    j.K = K;
    j.lddy = md.ld;
    j.ldx = mx.ld;
    j.ldw = mw.ld;
    j.ldpre = mp.ld;
    j.lddx = mdx.ld;
    j.lddw = mdw.ld;
    j.scale = (float)number(a[5]);
    j.in_type = md.type;
    j.pre_type = mp.type;
    j.dw_type = mdw.type;
    j.act = (uint32_t)integer(a[4]);
    at::Tensor ws = scratch(tensor(a[11], "ecc_linear_grad: ws"), ecc_linear_grad_workspace_bytes(&j), on.dev,
                            "ecc_linear_grad: ws");
    check(ecc_linear_grad(&j, where(ws), bytes_of(ws), status_word(status, on.dev, "ecc_linear_grad: status"), on.stream),
          "ecc_linear_grad");
    return results(dx, dw, db, status);
}

// x, w_gate, w_up, bias_gate, bias_up, act, scale, up_scale, out, out_dtype, out_scale, pre_gate, pre_up, ws, status
FUNCTION(gated_linear, 15)
{
    const at::Tensor &x = first(a[0], "ecc_gated_linear: needs CUDA tensors");
    const On on(x);
    const Matrix mx = matrix(x, on.dev, "ecc_gated_linear: x");
    Opt wg = tensor(a[1], "ecc_gated_linear: w_gate"), wu = tensor(a[2], "ecc_gated_linear: w_up");
    if (!wg || !wu || wg->dim() != 2 || wu->dim() != 2)
        refuse("ecc_gated_linear: w_gate and w_up");
    const uint64_t N = (uint64_t)wg->size(0);
    const Matrix mg = operand(wg, N, mx.cols, on.dev, "ecc_gated_linear: w_gate"), mu = operand(wu, N, mx.cols, on.dev, "ecc_gated_linear: w_up");
    if (mg.type != mx.type || mu.type != mx.type)
        refuse("ecc_gated_linear: x, w_gate and w_up of different types");
    Opt bg = tensor(a[3], "ecc_gated_linear: bias_gate"), bu = tensor(a[4], "ecc_gated_linear: bias_up");
    const at::ScalarType b_type = bg ? bg->scalar_type() : bu ? bu->scalar_type() : at::kFloat;
    at::DimVector size(x.sizes().begin(), x.sizes().end());
    size.back() = (int64_t)N;
    at::Tensor out = output(tensor(a[8], "ecc_gated_linear: out"), size,
                            dtype(a[9], "ecc_gated_linear: out_dtype").value_or(mx.type == ECC_E4M3 ? at::kBFloat16 : x.scalar_type()),
                            on.dev);
    at::Tensor status = output(tensor(a[14], "ecc_gated_linear: status"), {1}, at::kInt, on.dev);
    const Matrix mo = operand(&out, mx.rows, N, on.dev, "ecc_gated_linear: out");
    const Matrix pg = operand(tensor(a[11], "ecc_gated_linear: pre_gate"), mx.rows, N, on.dev, "ecc_gated_linear: pre_gate");
    const Matrix pu = operand(tensor(a[12], "ecc_gated_linear: pre_up"), mx.rows, N, on.dev, "ecc_gated_linear: pre_up");
    if ((a[11] == Py_None) != (a[12] == Py_None) || (pg.p && pg.type != pu.type))
        refuse("ecc_gated_linear: pre_gate and pre_up");
    ecc_gated_linear_job j{};
    j.x = mx.p;
    j.w_gate = mg.p;
    j.w_up = mu.p;
    j.bias_gate = vector(bg, N, on.dev, "ecc_gated_linear: bias_gate", b_type);
    j.bias_up = vector(bu, N, on.dev, "ecc_gated_linear: bias_up", b_type);
    j.out = mo.p;
    j.pre_gate = pg.p;
    j.pre_up = pu.p;
    j.M = mx.rows;
    j.N = N;
    j.K = mx.cols;
    j.ldx = mx.ld;
    j.ldgate = mg.ld;
    j.ldup = mu.ld;
    j.ldout = mo.ld;
    j.ldpre_gate = pg.ld;
    j.ldpre_up = pu.ld;
    j.scale = (float)number(a[6]);
    j.up_scale = a[7] == Py_None ? j.scale : (float)number(a[7]);
    j.out_scale = (float)number(a[10]);
    j.in_type = mx.type;
    j.bias_type = type_of(b_type, "ecc_gated_linear: bias");
    j.out_type = mo.type;
    j.pre_type = pg.type;
    j.act = (uint32_t)integer(a[5]);
    at::Tensor ws = scratch(tensor(a[13], "ecc_gated_linear: ws"), ecc_gated_linear_workspace_bytes(&j), on.dev, "ecc_gated_linear: ws");
    check(ecc_gated_linear(&j, where(ws), bytes_of(ws), status_word(status, on.dev, "ecc_gated_linear: status"), on.stream),
          "ecc_gated_linear");
    return results(out, status);
}

// dy, x, w_gate, w_up, pre_gate, pre_up, act, scale, up_scale, dx, dw_gate, dw_up, dbias_gate, dbias_up, dw_dtype,
// want (bits: 1 dx, 2 dw, 4 dbias), ws, status
FUNCTION(gated_linear_grad, 18)
{
    const at::Tensor &dy = first(a[0], "ecc_gated_linear_grad: needs CUDA tensors");
    const On on(dy);
    const Matrix md = matrix(dy, on.dev, "ecc_gated_linear_grad: dy");
    const at::Tensor &x = first(a[1], "ecc_gated_linear_grad: x");
    const at::Tensor &wg = first(a[2], "ecc_gated_linear_grad: w_gate"), &wu = first(a[3], "ecc_gated_linear_grad: w_up");
    if (!x.dim())
        refuse("ecc_gated_linear_grad: x");
    const uint64_t M = md.rows, N = md.cols, K = (uint64_t)x.size(-1);
    const Matrix mx = operand(&x, M, K, on.dev, "ecc_gated_linear_grad: x"), mg = operand(&wg, N, K, on.dev, "ecc_gated_linear_grad: w_gate"),
                 mu = operand(&wu, N, K, on.dev, "ecc_gated_linear_grad: w_up");
    if (mx.type != md.type || mg.type != md.type || mu.type != md.type)
        refuse("ecc_gated_linear_grad: dy, x, w_gate and w_up of different types");
    Opt og = tensor(a[4], "ecc_gated_linear_grad: pre_gate"), ou = tensor(a[5], "ecc_gated_linear_grad: pre_up");
    if (!og || !ou || og->scalar_type() != ou->scalar_type())
        refuse("ecc_gated_linear_grad: pre_gate and pre_up");
    const Matrix pg = operand(og, M, N, on.dev, "ecc_gated_linear_grad: pre_gate"), pu = operand(ou, M, N, on.dev, "ecc_gated_linear_grad: pre_up");
    const long want = integer(a[15]);
    Opt gx = tensor(a[9], "ecc_gated_linear_grad: dx"), gg = tensor(a[10], "ecc_gated_linear_grad: dw_gate");
    Opt gu = tensor(a[11], "ecc_gated_linear_grad: dw_up"), hg = tensor(a[12], "ecc_gated_linear_grad: dbias_gate");
    Opt hu = tensor(a[13], "ecc_gated_linear_grad: dbias_up");
    at::Tensor dx, dg, du, bg, bu;
    if (gx || (want & 1))
        dx = output(gx, x.sizes(), x.scalar_type(), on.dev);
    if (gg || gu || (want & 2)) {
        const at::ScalarType type = gg   ? gg->scalar_type()
                                    : gu ? gu->scalar_type()
                                         : dtype(a[14], "ecc_gated_linear_grad: dw_dtype").value_or(x.scalar_type());
        dg = output(gg, {(int64_t)N, (int64_t)K}, type, on.dev);
        du = output(gu, {(int64_t)N, (int64_t)K}, type, on.dev);
    }
    if (hg || hu || (want & 4)) {
        bg = output(hg, {(int64_t)N}, at::kFloat, on.dev);
        bu = output(hu, {(int64_t)N}, at::kFloat, on.dev);
    }
    at::Tensor status = output(tensor(a[17], "ecc_gated_linear_grad: status"), {1}, at::kInt, on.dev);
    const Matrix mdx = operand(dx.defined() ? &dx : nullptr, M, K, on.dev, "ecc_gated_linear_grad: dx");
    const Matrix mdg = operand(dg.defined() ? &dg : nullptr, N, K, on.dev, "ecc_gated_linear_grad: dw_gate");
    const Matrix mdu = operand(du.defined() ? &du : nullptr, N, K, on.dev, "ecc_gated_linear_grad: dw_up");
    if ((dx.defined() && mdx.type != md.type) || mdg.type != mdu.type)
        refuse("ecc_gated_linear_grad: dx, dw_gate or dw_up of another type");
    ecc_gated_linear_grad_job j{};
    j.dy = md.p;
    j.x = mx.p;
    j.w_gate = mg.p;
    j.w_up = mu.p;
    j.pre_gate = pg.p;
    j.pre_up = pu.p;
    j.dx = mdx.p;
    j.dw_gate = mdg.p;
    j.dw_up = mdu.p;
    j.dbias_gate = (float *)vector(bg.defined() ? &bg : nullptr, N, on.dev, "ecc_gated_linear_grad: dbias_gate", at::kFloat);
    j.dbias_up = (float *)vector(bu.defined() ? &bu : nullptr, N, on.dev, "ecc_gated_linear_grad: dbias_up", at::kFloat);
    j.M = M;
    j.N = N;
    j.K = K;
    j.lddy = md.ld;
    j.ldx = mx.ld;
    j.ldgate = mg.ld;
    j.ldup = mu.ld;
    j.ldpre_gate = pg.ld;
    j.ldpre_up = pu.ld;
    j.lddx = mdx.ld;
    j.lddw_gate = mdg.ld;
    j.lddw_up = mdu.ld;
    j.scale = (float)number(a[7]);
    j.up_scale = a[8] == Py_None ? j.scale : (float)number(a[8]);
    j.in_type = md.type;
    j.pre_type = pg.type;
    j.dw_type = mdg.type;
    j.act = (uint32_t)integer(a[6]);
    at::Tensor ws = scratch(tensor(a[16], "ecc_gated_linear_grad: ws"), ecc_gated_linear_grad_workspace_bytes(&j), on.dev,
                            "ecc_gated_linear_grad: ws");
    check(ecc_gated_linear_grad(&j, where(ws), bytes_of(ws), status_word(status, on.dev, "ecc_gated_linear_grad: status"), on.stream),
          "ecc_gated_linear_grad");
    return results(dx, dg, du, bg, bu, status);
}

// logits, tokens, top, scale
FUNCTION(token_logprob, 4)
{
    const at::Tensor &logits = first(a[0], "ecc_token_logprob: needs CUDA tensors");
    const On on(logits);
    const Matrix m = matrix(logits, on.dev, "ecc_token_logprob: logits");
    Opt tokens = tensor(a[1], "ecc_token_logprob: tokens");
    const long top = integer(a[2]);
    if (top < 0 || top > ECC_MAX_TOP)
        refuse("ecc_token_logprob: top");
    const auto lead = logits.sizes().slice(0, logits.dim() - 1);
    const void *tok = vector(tokens, m.rows, on.dev, "ecc_token_logprob: tokens", at::kLong);
    at::Tensor logprob, entropy = fresh(lead, at::kFloat, on.dev), lse = fresh(lead, at::kFloat, on.dev), value, index;
    if (tokens)
        logprob = fresh(lead, at::kFloat, on.dev);
    if (top) {
        at::DimVector size(lead.begin(), lead.end());
        size.push_back(top);
        value = fresh(size, at::kFloat, on.dev);
        index = fresh(size, at::kInt, on.dev);
    }
    check(ecc_token_logprob(m.p, m.ld, m.type, (const int64_t *)tok, m.rows, m.cols, (float)number(a[3]), (uint32_t)top,
                            (float *)where(logprob), (float *)where(entropy), (float *)where(lse), (float *)where(value),
                            (int32_t *)where(index), on.stream),
          "ecc_token_logprob");
    return results(logprob, entropy, lse, value, index);
}

// logits, tokens, lse, entropy, dlogprob, dentropy, scale, dlogits
FUNCTION(token_logprob_grad, 8)
{
    const at::Tensor &logits = first(a[0], "ecc_token_logprob_grad: needs CUDA tensors");
    const On on(logits);
    const Matrix m = matrix(logits, on.dev, "ecc_token_logprob_grad: logits");
    at::Tensor d = output(tensor(a[7], "ecc_token_logprob_grad: dlogits"), logits.sizes(), logits.scalar_type(), on.dev);
    if (d.sizes() != logits.sizes() || d.scalar_type() != logits.scalar_type())
        refuse("ecc_token_logprob_grad: dlogits");
    const Matrix md = matrix(d, on.dev, "ecc_token_logprob_grad: dlogits");
    auto f32 = [&](int i, const char *what) { return (const float *)vector(tensor(a[i], what), m.rows, on.dev, what, at::kFloat); };
    const char *tw = "ecc_token_logprob_grad: tokens";
    check(ecc_token_logprob_grad(m.p, m.ld, m.type, (const int64_t *)vector(tensor(a[1], tw), m.rows, on.dev, tw, at::kLong),
                                 m.rows, m.cols, (float)number(a[6]), f32(2, "ecc_token_logprob_grad: lse"),
                                 f32(3, "ecc_token_logprob_grad: entropy"), f32(4, "ecc_token_logprob_grad: dlogprob"),
                                 f32(5, "ecc_token_logprob_grad: dentropy"), md.p, md.ld, on.stream),
          "ecc_token_logprob_grad");
    return wrap(d);
}

// x, w, tokens, scale, ws, status
FUNCTION(linear_logprob, 6)
{
    const at::Tensor &x = first(a[0], "ecc_linear_logprob: needs CUDA tensors");
    const On on(x);
    const Matrix mx = matrix(x, on.dev, "ecc_linear_logprob: x");
    Opt w = tensor(a[1], "ecc_linear_logprob: w"), tokens = tensor(a[2], "ecc_linear_logprob: tokens");
    if (!w || w->dim() != 2)
        refuse("ecc_linear_logprob: w");
    const Matrix mw = operand(w, (uint64_t)w->size(0), mx.cols, on.dev, "ecc_linear_logprob: w");
    if (mw.type != mx.type)
        refuse("ecc_linear_logprob: x and w of different types");
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    ecc_linear_logprob_job j{};
    j.x = mx.p;
    j.w = mw.p;
    j.tokens = (const int64_t *)vector(tokens, mx.rows, on.dev, "ecc_linear_logprob: tokens", at::kLong);
    j.rows = mx.rows;
    j.vocab = (uint64_t)w->size(0);
    j.K = mx.cols;
    j.ldx = mx.ld;
    j.ldw = mw.ld;
    j.scale = (float)number(a[3]);
    j.in_type = mx.type;
    at::Tensor logprob, entropy = fresh(lead, at::kFloat, on.dev), lse = fresh(lead, at::kFloat, on.dev);
    if (tokens)
        logprob = fresh(lead, at::kFloat, on.dev);
    j.logprob = (float *)where(logprob);
    j.entropy = (float *)where(entropy);
    j.lse = (float *)where(lse);
    at::Tensor status = output(tensor(a[5], "ecc_linear_logprob: status"), {1}, at::kInt, on.dev);
    at::Tensor ws = scratch(tensor(a[4], "ecc_linear_logprob: ws"), ecc_linear_logprob_workspace_bytes(&j), on.dev,
                            "ecc_linear_logprob: ws");
    check(ecc_linear_logprob(&j, where(ws), bytes_of(ws), status_word(status, on.dev, "ecc_linear_logprob: status"), on.stream),
          "ecc_linear_logprob");
    return results(logprob, entropy, lse, status);
}

// x, w, tokens, lse, entropy, dlogprob, dentropy, scale, dx, dw, dw_dtype, want (bits: 1 dx, 2 dw), ws, status
FUNCTION(linear_logprob_grad, 14)
{
    const at::Tensor &x = first(a[0], "ecc_linear_logprob_grad: needs CUDA tensors");
    const On on(x);
    const Matrix mx = matrix(x, on.dev, "ecc_linear_logprob_grad: x");
    Opt w = tensor(a[1], "ecc_linear_logprob_grad: w");
    if (!w || w->dim() != 2)
        refuse("ecc_linear_logprob_grad: w");
    const uint64_t V = (uint64_t)w->size(0);
    const Matrix mw = operand(w, V, mx.cols, on.dev, "ecc_linear_logprob_grad: w");
    if (mw.type != mx.type)
        refuse("ecc_linear_logprob_grad: x and w of different types");
    auto f32 = [&](int i, const char *what) { return (const float *)vector(tensor(a[i], what), mx.rows, on.dev, what, at::kFloat); };
    const char *tw = "ecc_linear_logprob_grad: tokens";
    const long want = integer(a[11]);
    Opt gx = tensor(a[8], "ecc_linear_logprob_grad: dx"), gw = tensor(a[9], "ecc_linear_logprob_grad: dw");
    at::Tensor dx, dw;
    if (gx || (want & 1))
        dx = output(gx, x.sizes(), x.scalar_type(), on.dev);
    if (gw || (want & 2))
        dw = output(gw, {(int64_t)V, (int64_t)mx.cols}, dtype(a[10], "ecc_linear_logprob_grad: dw_dtype").value_or(x.scalar_type()), on.dev);
    at::Tensor status = output(tensor(a[13], "ecc_linear_logprob_grad: status"), {1}, at::kInt, on.dev);
    const Matrix mdx = operand(dx.defined() ? &dx : nullptr, mx.rows, mx.cols, on.dev, "ecc_linear_logprob_grad: dx");
    const Matrix mdw = operand(dw.defined() ? &dw : nullptr, V, mx.cols, on.dev, "ecc_linear_logprob_grad: dw");
    if (dx.defined() && mdx.type != mx.type)
        refuse("ecc_linear_logprob_grad: dx");
    ecc_linear_logprob_grad_job j{};
    j.x = mx.p;
    j.w = mw.p;
    j.tokens = (const int64_t *)vector(tensor(a[2], tw), mx.rows, on.dev, tw, at::kLong);
    j.lse = f32(3, "ecc_linear_logprob_grad: lse");
    j.entropy = f32(4, "ecc_linear_logprob_grad: entropy");
    j.dlogprob = f32(5, "ecc_linear_logprob_grad: dlogprob");
    j.dentropy = f32(6, "ecc_linear_logprob_grad: dentropy");
    j.dx = mdx.p;
    j.dw = mdw.p;
    j.rows = mx.rows;
    j.vocab = V;
    j.K = mx.cols;
    j.ldx = mx.ld;
    j.ldw = mw.ld;
    j.lddx = mdx.ld;
    j.lddw = mdw.ld;
    j.scale = (float)number(a[7]);
    j.in_type = mx.type;
    j.dw_type = mdw.type;
    at::Tensor ws = scratch(tensor(a[12], "ecc_linear_logprob_grad: ws"), ecc_linear_logprob_grad_workspace_bytes(&j), on.dev,
                            "ecc_linear_logprob_grad: ws");
    check(ecc_linear_logprob_grad(&j, where(ws), bytes_of(ws), status_word(status, on.dev, "ecc_linear_logprob_grad: status"),
                                  on.stream),
          "ecc_linear_logprob_grad");
    return results(dx, dw, status);
}

// A list argument: its tensors by number (None: none at all)
struct List {
    PyObject *seq = nullptr;
    List(PyObject *o, Py_ssize_t n, const char *what) // n < 0: as many as there are
    {
        if (o == Py_None)
            return;
        if (!PyList_Check(o) && !PyTuple_Check(o))
            refuse(what);
        if (n >= 0 && PySequence_Fast_GET_SIZE(o) != n)
            refuse(what);
        seq = o;
    }
    Opt operator()(Py_ssize_t i, const char *what) const
    {
        return seq ? tensor(PySequence_Fast_GET_ITEM(seq, i), what) : nullptr;
    }
};
// a number, or a tensor of one value that the kernel reads
template <typename T> const T *value_at(PyObject *o, c10::Device dev, const char *what)
{
    if (!THPVariable_Check(o))
        return nullptr;
    return (const T *)vector(tensor(o, what), 1, dev, what, sizeof(T) == 8 ? at::kLong : at::kFloat);
}

// params, grads, m, v, m_scale, v_scale, master, step, lr, beta1, beta2, eps, weight_decay, grad_scale, seed
FUNCTION(adamw, 15)
{
    const char *what = "ecc_adamw: params and grads";
    if (!PyList_Check(a[0]) && !PyTuple_Check(a[0]))
        refuse(what);
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[0]);
    const List params(a[0], n, what), grads(a[1], n, what), ms(a[2], n, "ecc_adamw: m"), vs(a[3], n, "ecc_adamw: v");
    const List mss(a[4], n, "ecc_adamw: m_scale"), vss(a[5], n, "ecc_adamw: v_scale"), masters(a[6], n, "ecc_adamw: master");
    if (!grads.seq || !ms.seq || !vs.seq)
        refuse(what);
    std::optional<On> on;
    std::vector<ecc_adamw_tensor> list;
    list.reserve((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        Opt p = params(i, what), g = grads(i, what);
        if (!g) // nothing to learn from
            continue;
        if (!p || !p->is_cuda() || p->sizes() != g->sizes())
            refuse(what);
        if (!on)
            on.emplace(*p);
        const c10::Device dev = on->dev;
        const uint64_t len = (uint64_t)p->numel();
        ecc_adamw_tensor t{};
        t.n = len;
        t.param = vector(p, len, dev, what);
        t.param_type = type_of(p->scalar_type(), what);
        t.grad = vector(g, len, dev, what);
        t.grad_type = type_of(g->scalar_type(), what);
        Opt m = ms(i, "ecc_adamw: m"), v = vs(i, "ecc_adamw: v");
        if (!m || !v)
            refuse("ecc_adamw: m and v");
        t.m = vector(m, len, dev, "ecc_adamw: m");
        t.state_type = type_of(m->scalar_type(), "ecc_adamw: m");
        t.v = vector(v, len, dev, "ecc_adamw: v", m->scalar_type());
        if (t.state_type == ECC_E4M3) {
            const uint64_t groups = (len + ECC_ADAMW_GROUP - 1) / ECC_ADAMW_GROUP;
            Opt s = mss(i, "ecc_adamw: m_scale"), r = vss(i, "ecc_adamw: v_scale");
            if (!s || !r)
                refuse("ecc_adamw: m_scale and v_scale");
            t.m_scale = (float *)vector(s, groups, dev, "ecc_adamw: m_scale", at::kFloat);
            t.v_scale = (float *)vector(r, groups, dev, "ecc_adamw: v_scale", at::kFloat);
        }
        t.master = (float *)vector(masters(i, "ecc_adamw: master"), len, dev, "ecc_adamw: master", at::kFloat);
        list.push_back(t);
    }
    ecc_adamw_job j{};
    j.tensors = list.data();
    j.count = list.size();
    if (!on)
        Py_RETURN_NONE;
    j.step_at = value_at<int64_t>(a[7], on->dev, "ecc_adamw: step");
    j.lr_at = value_at<float>(a[8], on->dev, "ecc_adamw: lr");
    j.grad_scale_at = value_at<float>(a[13], on->dev, "ecc_adamw: grad_scale");
    if (!j.step_at) {
        const long step = integer(a[7]);
        if (step < 1)
            refuse("ecc_adamw: step");
        j.step = (uint64_t)step;
    }
    j.lr = j.lr_at ? 0.0 : number(a[8]);
    j.beta1 = number(a[9]);
    j.beta2 = number(a[10]);
    j.eps = number(a[11]);
    j.weight_decay = number(a[12]);
    j.grad_scale = j.grad_scale_at ? 1.0 : number(a[13]);
    const long seed = integer(a[14]);
    if (seed < 0 || seed > 0xFFFFFFFFL)
        refuse("ecc_adamw: seed");
    j.seed = (uint32_t)seed;
    check(ecc_adamw(&j, on->stream), "ecc_adamw");
    Py_RETURN_NONE;
}

PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(layer_norm),    METHOD(layer_norm_grad), METHOD(linear), METHOD(linear_grad),
                           METHOD(token_logprob), METHOD(token_logprob_grad), METHOD(adamw),
                           METHOD(gated_linear), METHOD(gated_linear_grad),
                           METHOD(linear_logprob), METHOD(linear_logprob_grad), {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "ecc_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

extern "C" PyObject *PyInit_ecc_torch() { return PyModule_Create(&g_module); }
