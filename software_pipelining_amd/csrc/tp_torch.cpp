// The 8-bit layer's operators called straight from Python: what linear8.py
// does in Python (checks, outputs, the C call), for the calls that need
// nothing else. Any call it does not take (an argument that is wrong or
// unusual, another device than the current one, an error from the library)
// gives None, and the caller goes the long way, which also words the errors.
//
// On an MI355X host a call of rms_norm with four outputs took 12.0 us of host
// time through Python and ctypes; the launch itself takes 2.7.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tilepipe.h"

namespace {

constexpr int64_t kBlock = 128;

int number_code(at::ScalarType t)
{
    return t == at::kBFloat16 ? TP_BF16 : t == at::kHalf ? TP_FP16 : t == at::kFloat ? TP_FP32 : -1;
}

int eight_code(at::ScalarType t)
{
    return t == at::kFloat8_e4m3fn ? TP_E4M3 : t == at::kFloat8_e5m2 ? TP_E5M2 : -1;
}

at::ScalarType eight_type(int code) { return code == TP_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2; }

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Matrix {
    const at::Tensor *t;
    int64_t rows, cols, stride;
};

// A 2-D tensor on `device` with unit column stride and rows that do not
// overlap.
bool matrix(PyObject *o, c10::Device device, Matrix &m)
{
    m.t = tensor(o);
    if (!m.t || m.t->dim() != 2 || m.t->device() != device || m.t->layout() != at::kStrided)
        return false;
    m.rows = m.t->size(0);
    m.cols = m.t->size(1);
    m.stride = m.rows > 1 ? m.t->stride(0) : m.cols > 1 ? m.cols : 1;
    return (m.cols <= 1 || m.t->stride(1) == 1) && m.stride >= m.cols;
}

bool vector(PyObject *o, c10::Device device, at::ScalarType type, int64_t n)
{
    const at::Tensor *t = tensor(o);
    return t && t->dim() == 1 && t->size(0) == n && t->scalar_type() == type && t->device() == device &&
           t->is_contiguous();
}

bool scales(PyObject *o, c10::Device device, int64_t rows, int64_t cols)
{
    const at::Tensor *t = tensor(o);
    return t && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols && t->scalar_type() == at::kFloat &&
           t->device() == device && t->is_contiguous();
}

// The device of a call: that of its first argument, if it is the current one.
bool device_of(PyObject *o, c10::Device &d)
{
    const at::Tensor *t = tensor(o);
    if (!t || !t->device().is_cuda())
        return false;
    d = t->device();
    return d.index() == c10::hip::current_device();
}

void *stream_of(c10::Device d) { return (void *)c10::hip::getCurrentHIPStream(d.index()).stream(); }

at::Tensor empty(int64_t rows, int64_t cols, at::ScalarType type, c10::Device d)
{
    return at::Tensor(at::detail::empty_cuda({rows, cols}, type, d, std::nullopt));
}

at::Tensor empty(int64_t n, at::ScalarType type, c10::Device d)
{
    return at::Tensor(at::detail::empty_cuda({n}, type, d, std::nullopt));
}

int64_t padded(int64_t cols) { return (cols + 15) / 16 * 16; }

at::Tensor empty_eight(int64_t rows, int64_t cols, int code, c10::Device d)
{
    return cols % 16 == 0 ? empty(rows, cols, eight_type(code), d)
                          : at::Tensor(at::detail::empty_strided_cuda({rows, cols}, {padded(cols), 1},
                                                                      eight_type(code), d));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

PyObject *wrap(const at::Tensor &t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *wrap_all(std::initializer_list<at::Tensor> ts)
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

// No C++ exception leaves an entry: one gives None like anything else that is
// not taken here.
template <class F>
PyObject *guarded(F &&f)
{
    try {
        return f();
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (x, weight, eps, residual or None, 8-bit code or -1, save_rstd) -> (out, scale, sum, rstd)
PyObject *rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        c10::Device d(c10::kCUDA);
        Matrix x, r{};
        if (n != 6 || !device_of(args[0], d) || !matrix(args[0], d, x) || x.rows == 0 || x.cols == 0 ||
            !PyFloat_Check(args[2]) || !PyLong_Check(args[4]) || !PyBool_Check(args[5]))
            Py_RETURN_NONE;
        const at::ScalarType type = x.t->scalar_type();
        const int code = number_code(type);
        const long eight = PyLong_AsLong(args[4]);
        const bool residual = args[3] != Py_None;
        if (code < 0 || (eight != -1 && eight != TP_E4M3 && eight != TP_E5M2) ||
            !vector(args[1], d, type, x.cols) ||
            (residual && (!matrix(args[3], d, r) || r.rows != x.rows || r.cols != x.cols ||
                          r.t->scalar_type() != type)))
            Py_RETURN_NONE;
        at::Tensor out, scale, sum, rstd;
        if (residual)
            sum = empty(x.rows, x.cols, type, d);
        if (eight < 0) {
            out = empty(x.rows, x.cols, type, d);
        } else {
            out = empty_eight(x.rows, x.cols, (int)eight, d);
            scale = empty(x.rows, ceil_div(x.cols, kBlock), at::kFloat, d);
        }
        if (args[5] == Py_True)
            rstd = empty(x.rows, at::kFloat, d);
        const int st = tp_rms_norm(
            x.t->data_ptr(), x.stride, residual ? r.t->data_ptr() : nullptr, r.stride,
            tensor(args[1])->data_ptr(), x.rows, x.cols, code, (float)PyFloat_AS_DOUBLE(args[2]),
            residual ? sum.data_ptr() : nullptr, x.cols, out.data_ptr(), eight < 0 ? x.cols : padded(x.cols),
            eight < 0 ? code : (int)eight, scale.defined() ? (float *)scale.data_ptr() : nullptr,
            rstd.defined() ? (float *)rstd.data_ptr() : nullptr, stream_of(d));
        if (st != TP_OK)
            Py_RETURN_NONE;
        return wrap_all({out, scale, sum, rstd});
    });
}

// (dy, x, weight, rstd, dsum or None) -> (dx, dweight)
PyObject *rms_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        c10::Device d(c10::kCUDA);
        Matrix dy, x, ds{};
        if (n != 5 || !device_of(args[0], d) || !matrix(args[0], d, dy) || !matrix(args[1], d, x) ||
            x.cols == 0 || dy.rows != x.rows || dy.cols != x.cols)
            Py_RETURN_NONE;
        const at::ScalarType type = x.t->scalar_type();
        const int code = number_code(type);
        const bool more = args[4] != Py_None;
        if (code < 0 || dy.t->scalar_type() != type || !vector(args[2], d, type, x.cols) ||
            !vector(args[3], d, at::kFloat, x.rows) ||
            (more && (!matrix(args[4], d, ds) || ds.rows != x.rows || ds.cols != x.cols ||
                      ds.t->scalar_type() != type)))
            Py_RETURN_NONE;
        const int64_t need = tp_rms_norm_backward_workspace_bytes(x.rows, x.cols, code);
        if (need < 0)
            Py_RETURN_NONE;
        const at::Tensor dx = empty(x.rows, x.cols, type, d), dw = empty(x.cols, at::kFloat, d),
                         ws = empty(need, at::kByte, d);
        const int st = tp_rms_norm_backward(
            dy.t->data_ptr(), dy.stride, x.t->data_ptr(), x.stride, tensor(args[2])->data_ptr(),
            (const float *)tensor(args[3])->data_ptr(), more ? ds.t->data_ptr() : nullptr, ds.stride, x.rows,
            x.cols, code, dx.data_ptr(), x.cols, (float *)dw.data_ptr(), ws.data_ptr(), need, stream_of(d));
        if (st != TP_OK)
            Py_RETURN_NONE;
        return wrap_all({dx, dw});
    });
}

// (x, 8-bit code, square, straight, transposed) -> (q, scale, qt, scale_t)
PyObject *block_quantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        c10::Device d(c10::kCUDA);
        Matrix x;
        if (n != 5 || !device_of(args[0], d) || !matrix(args[0], d, x) || x.rows == 0 || x.cols == 0 ||
            !PyLong_Check(args[1]) || !PyBool_Check(args[2]) || !PyBool_Check(args[3]) || !PyBool_Check(args[4]))
            Py_RETURN_NONE;
        const int code = number_code(x.t->scalar_type());
        const int eight = (int)PyLong_AsLong(args[1]);
        const bool square = args[2] == Py_True, straight = args[3] == Py_True, turned = args[4] == Py_True;
        if (code < 0 || (eight != TP_E4M3 && eight != TP_E5M2) || (!straight && !turned))
            Py_RETURN_NONE;
        const int64_t down = ceil_div(x.rows, kBlock), across = ceil_div(x.cols, kBlock);
        at::Tensor q, scale, qt, scale_t;
        if (straight) {
            q = empty_eight(x.rows, x.cols, eight, d);
            scale = empty(square ? down : x.rows, across, at::kFloat, d);
        }
        if (turned) {
            qt = empty_eight(x.cols, x.rows, eight, d);
            scale_t = empty(square ? across : x.cols, down, at::kFloat, d);
        }
        const int st = tp_block_quantize(
            x.t->data_ptr(), x.stride, x.rows, x.cols, code, square, eight, straight ? q.data_ptr() : nullptr,
            padded(x.cols), straight ? (float *)scale.data_ptr() : nullptr, turned ? qt.data_ptr() : nullptr,
            padded(x.rows), turned ? (float *)scale_t.data_ptr() : nullptr, stream_of(d));
        if (st != TP_OK)
            Py_RETURN_NONE;
        return wrap_all({q, scale, qt, scale_t});
    });
}

// (a, a_scale, b, b_scale, out's code) -> out
PyObject *block_matmul(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        c10::Device d(c10::kCUDA);
        Matrix a, b;
        if (n != 5 || !device_of(args[0], d) || !matrix(args[0], d, a) || !matrix(args[2], d, b) ||
            a.cols != b.cols || a.rows == 0 || b.rows == 0 || !PyLong_Check(args[4]))
            Py_RETURN_NONE;
        const int a_code = eight_code(a.t->scalar_type()), b_code = eight_code(b.t->scalar_type());
        const int code = (int)PyLong_AsLong(args[4]);
        const int64_t blocks = ceil_div(a.cols, kBlock);
        if (a_code < 0 || b_code < 0 || code < 0 || !scales(args[1], d, a.rows, blocks))
            Py_RETURN_NONE;
        const bool square = scales(args[3], d, ceil_div(b.rows, kBlock), blocks);
        if (!square && !scales(args[3], d, b.rows, blocks))
            Py_RETURN_NONE;
        const int64_t need = tp_block_matmul_workspace_bytes(a.rows, b.rows, a.cols, code);
        if (need < 0)
            Py_RETURN_NONE;
        const at::Tensor out = empty(a.rows, b.rows,
                                     code == TP_BF16   ? at::kBFloat16
                                     : code == TP_FP16 ? at::kHalf
                                                       : at::kFloat,
                                     d);
        at::Tensor ws;
        if (need > 0)
            ws = empty(need, at::kByte, d);
        const int st = tp_block_matmul(
            a.t->data_ptr(), a.stride, a_code, (const float *)tensor(args[1])->data_ptr(), b.t->data_ptr(),
            b.stride, b_code, (const float *)tensor(args[3])->data_ptr(), square, a.rows, b.rows, a.cols,
            out.data_ptr(), b.rows, code, need > 0 ? ws.data_ptr() : nullptr, need, stream_of(d));
        if (st != TP_OK)
            Py_RETURN_NONE;
        return wrap(out);
    });
}

PyMethodDef g_methods[] = {
    {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, nullptr},
    {"rms_norm_backward", (PyCFunction)(void (*)(void))rms_norm_backward, METH_FASTCALL, nullptr},
    {"block_quantize", (PyCFunction)(void (*)(void))block_quantize, METH_FASTCALL, nullptr},
    {"block_matmul", (PyCFunction)(void (*)(void))block_matmul, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_linear8", "Direct calls of the 8-bit layer's operators.",
                        -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__linear8(void) { return PyModule_Create(&g_module); }
