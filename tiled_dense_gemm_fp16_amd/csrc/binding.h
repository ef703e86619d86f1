// binding.h -- what the compiled Python modules of the library share: checks
// of tensor arguments, outputs and workspaces from torch's allocator, calls of
// the C entry points on torch's current stream.  Nothing is computed here and
// nothing is kept between calls.
#ifndef GEMM_F16_BINDING_H
#define GEMM_F16_BINDING_H

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/util/Exception.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <utility>
#include <vector>

#include "gemm_f16.h"

namespace {

PyObject *g_error, *g_stream;   // GemmError, the current stream's address

struct Raised {};   // a Python exception is set

template <class... A>
[[noreturn]] void refuse(const char *format, A... a)
{
    PyErr_Format(PyExc_ValueError, format, a...);
    throw Raised{};
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised{};
    return v;
}
int small(PyObject *o)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "integer out of range");
        throw Raised{};
    }
    return (int)v;
}
double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised{};
    return v;
}

const at::Tensor *tensor(PyObject *o)
{
    if (!THPVariable_Check(o))
        return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.layout() == at::kStrided ? &t : nullptr;
}
bool on(const at::Tensor &t, int index) { return t.is_cuda() && t.get_device() == index; }

int device_of(PyObject *o, const char *name, PyObject *stream_device)
{
    const at::Tensor *t = tensor(o);
    if (!t || !t->is_cuda())
        refuse("%s must be a GPU tensor", name);
    const int index = (int)t->get_device();
    if (stream_device != Py_None && small(stream_device) != index)
        refuse("stream must be a stream of cuda:%d", index);
    return index;
}

const char *type_name(at::ScalarType t)
{
    return t == at::kHalf ? "float16" : t == at::kInt ? "int32" : t == at::kChar ? "int8" : "float32";
}

void *address(const at::Tensor &t) { return t.numel() ? t.data_ptr() : nullptr; }

// Address of a contiguous tensor of this dtype and shape on GPU `index`.
void *buffer(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, int index)
{
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != type || t->sizes() != shape) {
        PyObject *want = PyTuple_New((Py_ssize_t)shape.size());
        if (!want)
            throw Raised{};
        for (size_t i = 0; i < shape.size(); ++i)
            PyTuple_SET_ITEM(want, (Py_ssize_t)i, PyLong_FromLongLong(shape[i]));
        PyErr_Format(PyExc_ValueError, "%s must be a %s tensor of shape %R", name, type_name(type), want);
        Py_DECREF(want);
        throw Raised{};
    }
    if (!on(*t, index) || !t->is_contiguous())
        refuse("%s must be a contiguous tensor on cuda:%d", name, index);
    return address(*t);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int index)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)index)));
}

// A caller's float16 output, or a new one.
struct Output {
    at::Tensor made;
    PyObject *given = nullptr;
    void *at = nullptr;
    Output(PyObject *out, at::IntArrayRef shape, int index)
    {
        if (out != Py_None) {
            at = buffer(out, "out", at::kHalf, shape, index);
            given = out;
        } else {
            made = empty(shape, at::kHalf, index);
            at = address(made);
        }
    }
    PyObject *result()
    {
        if (!given)
            return THPVariable_Wrap(std::move(made));
        Py_INCREF(given);
        return given;
    }
};

// A caller's workspace, or one of `need` bytes from torch's caching allocator.
struct Workspace {
    at::Tensor made;
    void *at = nullptr;
    int64_t bytes = 0;
    Workspace() = default;
    Workspace(PyObject *given, int64_t need, int index)
    {
        if (given != Py_None) {
            const at::Tensor *t = tensor(given);
            if (!t || !on(*t, index) || !t->is_contiguous())
                refuse("workspace must be a contiguous tensor on cuda:%d", index);
            at = address(*t);
            bytes = (int64_t)t->nbytes();
        } else if (need > 0) {
            made = empty({(need + 3) / 4}, at::kFloat, index);
            at = made.data_ptr();
            bytes = need;
        }
    }
};

void check(int status, const char *what)
{
    if (status == GEMM_F16_SUCCESS)
        return;
    PyObject *e = PyObject_CallFunction(g_error, "is", status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// Call a C entry point on GPU `index` and the current stream of it.
template <class F>
void call(int index, const char *what, F f)
{
    PyObject *i = PyLong_FromLong(index), *raw = i ? PyObject_CallOneArg(g_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!raw)
        throw Raised{};
    void *stream = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (!stream && PyErr_Occurred())
        throw Raised{};
    int status = GEMM_F16_ERROR_NO_DEVICE;
    Py_BEGIN_ALLOW_THREADS
    int now = -1;
    if (hipGetDevice(&now) == hipSuccess) {
        if (now == index) {
            status = f(stream);
        } else if (hipSetDevice(index) == hipSuccess) {
            status = f(stream);
            (void)hipSetDevice(now);
        }
    }
    Py_END_ALLOW_THREADS
    check(status, what);
}

template <PyObject *(*F)(PyObject *const *), int COUNT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    if (count != COUNT || !g_error) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or no setup()");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

} // namespace

#define GEMM_F16_ENTRY(name, count) {#name, (PyCFunction)(void (*)(void))(entry<name, count>), METH_FASTCALL, nullptr}

#endif
