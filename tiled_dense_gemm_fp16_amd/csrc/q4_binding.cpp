// q4_binding.cpp -- the Python side of include/gemm_f16_q4.h: checks of tensor
// arguments, outputs and workspaces from torch's allocator, calls of the C
// entry points on torch's current stream.
//
// A decode step makes many calls whose kernels take a few microseconds; read
// attribute by attribute from Python, the 10 to 17 tensors of a call take
// longer than that (append and read of 64 tokens: 28 us of host time for 13 us
// of kernels).  Here a tensor's checks take some 20 ns.  Nothing is computed
// here and nothing is kept between calls.
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

#include "gemm_f16_q4.h"

namespace {

PyObject *g_matrix, *g_cache, *g_error, *g_stream;   // Q4Matrix, Q4Cache, GemmError, the current stream's address

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
    return t == at::kHalf ? "float16" : t == at::kInt ? "int32" : "float32";
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

int64_t known_group(int64_t group)
{
    if (group != 32 && group != 64 && group != 128)
        refuse("group must be one of (32, 64, 128), got %lld", (long long)group);
    return group;
}

struct Matrix {
    int64_t n, k;
    int group;
    PyObject *codes_tensor, *words_tensor;
    void *codes = nullptr, *words = nullptr;
    explicit Matrix(PyObject *w)
    {
        if (!PyObject_TypeCheck(w, (PyTypeObject *)g_matrix) || PyTuple_GET_SIZE(w) != 5)
            refuse("w must be a Q4Matrix (as q4_compress returns)");
        codes_tensor = PyTuple_GET_ITEM(w, 0);
        words_tensor = PyTuple_GET_ITEM(w, 1);
        n = integer(PyTuple_GET_ITEM(w, 2));
        k = integer(PyTuple_GET_ITEM(w, 3));
        group = (int)known_group(integer(PyTuple_GET_ITEM(w, 4)));
        if (n < 0 || k < 0 || n > (int64_t)1 << 40 || k > (int64_t)1 << 40)
            refuse("w.n and w.k must be a matrix's sizes");
    }
    void check(int index)
    {
        const int64_t nb = (n + 15) / 16, kb = (k + 127) / 128;
        codes = buffer(codes_tensor, "w.codes", at::kInt, {nb, kb, 4, 16, 4}, index);
        words = buffer(words_tensor, "w.words", at::kInt, {nb, kb, 16, 128 / group}, index);
    }
};

struct Cache {
    gemm_f16_q4_cache_t c;
    int index;
    Cache(PyObject *cache, PyObject *stream_device)
    {
        if (!PyObject_TypeCheck(cache, (PyTypeObject *)g_cache) || PyTuple_GET_SIZE(cache) != 5)
            refuse("cache must be a Q4Cache (as q4_cache returns)");
        const int64_t group = known_group(integer(PyTuple_GET_ITEM(cache, 4)));
        PyObject *k = PyTuple_GET_ITEM(cache, 0);
        const at::Tensor *codes = tensor(k);
        if (!codes || codes->dim() != 4)
            refuse("cache.k_codes must be a tensor of pages x heads x page_size x head_dim / 8");
        index = device_of(k, "cache.k_codes", stream_device);
        if (codes->size(1) > INT32_MAX || codes->size(2) > INT32_MAX || codes->size(3) > INT32_MAX / 8)
            refuse("cache.k_codes must be a tensor of pages x heads x page_size x head_dim / 8");
        const int64_t pages = codes->size(0), heads = codes->size(1), page = codes->size(2), d = 8 * codes->size(3);
        const int64_t words[4] = {pages, heads, d / group, page};
        c.k_codes = buffer(k, "cache.k_codes", at::kInt, codes->sizes(), index);
        c.k_words = buffer(PyTuple_GET_ITEM(cache, 1), "cache.k_words", at::kInt, words, index);
        c.v_codes = buffer(PyTuple_GET_ITEM(cache, 2), "cache.v_codes", at::kInt, {pages, heads, page / 8, 16, d / 16}, index);
        c.v_words = buffer(PyTuple_GET_ITEM(cache, 3), "cache.v_words", at::kInt, words, index);
        c.pages = pages;
        c.heads = (int32_t)heads;
        c.page_size = (int32_t)page;
        c.head_dim = (int32_t)d;
        c.group = (int32_t)group;
    }
};

struct Table {
    const int32_t *at;
    int64_t batch, width;
    Table(PyObject *o, int index)
    {
        const at::Tensor *t = tensor(o);
        if (!t || t->dim() != 2)
            refuse("table must be an int32 tensor of batch x max_pages");
        batch = t->size(0);
        width = t->size(1);
        at = (const int32_t *)buffer(o, "table", at::kInt, {batch, width}, index);
    }
};

// A tensor of rows x heads x d float16 whose heads are contiguous in each row.
struct Rows {
    void *at = nullptr;
    int64_t rows = 0, pitch = 0;
    Rows() = default;
    Rows(PyObject *o, const char *name, int64_t heads, int64_t d, int index, int64_t count = -1)
    {
        const at::Tensor *t = tensor(o);
        if (!t || t->scalar_type() != at::kHalf || t->dim() != 3 || !on(*t, index))
            refuse("%s must be a 3-D float16 tensor on cuda:%d", name, index);
        rows = t->size(0);
        if (t->size(1) != heads || t->size(2) != d || (count >= 0 && rows != count))
            refuse("%s must be %lld x %lld x %lld, got %lld x %lld x %lld", name, (long long)(count >= 0 ? count : rows),
                   (long long)heads, (long long)d, (long long)rows, (long long)t->size(1), (long long)t->size(2));
        if (t->stride(2) != 1 || (heads > 1 && t->stride(1) != d))
            refuse("%s's heads must be contiguous in each row", name);
        at = address(*t);
        pitch = rows > 1 ? t->stride(0) : heads * d;
    }
};

// ---- entry points: positional arguments as the functions of q4.py pass them; the last is the index of the device of an
// explicit stream, or None

PyObject *compress(PyObject *const *a)   // w, group, symmetric, device
{
    const int64_t group = known_group(integer(a[1]));
    const at::Tensor *w = tensor(a[0]);
    if (!w || w->dim() != 2)
        refuse("w must be a 2-D float16 tensor");
    const int index = device_of(a[0], "w", a[3]);
    const int64_t n = w->size(0), k = w->size(1), nb = (n + 15) / 16, kb = (k + 127) / 128;
    void *from = buffer(a[0], "w", at::kHalf, w->sizes(), index);
    const int symmetric = PyObject_IsTrue(a[2]);
    if (symmetric < 0)
        throw Raised{};
    at::Tensor codes = empty({nb, kb, 4, 16, 4}, at::kInt, index), words = empty({nb, kb, 16, 128 / group}, at::kInt, index);
    void *c = address(codes), *s = address(words);
    call(index, "gemm_f16_q4_compress",
         [&](void *stream) { return gemm_f16_q4_compress(n, k, (int)group, symmetric, from, c, s, stream); });
    return PyObject_CallFunction(g_matrix, "NNLLL", THPVariable_Wrap(std::move(codes)), THPVariable_Wrap(std::move(words)),
                                 (long long)n, (long long)k, (long long)group);
}

PyObject *expand(PyObject *const *a)   // w, out, device
{
    Matrix w(a[0]);
    const int index = device_of(w.codes_tensor, "w.codes", a[2]);
    w.check(index);
    Output out(a[1], {w.n, w.k}, index);
    call(index, "gemm_f16_q4_expand",
         [&](void *stream) { return gemm_f16_q4_expand(w.n, w.k, w.group, w.codes, w.words, out.at, stream); });
    return out.result();
}

PyObject *gemm(PyObject *const *p)   // a, w, epilogue, out, config, splits, workspace, alpha, device
{
    const at::Tensor *a = tensor(p[0]);
    if (!a || a->dim() != 2)
        refuse("a must be a 2-D float16 tensor");
    const int index = device_of(p[0], "a", p[8]);
    void *from = buffer(p[0], "a", at::kHalf, a->sizes(), index);
    Matrix w(p[1]);
    w.check(index);
    const int64_t m = a->size(0), k = a->size(1);
    if (k != w.k)
        refuse("inner dimensions differ: a is %lld x %lld, w is %lld x %lld", (long long)m, (long long)k, (long long)w.n,
               (long long)w.k);
    const int epilogue = small(p[2]), config = small(p[4]);
    int splits = p[5] == Py_None ? GEMM_F16_SPLITS_AUTO : small(p[5]);
    const float alpha = (float)real(p[7]);
    Output out(p[3], {m, w.n}, index);
    int64_t need = 0;
    if (p[6] == Py_None && m > 0 && w.n > 0) {
        gemm_f16_plan_t plan;
        check(gemm_f16_plan_q4(m, w.n, k, w.group, from, config, splits, &plan), "gemm_f16_plan_q4");
        need = plan.workspace_bytes;
    }
    Workspace ws;
    try {
        ws = Workspace(p[6], need, index);
    } catch (const c10::OutOfMemoryError &) {   // every shape also runs without one
        if (splits != GEMM_F16_SPLITS_AUTO || config != GEMM_F16_CONFIG_AUTO)
            throw;
        splits = 1;
    }
    call(index, "gemm_f16_q4", [&](void *stream) {
        return gemm_f16_q4(m, w.n, k, w.group, from, w.codes, w.words, out.at, alpha, epilogue, config, splits, ws.at, ws.bytes,
                           stream);
    });
    return out.result();
}

PyObject *append(PyObject *const *p)   // cache, k, v, table, lengths, starts, q, cos, sin, interleaved, out, device
{
    Cache cache(p[0], p[11]);
    const gemm_f16_q4_cache_t &c = cache.c;
    const int index = cache.index;
    const Rows k(p[1], "k", c.heads, c.head_dim, index), v(p[2], "v", c.heads, c.head_dim, index, k.rows);
    const Table table(p[3], index);
    if (p[5] == Py_None && k.rows != table.batch)
        refuse("without starts there is one row for each of the %lld sequences, got %lld", (long long)table.batch,
               (long long)k.rows);
    const auto *lengths = (const int32_t *)buffer(p[4], "lengths", at::kInt, {table.batch}, index);
    const auto *starts = p[5] == Py_None ? nullptr : (const int32_t *)buffer(p[5], "starts", at::kInt, {table.batch + 1}, index);
    if ((p[7] == Py_None) != (p[8] == Py_None))
        refuse("cos and sin come together");
    int64_t positions = 0, rotary = 0;
    const float *cos = nullptr, *sin = nullptr;
    if (p[7] != Py_None) {
        const at::Tensor *t = tensor(p[7]);
        if (!t || t->dim() != 2)
            refuse("cos must be a float32 tensor of positions x rotary / 2");
        positions = t->size(0);
        rotary = 2 * std::min<int64_t>(t->size(1), INT32_MAX);
        if (rotary < 16 || rotary > c.head_dim || rotary % 16 || !positions)
            refuse("cos must have 8, 16, ... %d columns and a row at least, got %lld x %lld", (int)(c.head_dim / 2),
                   (long long)positions, (long long)(rotary / 2));
        cos = (const float *)buffer(p[7], "cos", at::kFloat, t->sizes(), index);
        sin = (const float *)buffer(p[8], "sin", at::kFloat, t->sizes(), index);
    }
    const int interleaved = PyObject_IsTrue(p[9]);
    if (interleaved < 0)
        throw Raised{};
    Rows q;
    int64_t q_heads = 0;
    if (p[6] != Py_None) {
        const at::Tensor *t = tensor(p[6]);
        if (!t || t->dim() != 3 || t->size(1) < 1 || t->size(1) > INT32_MAX)
            refuse("q must be a tensor of tokens x q_heads x head_dim");
        q_heads = t->size(1);
        q = Rows(p[6], "q", q_heads, c.head_dim, index, k.rows);
    } else if (p[10] != Py_None) {
        refuse("out is for the rotated queries: give q");
    }
    const auto run = [&](void *to) {
        call(index, "gemm_f16_q4_cache_append", [&](void *stream) {
            return gemm_f16_q4_cache_append(&c, table.batch, k.rows, table.width, k.at, k.pitch, v.at, v.pitch, table.at, lengths,
                                            starts, q.at, q.pitch, to, (int)q_heads, cos, sin, positions, (int)rotary,
                                            interleaved, stream);
        });
    };
    if (p[6] == Py_None) {
        run(nullptr);
        Py_RETURN_NONE;
    }
    Output out(p[10], {k.rows, q_heads, (int64_t)c.head_dim}, index);
    run(out.at);
    return out.result();
}

PyObject *read(PyObject *const *p)   // cache, table, starts, total, first, device
{
    Cache cache(p[0], p[5]);
    const int index = cache.index;
    const Table table(p[1], index);
    const auto *starts = (const int32_t *)buffer(p[2], "starts", at::kInt, {table.batch + 1}, index);
    const auto *first = p[4] == Py_None ? nullptr : (const int32_t *)buffer(p[4], "first", at::kInt, {table.batch}, index);
    const int64_t total = integer(p[3]);
    if (total < 0)
        refuse("total must not be negative");
    const int64_t shape[3] = {total, cache.c.heads, cache.c.head_dim};
    at::Tensor k = empty(shape, at::kHalf, index), v = empty(shape, at::kHalf, index);
    void *k_at = address(k), *v_at = address(v);
    call(index, "gemm_f16_q4_cache_read", [&](void *stream) {
        return gemm_f16_q4_cache_read(&cache.c, table.batch, total, table.width, table.at, first, starts, k_at, v_at, stream);
    });
    return Py_BuildValue("NN", THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v)));
}

PyObject *attention(PyObject *const *p)   // q, cache, table, lengths, scale, out, splits, workspace, max_length, device
{
    Cache cache(p[1], p[9]);
    const gemm_f16_q4_cache_t &c = cache.c;
    const int index = cache.index;
    const at::Tensor *t = tensor(p[0]);
    if (!t || t->dim() != 3)
        refuse("q must be a tensor of batch x q_heads x head_dim");
    const int64_t q_heads = t->size(1);
    if (q_heads < 1 || q_heads > INT32_MAX || c.heads < 1 || q_heads % c.heads)
        refuse("q's heads must be a multiple of the cache's %d, got %lld", (int)c.heads, (long long)q_heads);
    const Rows q(p[0], "q", q_heads, c.head_dim, index);
    const Table table(p[2], index);
    if (table.batch != q.rows)
        refuse("table must be an int32 tensor of %lld x max_pages", (long long)q.rows);
    const auto *lengths = (const int32_t *)buffer(p[3], "lengths", at::kInt, {q.rows}, index);
    const float scale = p[4] == Py_None ? (float)(1.0 / std::sqrt((double)c.head_dim)) : (float)real(p[4]);
    const int splits = p[6] == Py_None ? GEMM_F16_SPLITS_AUTO : small(p[6]);
    int64_t longest = p[8] == Py_None ? 0 : integer(p[8]);
    if (longest < 0)
        refuse("max_length must not be negative");
    int64_t room;   // (a table without rows may be of any width)
    if (__builtin_mul_overflow(table.width, (int64_t)c.page_size, &room))
        room = INT64_MAX;
    longest = longest ? std::min(longest, room) : room;
    Output out(p[5], {q.rows, q_heads, (int64_t)c.head_dim}, index);
    int64_t need = 0;
    if (p[7] == Py_None) {
        gemm_f16_plan_t plan;
        check(gemm_f16_plan_q4_attention(q.rows, (int)q_heads, c.heads, c.head_dim, c.group, longest, splits, &plan),
              "gemm_f16_plan_q4_attention");
        need = plan.workspace_bytes;
    }
    Workspace ws(p[7], need, index);
    call(index, "gemm_f16_q4_attention", [&](void *stream) {
        return gemm_f16_q4_attention(&c, q.rows, (int)q_heads, table.width, q.at, q.pitch, table.at, lengths, scale, out.at,
                                     splits, longest, ws.at, ws.bytes, stream);
    });
    return out.result();
}

template <PyObject *(*F)(PyObject *const *), int COUNT>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    if (count != COUNT || !g_matrix) {
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

PyObject *setup(PyObject *, PyObject *args)
{
    if (!PyArg_ParseTuple(args, "OOOO", &g_matrix, &g_cache, &g_error, &g_stream))
        return nullptr;
    for (PyObject *o : {g_matrix, g_cache, g_error, g_stream})
        Py_INCREF(o);
    Py_RETURN_NONE;
}

#define GEMM_F16_Q4_ENTRY(name, count) {#name, (PyCFunction)(void (*)(void))(entry<name, count>), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {GEMM_F16_Q4_ENTRY(compress, 4), GEMM_F16_Q4_ENTRY(expand, 3), GEMM_F16_Q4_ENTRY(gemm, 9),
                           GEMM_F16_Q4_ENTRY(append, 12), GEMM_F16_Q4_ENTRY(read, 6), GEMM_F16_Q4_ENTRY(attention, 10),
                           {"setup", setup, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_q4_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__q4_binding() { return PyModule_Create(&g_module); }
