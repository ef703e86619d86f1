// i8_binding.cpp -- the Python side of include/gemm_f16_i8.h.  As in
// q4_binding.cpp: a layer of experts makes half a dozen calls whose kernels
// take a few microseconds each, so their checks are compiled.
#include "binding.h"

#include "gemm_f16_i8.h"

namespace {

PyObject *g_matrix, *g_order;   // I8Matrix, ExpertOrder

// a * b, the number of rows of a tensor (one without elements may have any sizes).
int64_t times(int64_t a, int64_t b)
{
    int64_t c;
    if (__builtin_mul_overflow(a, b, &c))
        refuse("too many rows");
    return c;
}

// An I8Matrix: codes of `lead` leading sizes, rows and a pitch, and a scale for each row.
struct Matrix {
    PyObject *codes_tensor, *scales_tensor;
    at::IntArrayRef sizes;   // of the codes
    int64_t k, pitch, rows = 1;
    void *codes = nullptr;
    const float *scales = nullptr;
    int index;
    Matrix(PyObject *m, const char *name, PyObject *stream_device)
    {
        if (!PyObject_TypeCheck(m, (PyTypeObject *)g_matrix) || PyTuple_GET_SIZE(m) != 3)
            refuse("%s must be an I8Matrix (as i8_compress returns)", name);
        codes_tensor = PyTuple_GET_ITEM(m, 0);
        scales_tensor = PyTuple_GET_ITEM(m, 1);
        k = integer(PyTuple_GET_ITEM(m, 2));
        const at::Tensor *t = tensor(codes_tensor);
        if (!t || t->dim() < 2)
            refuse("%s.codes must be an int8 tensor of ... x rows x pitch", name);
        index = device_of(codes_tensor, name, stream_device);
        sizes = t->sizes();
        pitch = sizes.back();
        if (k < 0 || k > GEMM_F16_I8_MAX_K || pitch < (k + 15) / 16 * 16 || pitch % 16)
            refuse("%s.codes must have rows of k = %lld codes padded to a multiple of 16, got %lld", name, (long long)k,
                   (long long)pitch);
        for (size_t i = 0; i + 1 < sizes.size(); ++i)
            rows = times(rows, sizes[i]);
        codes = buffer(codes_tensor, name, at::kChar, sizes, index);
        scales = (const float *)buffer(scales_tensor, name, at::kFloat, sizes.slice(0, sizes.size() - 1), index);
    }
};

// ---- entry points: positional arguments as the functions of i8.py pass them; the last is the index of the device of an
// explicit stream, or None

PyObject *compress(PyObject *const *a)   // x, device
{
    const at::Tensor *x = tensor(a[0]);
    if (!x || x->scalar_type() != at::kHalf || x->dim() < 2)
        refuse("x must be a float16 tensor of ... x rows x k");
    const int index = device_of(a[0], "x", a[1]);
    const int64_t dims = x->dim(), k = x->size(dims - 1);
    if (k > GEMM_F16_I8_MAX_K)
        refuse("x must have rows of at most %lld elements", (long long)GEMM_F16_I8_MAX_K);
    // rows may lie apart, all by the same distance
    int64_t rows = 1, stride = k;
    bool first = true;
    for (int64_t d = dims - 2; d >= 0; --d) {
        if (x->size(d) != 1 && x->numel()) {
            if (first)
                stride = x->stride(d);
            else if (x->stride(d) != times(stride, rows))
                refuse("x's rows must lie the same distance apart");
            first = false;
        }
        rows = times(rows, x->size(d));
    }
    if (x->numel() && k > 1 && x->stride(dims - 1) != 1)
        refuse("x's rows must be contiguous");
    if (x->numel() && stride < k)
        refuse("x's rows must not overlap");
    std::vector<int64_t> shape(x->sizes().begin(), x->sizes().end());
    shape.back() = gemm_f16_i8_pitch(k);
    at::Tensor codes = empty(shape, at::kChar, index);
    shape.pop_back();
    at::Tensor scales = empty(shape, at::kFloat, index);
    void *from = address(*x), *c = address(codes), *s = address(scales);
    call(index, "gemm_f16_i8_compress",
         [&](void *stream) { return gemm_f16_i8_compress(rows, k, from, stride, c, (float *)s, stream); });
    return PyObject_CallFunction(g_matrix, "NNL", THPVariable_Wrap(std::move(codes)), THPVariable_Wrap(std::move(scales)),
                                 (long long)k);
}

PyObject *expand(PyObject *const *p)   // x, out, device
{
    const Matrix x(p[0], "x", p[2]);
    std::vector<int64_t> shape(x.sizes.begin(), x.sizes.end());
    shape.back() = x.k;
    Output out(p[1], shape, x.index);
    call(x.index, "gemm_f16_i8_expand", [&](void *stream) {
        return gemm_f16_i8_expand(x.rows, x.k, x.codes, x.pitch, x.scales, out.at, stream);
    });
    return out.result();
}

PyObject *gemm(PyObject *const *p)   // a, w, epilogue, out, config, splits, workspace, alpha, device
{
    const Matrix a(p[0], "a", p[8]), w(p[1], "w", p[8]);
    if (a.sizes.size() != 2 || w.sizes.size() != 2)
        refuse("a and w must be matrices (2-D codes)");
    if (w.index != a.index)
        refuse("a and w are on different devices");
    if (a.k != w.k)
        refuse("inner dimensions differ: a is %lld x %lld, w is %lld x %lld", (long long)a.rows, (long long)a.k,
               (long long)w.rows, (long long)w.k);
    const int epilogue = small(p[2]), config = small(p[4]);
    int splits = p[5] == Py_None ? GEMM_F16_SPLITS_AUTO : small(p[5]);
    const float alpha = (float)real(p[7]);
    Output out(p[3], {a.rows, w.rows}, a.index);
    int64_t need = 0;
    if (p[6] == Py_None && a.rows > 0 && w.rows > 0) {
        gemm_f16_plan_t plan;
        check(gemm_f16_plan_i8(a.rows, w.rows, a.k, config, splits, &plan), "gemm_f16_plan_i8");
        need = plan.workspace_bytes;
    }
    Workspace ws;
    try {
        ws = Workspace(p[6], need, a.index);
    } catch (const c10::OutOfMemoryError &) {   // every shape also runs without one
        if (splits != GEMM_F16_SPLITS_AUTO)
            throw;
        splits = 1;
    }
    call(a.index, "gemm_f16_i8", [&](void *stream) {
        return gemm_f16_i8(a.rows, w.rows, a.k, a.codes, a.pitch, a.scales, w.codes, w.pitch, w.scales, out.at, alpha, epilogue,
                           config, splits, ws.at, ws.bytes, stream);
    });
    return out.result();
}

PyObject *route(PyObject *const *p)   // logits, top_k, score, bias, groups, top_groups, renormalise, scale, device
{
    const at::Tensor *x = tensor(p[0]);
    if (!x || x->dim() != 2 || (x->scalar_type() != at::kHalf && x->scalar_type() != at::kFloat))
        refuse("logits must be a float16 or float32 tensor of tokens x experts");
    const int index = device_of(p[0], "logits", p[8]);
    const int64_t tokens = x->size(0), experts = x->size(1);
    const int top_k = small(p[1]), score = small(p[2]), groups = small(p[4]), top_groups = small(p[5]);
    if (experts < 1 || experts > GEMM_F16_MAX_EXPERTS)
        refuse("logits must be of 1 to %d experts, got %lld", GEMM_F16_MAX_EXPERTS, (long long)experts);
    if (top_k < 1 || top_k > experts || top_k > GEMM_F16_MAX_TOP_K)
        refuse("top_k must be at least 1 and at most %d and the number of experts, got %d", GEMM_F16_MAX_TOP_K, top_k);
    if (groups < 1 || experts % groups || groups > GEMM_F16_MAX_EXPERT_GROUPS || top_groups < 1 || top_groups > groups)
        refuse("groups must divide the %lld experts (at most %d groups) and top_groups be 1 to groups, got %d and %d",
               (long long)experts, GEMM_F16_MAX_EXPERT_GROUPS, groups, top_groups);
    if (x->numel() && experts > 1 && x->stride(1) != 1)
        refuse("logits' rows must be contiguous");
    const int64_t stride = tokens > 1 ? x->stride(0) : experts;
    if (stride < experts)
        refuse("logits' rows must not overlap");
    const auto *bias = p[3] == Py_None ? nullptr : (const float *)buffer(p[3], "bias", at::kFloat, {experts}, index);
    const int renormalise = PyObject_IsTrue(p[6]);
    if (renormalise < 0)
        throw Raised{};
    const float scale = (float)real(p[7]);
    const int half = x->scalar_type() == at::kHalf;
    at::Tensor ids = empty({tokens, top_k}, at::kInt, index), weights = empty({tokens, top_k}, at::kFloat, index);
    void *from = address(*x), *i = address(ids), *w = address(weights);
    call(index, "gemm_f16_route", [&](void *stream) {
        return gemm_f16_route(tokens, (int)experts, top_k, from, half, stride, score, bias, groups, top_groups, renormalise, scale,
                              (int32_t *)i, (float *)w, stream);
    });
    return Py_BuildValue("NN", THPVariable_Wrap(std::move(ids)), THPVariable_Wrap(std::move(weights)));
}

PyObject *order(PyObject *const *p)   // ids, experts, device
{
    const at::Tensor *t = tensor(p[0]);
    if (!t || t->dim() != 2)
        refuse("ids must be an int32 tensor of tokens x top_k");
    const int index = device_of(p[0], "ids", p[2]), experts = small(p[1]);
    if (experts < 1 || experts > GEMM_F16_MAX_EXPERTS)
        refuse("experts must be 1 to %d, got %d", GEMM_F16_MAX_EXPERTS, experts);
    const auto *ids = (const int32_t *)buffer(p[0], "ids", at::kInt, t->sizes(), index);
    at::Tensor made = empty(t->sizes(), at::kInt, index), starts = empty({experts + 1}, at::kInt, index);
    const int64_t pairs = t->numel();
    void *o = address(made), *s = address(starts);
    call(index, "gemm_f16_expert_order", [&](void *stream) {
        return gemm_f16_expert_order(pairs, experts, ids, (int32_t *)o, (int32_t *)s, stream);
    });
    return PyObject_CallFunction(g_order, "NN", THPVariable_Wrap(std::move(made)), THPVariable_Wrap(std::move(starts)));
}

PyObject *experts(PyObject *const *p)   // a, w, order, epilogue, out, config, alpha, device
{
    const Matrix a(p[0], "a", p[7]), w(p[1], "w", p[7]);
    if (w.sizes.size() != 3)
        refuse("w must be of experts x n x k (3-D codes)");
    if (w.index != a.index)
        refuse("a and w are on different devices");
    if (a.k != w.k)
        refuse("inner dimensions differ: a's rows have %lld elements, w's %lld", (long long)a.k, (long long)w.k);
    if (!PyObject_TypeCheck(p[2], (PyTypeObject *)g_order) || PyTuple_GET_SIZE(p[2]) != 2)
        refuse("order must be an ExpertOrder (as expert_order returns)");
    PyObject *o = PyTuple_GET_ITEM(p[2], 0);
    const at::Tensor *t = tensor(o);
    if (!t || t->dim() != 2)
        refuse("order.order must be an int32 tensor of tokens x top_k");
    const int64_t tokens = t->size(0), top_k = t->size(1), pairs = t->numel(), count = w.sizes[0], n = w.sizes[1];
    const auto *places = (const int32_t *)buffer(o, "order.order", at::kInt, t->sizes(), a.index);
    const auto *starts = (const int32_t *)buffer(PyTuple_GET_ITEM(p[2], 1), "order.starts", at::kInt, {count + 1}, a.index);
    if (count < 1 || count > GEMM_F16_MAX_EXPERTS)
        refuse("w must be of 1 to %d experts, got %lld", GEMM_F16_MAX_EXPERTS, (long long)count);
    if (a.rows != tokens && a.rows != pairs)
        refuse("a must have a row for each of %lld tokens or of %lld pairs, got %lld", (long long)tokens, (long long)pairs,
               (long long)a.rows);
    const int epilogue = small(p[3]), config = small(p[5]);
    const float alpha = (float)real(p[6]);
    Output out(p[4], {tokens, top_k, n}, a.index);
    const int64_t per_row = a.rows > 0 && pairs > 0 ? pairs / a.rows : 1;
    call(a.index, "gemm_f16_i8_experts", [&](void *stream) {
        return gemm_f16_i8_experts(pairs, per_row, (int)count, n, a.k, a.codes, a.pitch, a.scales, w.codes, w.pitch, w.scales,
                                   places, starts, out.at, alpha, epilogue, config, stream);
    });
    return out.result();
}

PyObject *sum(PyObject *const *p)   // y, weights, out, device
{
    const at::Tensor *y = tensor(p[0]);
    if (!y || y->dim() != 3)
        refuse("y must be a float16 tensor of tokens x top_k x n");
    const int index = device_of(p[0], "y", p[3]);
    const int64_t tokens = y->size(0), top_k = y->size(1), n = y->size(2);
    void *from = buffer(p[0], "y", at::kHalf, y->sizes(), index);
    const auto *weights = (const float *)buffer(p[1], "weights", at::kFloat, {tokens, top_k}, index);
    Output out(p[2], {tokens, n}, index);
    call(index, "gemm_f16_expert_sum",
         [&](void *stream) { return gemm_f16_expert_sum(tokens, top_k, n, from, weights, out.at, stream); });
    return out.result();
}

PyObject *setup(PyObject *, PyObject *args)
{
    if (!PyArg_ParseTuple(args, "OOOO", &g_matrix, &g_order, &g_error, &g_stream))
        return nullptr;
    for (PyObject *o : {g_matrix, g_order, g_error, g_stream})
        Py_INCREF(o);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {GEMM_F16_ENTRY(compress, 2), GEMM_F16_ENTRY(expand, 3), GEMM_F16_ENTRY(gemm, 9),
                           GEMM_F16_ENTRY(route, 9), GEMM_F16_ENTRY(order, 3), GEMM_F16_ENTRY(experts, 8),
                           GEMM_F16_ENTRY(sum, 4), {"setup", setup, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_i8_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__i8_binding() { return PyModule_Create(&g_module); }
