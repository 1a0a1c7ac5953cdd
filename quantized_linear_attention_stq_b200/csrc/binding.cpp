// binding.cpp -- the usual case of the binding's calls for the layers next to the quantized ones: arguments
// of the right types, shapes and layout, on the current device. A call's checks and its hand-over through
// ctypes cost 7 us of host time, three times the kernel of a small step; here they cost 1.
//
// Each function takes the arguments of the api.py function of its name, checks them and calls the library.
// It returns the library's status, or -1 without having called it where anything is out of the ordinary: the
// Python code then goes on, which knows the rarer cases and names what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <initializer_list>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/stq.h"

namespace {

using Shape = std::initializer_list<int64_t>;

// One call's tensors: all on the device of the first, which is the current one.
struct Args {
    PyObject *const *v;
    bool ok = true;
    int device = -1;

    const c10::TensorImpl *any(int i)
    {
        if (!ok || !THPVariable_CheckExact(v[i])) {
            ok = false;
            return nullptr;
        }
        const c10::TensorImpl *t = THPVariable_Unpack(v[i]).unsafeGetTensorImpl();
        const c10::Device d = t->device();
        ok = t->layout() == c10::kStrided && d.is_cuda() && (device < 0 || d.index() == device);
        if (!ok) return nullptr;
        if (device < 0) {
            device = d.index();
            ok = device == c10::cuda::current_device();
        }
        return t;
    }
    // a contiguous tensor of this type and number of dimensions
    const c10::TensorImpl *tensor(int i, c10::ScalarType kind, int64_t dims)
    {
        const c10::TensorImpl *t = any(i);
        if (t && (t->dtype() != c10::scalarTypeToTypeMeta(kind) || t->dim() != dims || !t->is_contiguous())) ok = false;
        return ok ? t : nullptr;
    }
    void *data(int i, c10::ScalarType kind, Shape shape)
    {
        const c10::TensorImpl *t = tensor(i, kind, (int64_t)shape.size());
        if (!ok || t->sizes() != c10::IntArrayRef(shape)) {
            ok = false;
            return nullptr;
        }
        return const_cast<void *>(t->data());
    }
    // float32 or bfloat16
    const c10::TensorImpl *floats(int i, int64_t dims, c10::ScalarType *kind, int32_t *code)
    {
        const c10::TensorImpl *t = any(i);
        if (!t) return nullptr;
        *kind = c10::typeMetaToScalarType(t->dtype());
        *code = *kind == c10::kBFloat16 ? STQ_BF16 : STQ_F32;
        ok = (*kind == c10::kBFloat16 || *kind == c10::kFloat) && t->dim() == dims;
        return ok ? t : nullptr;
    }
    int32_t *status(int i) { return v[i] == Py_None ? nullptr : static_cast<int32_t *>(data(i, c10::kInt, {1})); }
    // the stream argument (None: the current one)
    void *stream(int i)
    {
        if (ok && v[i] == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        ok = false;
        return nullptr;
    }
    // a workspace argument (None: none)
    void *workspace(int i, size_t need, size_t *bytes)
    {
        *bytes = 0;
        if (!ok || v[i] == Py_None || need == 0) return nullptr;
        const c10::TensorImpl *t = any(i);
        if (!t || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        *bytes = (size_t)t->numel() * t->itemsize();
        ok = *bytes >= need;
        return const_cast<void *>(t->data());
    }
};

bool fits(std::initializer_list<int64_t> sizes)
{
    for (int64_t n : sizes)
        if (n > 2147483647 || n < -2147483648LL) return false;
    return true;
}

// The call without the interpreter's lock; -1 where an argument was not the usual one.
template <class Call>
PyObject *finish(const Args &a, Call call)
{
    if (!a.ok) return PyLong_FromLong(-1);
    stq_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong((long)st);
}

bool count(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected", want);
    return false;
}

// states, slots, q, k, v, alpha, o, status, stream
PyObject *decay_step(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (!count(n, 9)) return nullptr;
    Args a{args};
    c10::ScalarType kind;
    int32_t code;
    const c10::TensorImpl *q = a.floats(2, 3, &kind, &code), *st = a.tensor(0, c10::kFloat, 4);
    if (!a.ok) return PyLong_FromLong(-1);
    const int64_t B = q->size(0), H = q->size(1), d = q->size(2), P = st->size(0);
    float *states = (float *)a.data(0, c10::kFloat, {P, H, d, d});
    const int32_t *slots = (int32_t *)a.data(1, c10::kInt, {B});
    const void *x[3] = {a.data(2, kind, {B, H, d}), a.data(3, kind, {B, H, d}), a.data(4, kind, {B, H, d})};
    const float *alpha = (float *)a.data(5, c10::kFloat, {B, H});
    float *o = (float *)a.data(6, c10::kFloat, {B, H, d});
    int32_t *status = a.status(7);
    void *s = a.stream(8);
    a.ok = a.ok && fits({B, H, d, P});
    return finish(a, [&] {
        return stq_decay_step((int32_t)B, (int32_t)H, (int32_t)d, code, states, (int32_t)P, slots, x[0], x[1], x[2],
                              alpha, o, status, s);
    });
}

// states, slots, q, k, v, alpha, o, lens, workspace, status, stream
PyObject *decay_prefill(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (!count(n, 11)) return nullptr;
    Args a{args};
    c10::ScalarType kind;
    int32_t code;
    const c10::TensorImpl *q = a.floats(2, 4, &kind, &code), *st = a.tensor(0, c10::kFloat, 4);
    if (!a.ok) return PyLong_FromLong(-1);
    const int64_t B = q->size(0), H = q->size(1), T = q->size(2), d = q->size(3), P = st->size(0);
    float *states = (float *)a.data(0, c10::kFloat, {P, H, d, d});
    const int32_t *slots = (int32_t *)a.data(1, c10::kInt, {B});
    const void *x[3] = {a.data(2, kind, {B, H, T, d}), a.data(3, kind, {B, H, T, d}), a.data(4, kind, {B, H, T, d})};
    const float *alpha = (float *)a.data(5, c10::kFloat, {B, H, T});
    float *o = (float *)a.data(6, c10::kFloat, {B, H, T, d});
    const int32_t *lens = args[7] == Py_None ? nullptr : (int32_t *)a.data(7, c10::kInt, {B});
    a.ok = a.ok && fits({B, H, T, d, P});
    size_t bytes = 0;
    const size_t need = a.ok ? stq_decay_prefill_workspace_bytes((int32_t)B, (int32_t)H, (int32_t)T, (int32_t)d,
        code) : 0;
    void *ws = a.workspace(8, need, &bytes);
    int32_t *status = a.status(9);
    void *s = a.stream(10);
    return finish(a, [&] {
        return stq_decay_prefill((int32_t)B, (int32_t)H, (int32_t)T, (int32_t)d, code, states, (int32_t)P, slots,
                                 x[0], x[1], x[2], alpha, lens, o, ws, bytes, status, s);
    });
}

// table, lens, fresh, free_pages, free_head, slot_map, starts, lens_out, head_out, page_size, status, stream
PyObject *page_plan(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (!count(n, 12)) return nullptr;
    Args a{args};
    const c10::TensorImpl *t = a.tensor(0, c10::kInt, 2), *f = a.tensor(3, c10::kInt, 1), *m = a.tensor(5,
        c10::kInt, 1);
    if (!a.ok || !PyLong_CheckExact(args[9])) return PyLong_FromLong(-1);
    int over = 0;
    const long page = PyLong_AsLongAndOverflow(args[9], &over);
    const int64_t B = t->size(0), W = t->size(1), F = f->size(0), N = m->size(0);
    int32_t *x[9];
    const int64_t len[9] = {0, B, B, F, 1, N, B + 1, B, 1};
    x[0] = (int32_t *)a.data(0, c10::kInt, {B, W});
    for (int i = 1; i < 9; ++i) x[i] = (int32_t *)a.data(i, c10::kInt, {len[i]});
    int32_t *status = a.status(10);
    void *s = a.stream(11);
    a.ok = a.ok && !over && fits({B, W, F, N, page});
    return finish(a, [&] {
        return stq_page_plan((int32_t)B, (int32_t)W, (int32_t)page, x[0], x[1], x[2], x[3], (int32_t)F, x[4], x[5],
                             (int32_t)N, x[6], x[7], x[8], status, s);
    });
}

// k_pages, v_pages, slot_map, k, v, status, stream
PyObject *page_write(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (!count(n, 7)) return nullptr;
    Args a{args};
    c10::ScalarType kind;
    int32_t code;
    const c10::TensorImpl *k = a.floats(3, 3, &kind, &code), *v = a.any(4), *kp = a.any(0);
    if (!a.ok || kp->dim() != 4 || v->dtype() != k->dtype() || v->sizes() != k->sizes()) return PyLong_FromLong(-1);
    const int64_t N = k->size(0), H = k->size(1), d = k->size(2), P = kp->size(0), page = kp->size(2);
    int64_t row[2] = {H * d, H * d};
    for (int i = 0; i < 2; ++i) {  // the stride of a single entry means nothing
        const c10::TensorImpl *t = i ? v : k;
        if (N > 1) row[i] = t->stride(0);
        a.ok = a.ok && (d < 2 || t->stride(2) == 1) && (H < 2 || t->stride(1) == d) && row[i] >= H * d;
    }
    void *pages[2] = {a.data(0, kind, {P, H, page, d}), a.data(1, kind, {P, H, page, d})};
    const int32_t *slots = (int32_t *)a.data(2, c10::kInt, {N});
    int32_t *status = a.status(5);
    void *s = a.stream(6);
    a.ok = a.ok && fits({N, H, d, P, page});
    return finish(a, [&] {
        return stq_page_write((int32_t)N, (int32_t)H, (int32_t)d, code, (int32_t)page, (int32_t)P, pages[0], pages[1],
                              slots, k->data(), v->data(), row[0], row[1], status, s);
    });
}

// q, k_pages, v_pages, table, lens, o, scale, workspace, status, stream
PyObject *paged_attention(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (!count(n, 10)) return nullptr;
    Args a{args};
    c10::ScalarType kind;
    int32_t code;
    const c10::TensorImpl *q = a.floats(0, 3, &kind, &code), *kp = a.any(1), *t = a.tensor(3, c10::kInt, 2);
    if (!a.ok || kp->dim() != 4 || !PyFloat_CheckExact(args[6])) return PyLong_FromLong(-1);
    const double scale = PyFloat_AS_DOUBLE(args[6]);
    const int64_t B = q->size(0), Hq = q->size(1), d = q->size(2), P = kp->size(0), H = kp->size(1), page =
        kp->size(2), W = t->size(1);
    const void *x = a.data(0, kind, {B, Hq, d});
    const void *pages[2] = {a.data(1, kind, {P, H, page, d}), a.data(2, kind, {P, H, page, d})};
    const int32_t *table = (int32_t *)a.data(3, c10::kInt, {B, W}), *lens = (int32_t *)a.data(4, c10::kInt, {B});
    float *o = (float *)a.data(5, c10::kFloat, {B, Hq, d});
    a.ok = a.ok && fits({B, Hq, d, P, H, page, W});
    size_t bytes = 0;
    const size_t need = a.ok ? stq_paged_attention_workspace_bytes((int32_t)B, (int32_t)Hq, (int32_t)d, (int32_t)H) : 0;
    void *ws = a.workspace(7, need, &bytes);
    int32_t *status = a.status(8);
    void *s = a.stream(9);
    return finish(a, [&] {
        return stq_paged_attention((int32_t)B, (int32_t)Hq, (int32_t)H, (int32_t)d, code, (int32_t)page, (int32_t)P,
                                   (int32_t)W, x, pages[0], pages[1], table, lens, (float)scale, o, ws, bytes, status,
                                   s);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    try {
        return F(self, args, n);
    } catch (...) {  // what c10 has to say about a tensor is said by the Python code again
        return PyLong_FromLong(-1);
    }
}

#define STQ_METHOD(f) {#f, (PyCFunction)(void (*)(void))guarded<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {STQ_METHOD(decay_step),  STQ_METHOD(decay_prefill), STQ_METHOD(page_plan),
                         STQ_METHOD(page_write),  STQ_METHOD(paged_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#ifndef STQ_BUILT_FOR
#error "STQ_BUILT_FOR names the torch and Python that this is built against"
#endif

PyMODINIT_FUNC PyInit__binding()
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", STQ_BUILT_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
