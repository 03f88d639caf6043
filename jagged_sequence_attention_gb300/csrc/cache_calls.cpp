// The two paged-cache calls of a served step, from Python: argument checks and marshalling of
// jfa_cache_append and jfa_cache_fwd on tensors, compiled because a small call takes a few
// microseconds on the GPU and the same checks took about ten in the interpreter.  Nothing is
// computed here; the calls go to the entry points of the loaded library, whose addresses the
// Python binding hands over.
//
// A failed check raises ValueError with what is wrong; the Python binding turns it into its
// own error with JFA_ERR_INVALID_ARG.  Otherwise a call returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "jfa.h"

namespace {

decltype(&jfa_cache_append) g_append = nullptr;
decltype(&jfa_cache_fwd) g_fwd = nullptr;

struct Info {  // of a cache, in a capsule that its Python object holds
    jfa_cache handle;
    c10::ScalarType type;
    int device, Hkv, D;
};

Info* info_of(PyObject* o) { return static_cast<Info*>(PyCapsule_GetPointer(o, "jfa_cache")); }

bool bad(const char* what) {
    PyErr_SetString(PyExc_ValueError, what);
    return false;
}

bool tensor(PyObject* o, const at::Tensor** t) {
    if (!THPVariable_Check(o)) return bad("a tensor was expected");
    *t = &THPVariable_Unpack(o);
    return true;
}

struct Batch {
    int32_t B, max_pages;
    const int32_t *q_off, *kv_lens, *table;
};

bool batch(const Info* c, PyObject* qo, PyObject* kl, PyObject* pt, Batch* b) {
    const at::Tensor *q, *k, *t;
    if (!tensor(qo, &q) || !tensor(kl, &k) || !tensor(pt, &t)) return false;
    if (t->dim() != 2 || k->numel() != t->size(0) || q->numel() != t->size(0) + 1 || t->size(0) > INT32_MAX ||
        t->size(1) > INT32_MAX)
        return bad("q_offsets [B + 1], kv_lens [B] and page_table [B, max_pages] disagree");
    for (const at::Tensor* x : {q, k, t})
        if (x->scalar_type() != at::kInt || x->get_device() != c->device || !x->is_contiguous())
            return bad("q_offsets, kv_lens and page_table must be contiguous int32 tensors on the cache's device");
    *b = Batch{int32_t(t->size(0)), int32_t(t->size(1)), static_cast<const int32_t*>(q->data_ptr()),
               static_cast<const int32_t*>(k->data_ptr()), static_cast<const int32_t*>(t->data_ptr())};
    return true;
}

// Rows [T, heads, D] whose heads are dense (heads, T: required, or -1 and set), their token
// stride and address.
bool rows(const Info* c, PyObject* o, int64_t* heads, int64_t* T, int64_t* stride, void** p) {
    const at::Tensor* t;
    if (!tensor(o, &t)) return false;
    if (t->dim() != 3 || t->size(2) != c->D || (*heads >= 0 && t->size(1) != *heads) || (*T >= 0 && t->size(0) != *T) ||
        t->scalar_type() != c->type || t->get_device() != c->device || t->size(1) > INT32_MAX)
        return bad("rows must be [T, heads, D] in the cache's type, on its device");
    *T = t->size(0);
    *heads = t->size(1);
    if (*T * *heads > 0 && (t->stride(2) != 1 || (*heads > 1 && t->stride(1) != c->D)))
        return bad("the heads of a row must be dense");
    *stride = *T > 1 ? t->stride(0) : *heads * c->D;  // one token (or none): torch leaves its stride free
    *p = t->data_ptr();
    return true;
}

// The given stream (a handle), or the current one of the cache's device.
bool stream_of(const Info* c, PyObject* o, void** s) {
    if (o == Py_None) {
        *s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c->device)).stream();
        return true;
    }
    *s = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
}

// set(address of jfa_cache_append, of jfa_cache_fwd)
PyObject* set_calls(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "two addresses");
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_fwd = reinterpret_cast<decltype(g_fwd)>(PyLong_AsVoidPtr(a[1]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// describe(handle, K): the cache's facts, taken from its key array
PyObject* describe(PyObject*, PyObject* const* a, Py_ssize_t n) {
    const at::Tensor* k;
    if (n != 2) return PyErr_Format(PyExc_TypeError, "a handle and the key array");
    void* h = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred() || !tensor(a[1], &k)) return nullptr;
    if (k->dim() != 4) return bad("the key array has four dimensions"), nullptr;
    Info* i = new (std::nothrow) Info{static_cast<jfa_cache>(h), k->scalar_type(), int(k->get_device()), int(k->size(2)),
                                      int(k->size(3))};
    if (!i) return PyErr_NoMemory();
    return PyCapsule_New(i, "jfa_cache", [](PyObject* o) { delete info_of(o); });
}

// append(info, K, V, q_offsets, kv_lens, page_table, Q, Q_out, rot, rot_kind, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 11) return PyErr_Format(PyExc_TypeError, "11 arguments");
    const Info* c = info_of(a[0]);
    Batch b;
    if (!c || !g_append || !batch(c, a[3], a[4], a[5], &b)) return nullptr;
    int64_t T = -1, kh = c->Hkv, H = -1, ks, vs, qs = 0, os = 0;
    void *K, *V, *Q = nullptr, *O = nullptr, *st;
    if (!rows(c, a[1], &kh, &T, &ks, &K) || !rows(c, a[2], &kh, &T, &vs, &V)) return nullptr;
    if (a[6] != Py_None) {
        if (!rows(c, a[6], &H, &T, &qs, &Q) || !rows(c, a[7], &H, &T, &os, &O)) return nullptr;
    } else if (a[7] != Py_None) {
        return bad("Q_out without Q"), nullptr;
    }
    const float* rot = nullptr;
    int64_t rot_len = 0, rot_dim = 0;
    if (a[8] != Py_None) {
        const at::Tensor* r;
        if (!tensor(a[8], &r)) return nullptr;
        if (r->dim() != 2 || r->scalar_type() != at::kFloat || r->get_device() != c->device || !r->is_contiguous() ||
            r->size(1) > INT32_MAX)
            return bad("rot must be a contiguous fp32 tensor [rot_len, rot_dim] on the cache's device"), nullptr;
        rot = static_cast<const float*>(r->data_ptr());
        rot_len = r->size(0);
        rot_dim = r->size(1);
    }
    const long kind = PyLong_AsLong(a[9]);
    if (PyErr_Occurred() || !stream_of(c, a[10], &st)) return nullptr;
    return PyLong_FromLong(g_append(c->handle, b.B, T, b.q_off, b.kv_lens, b.table, b.max_pages, K, ks, V, vs, Q, qs,
                                    H < 0 ? 1 : int32_t(H), O, os, rot, int32_t(rot_dim), rot_len, int32_t(kind), st));
}

// fwd(info, Q, q_offsets, kv_lens, page_table, bias, scale, causal, window, max_q_len, O, lse,
//     workspace, stream)
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 14) return PyErr_Format(PyExc_TypeError, "14 arguments");
    const Info* c = info_of(a[0]);
    Batch b;
    if (!c || !g_fwd || !batch(c, a[2], a[3], a[4], &b)) return nullptr;
    int64_t T = -1, H = -1, qs;
    void *Q, *st;
    if (!rows(c, a[1], &H, &T, &qs, &Q)) return nullptr;
    const at::Tensor *O, *lse, *ws;
    if (!tensor(a[10], &O) || !tensor(a[11], &lse) || !tensor(a[12], &ws)) return nullptr;
    if (O->dim() != 3 || O->size(0) != T || O->size(1) != H || O->size(2) != c->D || !O->is_contiguous() ||
        O->get_device() != c->device)
        return bad("O must be a contiguous tensor of Q's shape"), nullptr;
    int32_t od = -1;
    if (O->scalar_type() == at::kBFloat16) od = JFA_BF16;
    if (O->scalar_type() == at::kFloat) od = JFA_F32;
    if (od < 0) return PyLong_FromLong(JFA_ERR_UNSUPPORTED);
    if (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != T || lse->size(1) != H ||
        !lse->is_contiguous() || lse->get_device() != c->device)
        return bad("lse must be a contiguous fp32 tensor [T, H]"), nullptr;
    if (ws->get_device() != c->device || !ws->is_contiguous())
        return bad("workspace must be a contiguous tensor on the cache's device"), nullptr;
    const float* bias = nullptr;
    if (a[5] != Py_None) {
        const at::Tensor* t;
        if (!tensor(a[5], &t)) return nullptr;
        if (t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(0) != H || t->size(1) != 32 || !t->is_contiguous() ||
            t->get_device() != c->device)
            return bad("bias must be a contiguous fp32 tensor [H, 32]"), nullptr;
        bias = static_cast<const float*>(t->data_ptr());
    }
    const double scale = PyFloat_AsDouble(a[6]);
    const int causal = PyObject_IsTrue(a[7]);
    const long window = a[8] == Py_None ? -1 : PyLong_AsLong(a[8]), max_q = a[9] == Py_None ? 0 : PyLong_AsLong(a[9]);
    if (PyErr_Occurred() || !stream_of(c, a[13], &st)) return nullptr;
    auto i32 = [](long v) { return int32_t(v < INT32_MIN ? INT32_MIN : v > INT32_MAX ? INT32_MAX : v); };
    return PyLong_FromLong(g_fwd(c->handle, b.B, T, i32(max_q), b.q_off, b.kv_lens, b.table, b.max_pages, Q, qs, int32_t(H),
                                 causal, i32(window), bias ? JFA_BIAS_RELPOS32 : JFA_BIAS_NONE, bias, float(scale),
                                 O->data_ptr(), od, static_cast<float*>(lse->data_ptr()), ws->data_ptr(), ws->nbytes(), st));
}

// No C++ exception leaves a call: a tensor without storage, or a stream asked for without a
// device, raises RuntimeError.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<set_calls>("set_calls"), method<describe>("describe"), method<append>("append"),
                         method<fwd>("fwd"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_calls() { return PyModule_Create(&module); }
