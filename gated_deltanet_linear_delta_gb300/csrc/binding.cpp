// binding.cpp -- the paged cache calls of gdn.h for torch tensors, as a CPython module.
//
// A decode step's call on the GPU is shorter than reading twenty tensor attributes in Python and
// converting twenty-six arguments (about 12 us of host time for gdn_paged_attn), so these three calls
// check their tensors and marshal their arguments here; __init__.py declares them. Each returns the C
// call's status; tensors that do not fit together raise TypeError or ValueError, and what torch throws
// while they are read (C++ exceptions must not reach the interpreter) becomes a RuntimeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <exception>

#include <torch/csrc/autograd/python_variable.h>

#include "gdn.h"

namespace {

using at::Tensor;

struct Call {
    int B, T, H, Hkv, d, pages, page, width, dtype, cache_dtype;
    void *k_cache, *v_cache;
    float *k_scale = nullptr, *v_scale = nullptr;
    const int32_t *table, *lens, *cu = nullptr;
};

bool refuse(PyObject *kind, const char *why) {
    PyErr_SetString(kind, why);
    return false;
}

// A tensor argument, or null for None where that is allowed; false with an exception set otherwise.
bool tensor(PyObject *o, const Tensor *&t, bool optional = false) {
    t = nullptr;
    if (o == Py_None && optional) return true;
    if (!THPVariable_Check(o)) return refuse(PyExc_TypeError, "expected a torch tensor");
    t = &THPVariable_Unpack(o);
    // (sparse and nested tensors have no strides to ask for)
    if (t->layout() != at::kStrided || t->is_nested()) return refuse(PyExc_TypeError, "expected a dense tensor");
    return true;
}

bool integer(PyObject *o, long long missing, long long &v) {
    if (o == Py_None) {
        v = missing;
        return true;
    }
    v = PyLong_AsLongLong(o);
    return !(v == -1 && PyErr_Occurred());
}

int dtype_code(at::ScalarType t, bool cache) {
    if (t == at::kBFloat16) return GDN_BF16;
    if (t == at::kFloat) return GDN_F32;
    if (cache && t == at::kFloat8_e4m3fn) return GDN_FP8;
    if (cache && t == at::kChar) return GDN_INT8;
    return -1;
}

// Elements from a token's rows to the next token's; -1 unless heads and elements are contiguous.
int64_t token_stride(const Tensor &t) {
    const auto s = t.sizes(), st = t.strides();
    if ((s[2] > 1 && st[2] != 1) || (s[1] > 1 && st[1] != s[2])) return -1;
    return s[0] > 1 ? st[0] : s[1] * s[2];
}

// What the three calls share. `rows` and `rows2` are the packed rows: k and v, or q and out.
bool kv_call(const Tensor &rows, const Tensor &rows2, PyObject *const *a, Call &c) {
    // a: k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, B, T
    const Tensor *kc, *vc, *ks, *vs, *table, *lens, *cu;
    if (!tensor(a[0], kc) || !tensor(a[1], vc) || !tensor(a[2], ks, true) || !tensor(a[3], vs, true) ||
        !tensor(a[4], table) || !tensor(a[5], lens) || !tensor(a[6], cu, true))
        return false;
    if (rows.dim() != 3 || rows2.dim() != 3 || token_stride(rows) < 0 || token_stride(rows2) < 0)
        return refuse(PyExc_ValueError,
                      "packed rows must be tensors [tokens, heads, d] with contiguous heads and elements");
    c.dtype = dtype_code(rows.scalar_type(), false);
    if (c.dtype < 0) return refuse(PyExc_TypeError, "unsupported dtype: use bfloat16 or float32");
    if (rows2.sizes() != rows.sizes() || rows2.scalar_type() != rows.scalar_type())
        return refuse(PyExc_ValueError, "the call's packed rows (k and v, or q and out) must share one shape and dtype");
    if (kc->dim() != 4 || vc->sizes() != kc->sizes() || vc->scalar_type() != kc->scalar_type())
        return refuse(PyExc_ValueError,
                      "k_cache and v_cache must share one dtype and the shape [num_pages, Hkv, page_size, d]");
    if (rows.size(2) != kc->size(3))
        return refuse(PyExc_ValueError, "the rows' last dimension is not the cache's head dimension");
    c.cache_dtype = dtype_code(kc->scalar_type(), true);
    if (c.cache_dtype < 0)
        return refuse(PyExc_TypeError, "unsupported cache dtype: use the rows' dtype, float8_e4m3fn or int8");
    if (c.cache_dtype >= GDN_FP8)
        for (const Tensor *s : {ks, vs})
            if (!s || s->scalar_type() != at::kFloat || s->sizes() != kc->sizes().slice(0, 3))
                return refuse(PyExc_TypeError,
                              "an 8-bit cache needs fp32 k_scale and v_scale [num_pages, Hkv, page_size]");
    if (table->scalar_type() != at::kInt || lens->scalar_type() != at::kInt || (cu && cu->scalar_type() != at::kInt))
        return refuse(PyExc_TypeError, "block_table, kv_lens and cu_seqlens must be int32");
    if (lens->dim() != 1 || table->dim() != 2 || (cu && (cu->dim() != 1 || cu->numel() < 1)))
        return refuse(PyExc_ValueError, "kv_lens must be [B], block_table [B, max_pages] and cu_seqlens [B + 1]");
    const long long tokens = rows.size(0);
    long long B, T;
    if (cu) {
        B = cu->numel() - 1;
        T = tokens;
    } else {
        if (!integer(a[7], lens->numel(), B)) return false;
        if (!integer(a[8], B > 0 ? tokens / B : 0, T)) return false;
        if (B < 0 || T < 0 || B * T != tokens)
            return refuse(PyExc_ValueError, "the packed rows are not B sequences of T tokens");
    }
    if (lens->numel() != B || table->size(0) != B)
        return refuse(PyExc_ValueError, "kv_lens must be [B], block_table [B, max_pages] and cu_seqlens [B + 1]");
    const int device = rows.is_cuda() ? (int)rows.get_device() : -1;
    for (const Tensor *t : {&rows, &rows2, kc, vc, ks, vs, table, lens, cu})
        if (t && (!t->is_cuda() || (int)t->get_device() != device))
            return refuse(PyExc_ValueError, "tensors must be CUDA tensors of one device");
    for (const Tensor *t : {kc, vc, ks, vs, table, lens, cu})
        if (t && !t->is_contiguous())
            return refuse(PyExc_ValueError, "caches, scales, block_table, kv_lens and cu_seqlens must be contiguous");
    for (int64_t v : {(int64_t)B, (int64_t)T, rows.size(1), kc->size(0), kc->size(1), kc->size(2), kc->size(3), table->size(1)})
        if (v > INT32_MAX) return refuse(PyExc_ValueError, "a size is beyond 2^31 - 1");
    c.B = (int)B;
    c.T = (int)T;
    c.H = (int)rows.size(1);
    c.pages = (int)kc->size(0);
    c.Hkv = (int)kc->size(1);
    c.page = (int)kc->size(2);
    c.d = (int)kc->size(3);
    c.width = (int)table->size(1);
    c.k_cache = kc->data_ptr();
    c.v_cache = vc->data_ptr();
    if (c.cache_dtype >= GDN_FP8) {
        c.k_scale = static_cast<float *>(ks->data_ptr());
        c.v_scale = static_cast<float *>(vs->data_ptr());
    }
    c.table = static_cast<const int32_t *>(table->data_ptr());
    c.lens = static_cast<const int32_t *>(lens->data_ptr());
    if (cu) c.cu = static_cast<const int32_t *>(cu->data_ptr());
    return true;
}

bool arguments(Py_ssize_t got, Py_ssize_t want) {
    return got == want || refuse(PyExc_TypeError, "wrong number of arguments");
}

// A call as the interpreter makes it, with what it throws as a Python exception. (It may throw only with the
// interpreter's lock held.)
template <PyObject *(*CALL)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        return CALL(a, n);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// (k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, B, T, stream)
template <bool WRITE>
PyObject *kv_copy(PyObject *const *a, Py_ssize_t n) {
    const Tensor *k, *v;
    Call c;
    if (!arguments(n, 12) || !tensor(a[0], k) || !tensor(a[1], v) || !kv_call(*k, *v, a + 2, c)) return nullptr;
    if (c.H != c.Hkv) {
        refuse(PyExc_ValueError, "k and v must have the caches' heads");
        return nullptr;
    }
    void *stream = PyLong_AsVoidPtr(a[11]);
    if (PyErr_Occurred()) return nullptr;
    void *kp = k->data_ptr(), *vp = v->data_ptr();
    const int64_t ks = token_stride(*k), vs = token_stride(*v);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    if (WRITE)
        rc = gdn_kv_write(kp, vp, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.lens, c.cu, c.B, c.T, c.Hkv, c.d,
                          c.pages, c.page, c.width, ks, vs, c.dtype, c.cache_dtype, stream);
    else
        rc = gdn_kv_read(c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.lens, c.cu, kp, vp, c.B, c.T, c.Hkv, c.d,
                         c.pages, c.page, c.width, ks, vs, c.dtype, c.cache_dtype, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// (q, out, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, B, T, scale, workspace, stream)
PyObject *paged_attn(PyObject *const *a, Py_ssize_t n) {
    const Tensor *q, *out, *ws;
    Call c;
    if (!arguments(n, 14) || !tensor(a[0], q) || !tensor(a[1], out) || !kv_call(*q, *out, a + 2, c) || !tensor(a[12], ws))
        return nullptr;
    if (!out->is_contiguous() || !ws->is_contiguous() || !ws->is_cuda() || ws->get_device() != q->get_device()) {
        refuse(PyExc_ValueError, "out and workspace must be contiguous CUDA tensors of q's device");
        return nullptr;
    }
    const double scale = a[11] == Py_None ? 1.0 / std::sqrt((double)c.d) : PyFloat_AsDouble(a[11]);
    void *stream = PyLong_AsVoidPtr(a[13]);
    if (PyErr_Occurred()) return nullptr;
    void *qp = q->data_ptr(), *op = out->data_ptr(), *wp = ws->data_ptr();
    const int64_t stride = token_stride(*q);
    const size_t bytes = ws->nbytes();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = gdn_paged_attn(qp, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.lens, c.cu, op, c.B, c.T, c.H, c.Hkv, c.d,
                        c.pages, c.page, c.width, stride, (float)scale, c.dtype, c.cache_dtype, wp, bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

PyMethodDef methods[] = {
    {"kv_write", (PyCFunction)(void (*)(void))entry<kv_copy<true>>, METH_FASTCALL, "gdn_kv_write"},
    {"kv_read", (PyCFunction)(void (*)(void))entry<kv_copy<false>>, METH_FASTCALL, "gdn_kv_read"},
    {"paged_attn", (PyCFunction)(void (*)(void))entry<paged_attn>, METH_FASTCALL, "gdn_paged_attn"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "The paged cache calls for torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
