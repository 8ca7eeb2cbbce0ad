// binding.cpp -- the paged cache calls and the calls on trees of gdn.h for torch tensors, as a CPython module.
//
// A decode step's call on the GPU is shorter than reading twenty tensor attributes in Python and
// converting twenty-six arguments (about 12 us of host time for gdn_paged_attn), so these calls
// check their tensors and marshal their arguments here; __init__.py declares them. Each returns the C
// call's status; tensors that do not fit together raise TypeError or ValueError, and what torch throws
// while they are read (C++ exceptions must not reach the interpreter) becomes a RuntimeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <cstdio>
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

// What the calls on paged caches share. `rows` and `rows2` are the packed rows: k and v, or q and out. gdn_kv_keep,
// which has none, passes null.
bool kv_call(const Tensor *rows_, const Tensor *rows2_, PyObject *const *a, Call &c) {
    // a: k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, B, T
    const Tensor *kc, *vc, *ks, *vs, *table, *lens, *cu;
    if (!tensor(a[0], kc) || !tensor(a[1], vc) || !tensor(a[2], ks, true) || !tensor(a[3], vs, true) ||
        !tensor(a[4], table) || !tensor(a[5], lens) || !tensor(a[6], cu, true))
        return false;
    if (rows_) {
        const Tensor &rows = *rows_, &rows2 = *rows2_;
        if (rows.dim() != 3 || rows2.dim() != 3 || token_stride(rows) < 0 || token_stride(rows2) < 0)
            return refuse(PyExc_ValueError,
                          "packed rows must be tensors [tokens, heads, d] with contiguous heads and elements");
        c.dtype = dtype_code(rows.scalar_type(), false);
        if (c.dtype < 0) return refuse(PyExc_TypeError, "unsupported dtype: use bfloat16 or float32");
        if (rows2.sizes() != rows.sizes() || rows2.scalar_type() != rows.scalar_type())
            return refuse(PyExc_ValueError, "the call's packed rows (k and v, or q and out) must share one shape and dtype");
    }
    if (kc->dim() != 4 || vc->sizes() != kc->sizes() || vc->scalar_type() != kc->scalar_type())
        return refuse(PyExc_ValueError,
                      "k_cache and v_cache must share one dtype and the shape [num_pages, Hkv, page_size, d]");
    if (rows_ && rows_->size(2) != kc->size(3))
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
    long long B, T;
    if (!rows_) {
        B = lens->numel();
        if (!integer(a[8], cu ? 0 : -1, T)) return false;
        if (T < 0) return refuse(PyExc_ValueError, "T, the nodes of each sequence, must be given where cu_seqlens is not");
        if (cu && cu->numel() - 1 != B) return refuse(PyExc_ValueError, "cu_seqlens must be [B + 1]");
    } else if (cu) {
        B = cu->numel() - 1;
        T = rows_->size(0);
    } else {
        const long long tokens = rows_->size(0);
        if (!integer(a[7], lens->numel(), B)) return false;
        if (!integer(a[8], B > 0 ? tokens / B : 0, T)) return false;
        if (B < 0 || T < 0 || B * T != tokens)
            return refuse(PyExc_ValueError, "the packed rows are not B sequences of T tokens");
    }
    if (lens->numel() != B || table->size(0) != B)
        return refuse(PyExc_ValueError, "kv_lens must be [B], block_table [B, max_pages] and cu_seqlens [B + 1]");
    const int device = kc->is_cuda() ? (int)kc->get_device() : -1;
    for (const Tensor *t : {rows_, rows2_, kc, vc, ks, vs, table, lens, cu})
        if (t && (!t->is_cuda() || (int)t->get_device() != device))
            return refuse(PyExc_ValueError, "tensors must be CUDA tensors of one device");
    for (const Tensor *t : {kc, vc, ks, vs, table, lens, cu})
        if (t && !t->is_contiguous())
            return refuse(PyExc_ValueError, "caches, scales, block_table, kv_lens and cu_seqlens must be contiguous");
    for (int64_t v : {(int64_t)B, (int64_t)T, rows_ ? rows_->size(1) : 0, kc->size(0), kc->size(1), kc->size(2), kc->size(3),
                      table->size(1)})
        if (v > INT32_MAX) return refuse(PyExc_ValueError, "a size is beyond 2^31 - 1");
    c.B = (int)B;
    c.T = (int)T;
    c.H = rows_ ? (int)rows_->size(1) : 0;
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

// A contiguous tensor of a type, a number of dimensions and a device (the others of the call's).
bool plain(const Tensor &t, at::ScalarType type, int dims, const Tensor &like, const char *name) {
    char why[160];
    if (t.scalar_type() != type) {
        std::snprintf(why, sizeof why, "%s has the wrong dtype", name);
        return refuse(PyExc_TypeError, why);
    }
    if (t.dim() != dims || !t.is_contiguous()) {
        std::snprintf(why, sizeof why, "%s must be a contiguous tensor of %d dimensions", name, dims);
        return refuse(PyExc_ValueError, why);
    }
    if (!t.is_cuda() || t.get_device() != like.get_device()) return refuse(PyExc_ValueError, "tensors must be CUDA tensors of one device");
    return true;
}
int32_t *ints(const Tensor *t) { return t ? static_cast<int32_t *>(t->data_ptr()) : nullptr; }

// The sequences of a call on trees: `tokens` packed ones as cu_seqlens says, or B times T.
bool sequences(const Tensor *cu, PyObject *B_, PyObject *T_, long long tokens, long long B_default, const Tensor &like, long long &B,
               long long &T) {
    if (cu) {
        if (!plain(*cu, at::kInt, 1, like, "cu_seqlens")) return false;
        if (cu->numel() < 1) return refuse(PyExc_ValueError, "cu_seqlens must be [B + 1]");
        B = cu->numel() - 1;
        T = tokens;
    } else {
        if (!integer(B_, B_default, B)) return false;
        if (!integer(T_, B > 0 ? tokens / B : 0, T)) return false;
        if (B < 0 || T < 0 || (B > 0 && T > tokens) || B * T != tokens)
            return refuse(PyExc_ValueError, "the packed tokens are not B sequences of T nodes");
    }
    if (B > INT32_MAX || T > INT32_MAX) return refuse(PyExc_ValueError, "a size is beyond 2^31 - 1");
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
    if (!arguments(n, 12) || !tensor(a[0], k) || !tensor(a[1], v) || !kv_call(k, v, a + 2, c)) return nullptr;
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

// (q, out, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, B, T, scale, workspace, stream), and with
// TREE parents
template <bool TREE>
PyObject *paged_attn(PyObject *const *a, Py_ssize_t n) {
    const Tensor *q, *out, *ws, *parents = nullptr;
    Call c;
    if (!arguments(n, TREE ? 15 : 14) || !tensor(a[0], q) || !tensor(a[1], out) || !kv_call(q, out, a + 2, c) || !tensor(a[12], ws))
        return nullptr;
    if (!out->is_contiguous() || !ws->is_contiguous() || !ws->is_cuda() || ws->get_device() != q->get_device()) {
        refuse(PyExc_ValueError, "out and workspace must be contiguous CUDA tensors of q's device");
        return nullptr;
    }
    if (TREE) {
        if (!tensor(a[14], parents) || !plain(*parents, at::kInt, 1, *q, "parents")) return nullptr;
        if (parents->numel() != q->size(0)) {
            refuse(PyExc_ValueError, "parents must be [tokens]");
            return nullptr;
        }
    }
    const double scale = a[11] == Py_None ? 1.0 / std::sqrt((double)c.d) : PyFloat_AsDouble(a[11]);
    void *stream = PyLong_AsVoidPtr(a[13]);
    if (PyErr_Occurred()) return nullptr;
    void *qp = q->data_ptr(), *op = out->data_ptr(), *wp = ws->data_ptr();
    const int32_t *pp = ints(parents);
    const int64_t stride = token_stride(*q);
    const size_t bytes = ws->nbytes();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    if (TREE)
        rc = gdn_tree_attn(qp, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.lens, c.cu, pp, op, c.B, c.T, c.H, c.Hkv,
                           c.d, c.pages, c.page, c.width, stride, (float)scale, c.dtype, c.cache_dtype, wp, bytes, stream);
    else
        rc = gdn_paged_attn(qp, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.lens, c.cu, op, c.B, c.T, c.H, c.Hkv, c.d,
                            c.pages, c.page, c.width, stride, (float)scale, c.dtype, c.cache_dtype, wp, bytes, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// Accepted paths [B, path_stride] and counts [B]
bool accepted(PyObject *path_, PyObject *counts_, long long B, const Tensor &like, const Tensor *&path, const Tensor *&counts) {
    if (!tensor(path_, path) || !tensor(counts_, counts) || !plain(*path, at::kInt, 2, like, "path") ||
        !plain(*counts, at::kInt, 1, like, "counts"))
        return false;
    if (path->size(0) != B || counts->numel() != B || path->size(1) > INT32_MAX)
        return refuse(PyExc_ValueError, "path must be [B, nodes] and counts [B]");
    return true;
}

// (k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, None, T, path, counts, stream)
PyObject *kv_keep(PyObject *const *a, Py_ssize_t n) {
    const Tensor *path, *counts, *like;
    Call c;
    if (!arguments(n, 12) || !kv_call(nullptr, nullptr, a, c) || !tensor(a[0], like) ||
        !accepted(a[9], a[10], c.B, *like, path, counts))
        return nullptr;
    void *stream = PyLong_AsVoidPtr(a[11]);
    if (PyErr_Occurred()) return nullptr;
    const int32_t *pp = ints(path), *cp = ints(counts);
    const int stride = (int)path->size(1);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = gdn_kv_keep(c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.lens, c.cu, pp, cp, c.B, c.T, stride, c.Hkv, c.d,
                     c.pages, c.page, c.width, c.cache_dtype, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// A layer's packed inputs on trees: k [tokens, Hk, dk] (and q), v [tokens, Hv, dv] (and out), g and b [tokens, Hv]
struct Layer {
    long long B, T;
    int Hk, Hv, dk, dv, dtype, num_slots = 0;
    const Tensor *cu, *slots;
};
bool layer_call(const Tensor &k, const Tensor *q, const Tensor &v, const Tensor *out, const Tensor &g, const Tensor &b,
                const Tensor &state, const Tensor *state2, PyObject *slots, PyObject *cu, PyObject *B, PyObject *T, Layer &l) {
    l.dtype = dtype_code(k.scalar_type(), false);
    if (l.dtype < 0) return refuse(PyExc_TypeError, "unsupported dtype: use bfloat16 or float32");
    const at::ScalarType type = k.scalar_type();
    if (!plain(k, type, 3, k, "k") || !plain(v, type, 3, k, "v") || !plain(g, type, 2, k, "g") || !plain(b, type, 2, k, "b") ||
        (q && !plain(*q, type, 3, k, "q")) || (out && !plain(*out, type, 3, k, "out")) ||
        !plain(state, at::kFloat, 4, k, "the state") || (state2 && !plain(*state2, at::kFloat, 4, k, "state_out")))
        return false;
    if (!tensor(slots, l.slots, true) || !tensor(cu, l.cu, true)) return false;
    if (l.slots && !plain(*l.slots, at::kInt, 1, k, "slots")) return false;
    const int64_t tokens = k.size(0), Hv = v.size(1);
    if ((q && q->sizes() != k.sizes()) || v.size(0) != tokens || (out && out->sizes() != v.sizes()) || g.size(0) != tokens ||
        g.size(1) != Hv || b.sizes() != g.sizes())
        return refuse(PyExc_ValueError, "the packed inputs must be q, k [tokens, Hk, dk], v, out [tokens, Hv, dv], g, b [tokens, Hv]");
    if (state.size(1) != Hv || state.size(2) != v.size(2) || state.size(3) != k.size(2) || (state2 && state2->sizes() != state.sizes()))
        return refuse(PyExc_ValueError, "states must be [B or num_slots, Hv, dv, dk]");
    if (!sequences(l.cu, B, T, tokens, l.slots ? l.slots->numel() : state.size(0), k, l.B, l.T)) return false;
    if ((l.slots ? l.slots->numel() : state.size(0)) != l.B)
        return refuse(PyExc_ValueError, l.slots ? "slots must be [B]" : "states must be [B, Hv, dv, dk]");
    for (int64_t x : {state.size(0), k.size(1), Hv, k.size(2), v.size(2)})
        if (x > INT32_MAX) return refuse(PyExc_ValueError, "a size is beyond 2^31 - 1");
    l.Hk = (int)k.size(1);
    l.Hv = (int)Hv;
    l.dk = (int)k.size(2);
    l.dv = (int)v.size(2);
    if (l.slots) l.num_slots = (int)state.size(0);
    return true;
}

// (q, k, v, g, b, state, slots, parents, cu_seqlens, out, B, T, stream)
PyObject *tree_scan(PyObject *const *a, Py_ssize_t n) {
    const Tensor *q, *k, *v, *g, *b, *state, *parents, *out;
    Layer l;
    if (!arguments(n, 13) || !tensor(a[0], q) || !tensor(a[1], k) || !tensor(a[2], v) || !tensor(a[3], g) || !tensor(a[4], b) ||
        !tensor(a[5], state) || !tensor(a[7], parents) || !tensor(a[9], out) ||
        !layer_call(*k, q, *v, out, *g, *b, *state, nullptr, a[6], a[8], a[10], a[11], l) ||
        !plain(*parents, at::kInt, 1, *k, "parents"))
        return nullptr;
    if (parents->numel() != k->size(0)) {
        refuse(PyExc_ValueError, "parents must be [tokens]");
        return nullptr;
    }
    void *stream = PyLong_AsVoidPtr(a[12]);
    if (PyErr_Occurred()) return nullptr;
    const void *qp = q->data_ptr(), *kp = k->data_ptr(), *vp = v->data_ptr(), *gp = g->data_ptr(), *bp = b->data_ptr();
    const float *sp = static_cast<const float *>(state->data_ptr());
    const int32_t *slots = ints(l.slots), *pp = ints(parents), *cu = ints(l.cu);
    void *op = out->data_ptr();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = gdn_tree_scan(qp, kp, vp, gp, bp, sp, slots, pp, cu, op, (int)l.B, (int)l.T, l.num_slots, l.Hk, l.Hv, l.dk, l.dv, l.dtype,
                       stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// (k, v, g, b, state_in, state_out, slots, path, counts, cu_seqlens, B, T, stream)
PyObject *tree_advance(PyObject *const *a, Py_ssize_t n) {
    const Tensor *k, *v, *g, *b, *in, *out, *path, *counts;
    Layer l;
    if (!arguments(n, 13) || !tensor(a[0], k) || !tensor(a[1], v) || !tensor(a[2], g) || !tensor(a[3], b) || !tensor(a[4], in) ||
        !tensor(a[5], out) || !layer_call(*k, nullptr, *v, nullptr, *g, *b, *in, out, a[6], a[9], a[10], a[11], l) ||
        !accepted(a[7], a[8], l.B, *k, path, counts))
        return nullptr;
    void *stream = PyLong_AsVoidPtr(a[12]);
    if (PyErr_Occurred()) return nullptr;
    const void *kp = k->data_ptr(), *vp = v->data_ptr(), *gp = g->data_ptr(), *bp = b->data_ptr();
    const float *ip = static_cast<const float *>(in->data_ptr());
    float *op = static_cast<float *>(out->data_ptr());
    const int32_t *slots = ints(l.slots), *pp = ints(path), *cp = ints(counts), *cu = ints(l.cu);
    const int stride = (int)path->size(1);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = gdn_tree_advance(kp, vp, gp, bp, ip, op, slots, pp, cp, cu, (int)l.B, (int)l.T, stride, l.num_slots, l.Hk, l.Hv, l.dk,
                          l.dv, l.dtype, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// Elements from a row of probabilities to the next; -1 unless a row's are contiguous
int64_t row_stride(const Tensor &t) {
    const int64_t V = t.size(1);
    if (V > 1 && t.stride(1) != 1) return -1;
    return t.size(0) > 1 ? t.stride(0) : V;
}

// (target_probs, draft_probs, tokens, parents, r, r_last, cu_seqlens, path, counts, next, B, T, stream)
PyObject *tree_verify(PyObject *const *a, Py_ssize_t n) {
    const Tensor *target, *draft, *tokens, *parents, *r, *last, *cu, *path, *counts, *next;
    if (!arguments(n, 13) || !tensor(a[0], target) || !tensor(a[1], draft, true) || !tensor(a[2], tokens) || !tensor(a[3], parents) ||
        !tensor(a[4], r) || !tensor(a[5], last) || !tensor(a[6], cu, true))
        return nullptr;
    for (const Tensor *t : {target, draft})
        if (t) {
            if (t->scalar_type() != at::kFloat) {
                refuse(PyExc_TypeError, "probabilities must be float32");
                return nullptr;
            }
            if (t->dim() != 2 || row_stride(*t) < 0 || t->sizes() != target->sizes() || !t->is_cuda() ||
                t->get_device() != target->get_device()) {
                refuse(PyExc_ValueError, "probabilities must be CUDA tensors [tokens, V] of one device with contiguous rows");
                return nullptr;
            }
        }
    const int64_t all = target->size(0);
    long long B, T;
    if (!plain(*tokens, at::kInt, 1, *target, "tokens") || !plain(*parents, at::kInt, 1, *target, "parents") ||
        !plain(*r, at::kFloat, 1, *target, "r") || !plain(*last, at::kFloat, 1, *target, "r_last") ||
        !sequences(cu, a[10], a[11], all, last->numel(), *target, B, T) || !accepted(a[7], a[8], B, *target, path, counts) ||
        !tensor(a[9], next) || !plain(*next, at::kInt, 1, *target, "next"))
        return nullptr;
    if (tokens->numel() != all || parents->numel() != all || r->numel() != all || last->numel() != B || next->numel() != B) {
        refuse(PyExc_ValueError, "tokens, parents and r must be [tokens], r_last and next [B]");
        return nullptr;
    }
    if (target->size(1) > INT32_MAX) {
        refuse(PyExc_ValueError, "a size is beyond 2^31 - 1");
        return nullptr;
    }
    void *stream = PyLong_AsVoidPtr(a[12]);
    if (PyErr_Occurred()) return nullptr;
    const float *tp = static_cast<const float *>(target->data_ptr()), *dp = draft ? static_cast<const float *>(draft->data_ptr()) : nullptr;
    const float *rp = static_cast<const float *>(r->data_ptr()), *lp = static_cast<const float *>(last->data_ptr());
    const int32_t *xp = ints(tokens), *up = ints(parents), *cp = ints(cu);
    int32_t *pp = ints(path), *np = ints(counts), *op = ints(next);
    const int64_t ts = row_stride(*target), ds = draft ? row_stride(*draft) : 0;
    const int V = (int)target->size(1), stride = (int)path->size(1);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = gdn_tree_verify(tp, dp, xp, up, rp, lp, cp, pp, np, op, (int)B, (int)T, V, ts, ds, stride, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

PyMethodDef methods[] = {
    {"kv_write", (PyCFunction)(void (*)(void))entry<kv_copy<true>>, METH_FASTCALL, "gdn_kv_write"},
    {"kv_read", (PyCFunction)(void (*)(void))entry<kv_copy<false>>, METH_FASTCALL, "gdn_kv_read"},
    {"paged_attn", (PyCFunction)(void (*)(void))entry<paged_attn<false>>, METH_FASTCALL, "gdn_paged_attn"},
    {"tree_attn", (PyCFunction)(void (*)(void))entry<paged_attn<true>>, METH_FASTCALL, "gdn_tree_attn"},
    {"kv_keep", (PyCFunction)(void (*)(void))entry<kv_keep>, METH_FASTCALL, "gdn_kv_keep"},
    {"tree_scan", (PyCFunction)(void (*)(void))entry<tree_scan>, METH_FASTCALL, "gdn_tree_scan"},
    {"tree_advance", (PyCFunction)(void (*)(void))entry<tree_advance>, METH_FASTCALL, "gdn_tree_advance"},
    {"tree_verify", (PyCFunction)(void (*)(void))entry<tree_verify>, METH_FASTCALL, "gdn_tree_verify"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "The paged cache calls and the calls on trees for torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
