// The per-step calls (kv_append, attention_paged, attention_window, rope_axes, and
// those of a short training step: attention_backward, checkpoint_store) from Python
// tensors to the C ABI without the interpreter in between. A decode step makes
// two such calls a layer, each of a few microseconds on the GPU: the checks of
// a call cost 3 us in Python and its conversion by ctypes 2 us, 0.5 us here.
//
// Each function takes the arguments that the wrappers of attn.py would pass on,
// on the current device and stream. It returns None, having done nothing, for
// whatever is not plainly right (other types, shapes or devices, tensor
// subclasses): the wrappers then go through their own checks, which say what is
// wrong or handle the case. An int is the C ABI's status.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "../../include/attn.h"

namespace {

using at::Tensor;

// A plain tensor's value, or null (None and anything else).
const Tensor* plain(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// True for a contiguous tensor of this type on CUDA device `at`.
bool good(const Tensor* t, c10::ScalarType type, int at) {
    return t && t->defined() && t->is_cuda() && t->device().index() == at && t->scalar_type() == type && t->is_contiguous();
}

// Elements from token to token of a (B, S, H, D) tensor, or -1 where the tokens
// are not evenly spaced and contiguous inside.
long long token_stride(const Tensor& t) {
    const auto n = t.sizes();
    const auto s = t.strides();
    if (t.is_contiguous()) return (long long)n[2] * n[3];
    if ((n[3] > 1 && s[3] != 1) || (n[2] > 1 && s[2] != n[3])) return -1;
    if (n[1] == 1) return n[0] > 1 ? s[0] : std::max<long long>(s[1], n[2] * n[3]);
    if (n[0] > 1 && s[0] != n[1] * s[1]) return -1;
    return s[1];
}

// What the cache's calls share, checked against x (B, S, H, D) on the current
// device. Sizes are bounded to C ints.
struct Cache {
    int at = -1, kind = ATTN_CACHE_16BIT;
    int B = 0, S = 0, H = 0, Hkv = 0, D = 0, page = 0, max_pages = 0, n_pages = 0, max_pos = 0;
    const void *k = nullptr, *v = nullptr;
    float *ks = nullptr, *vs = nullptr;
    const int *table = nullptr, *kv_lens = nullptr, *lens = nullptr;
    const float* rope = nullptr;
    cudaStream_t stream = nullptr;
};

bool fits(at::IntArrayRef n) {
    for (const int64_t e : n)
        if (e > INT_MAX) return false;
    return true;
}

bool begin(const Tensor* x, int* at, cudaStream_t* stream) {
    if (!x || !x->defined() || !x->is_cuda() || x->dim() != 4 || !fits(x->sizes())) return false;
    if (x->scalar_type() != at::kBFloat16 && x->scalar_type() != at::kHalf) return false;
    *at = x->device().index();
    if (*at != c10::cuda::current_device()) return false;
    *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)*at).stream();
    return true;
}

bool open_cache(const Tensor* x, PyObject* k_cache, PyObject* v_cache, PyObject* block_table, PyObject* kv_lens,
                PyObject* lens, PyObject* k_scale, PyObject* v_scale, PyObject* table, Cache* c) {
    if (!begin(x, &c->at, &c->stream)) return false;
    const auto xs = x->sizes();
    c->B = (int)xs[0], c->S = (int)xs[1], c->H = (int)xs[2];
    const Tensor *k = plain(k_cache), *v = plain(v_cache), *bt = plain(block_table), *kl = plain(kv_lens);
    if (!k || !k->defined() || k->dim() != 4) return false;
    const c10::ScalarType type = k->scalar_type();
    if (!good(k, type, c->at) || !good(v, type, c->at) || v->sizes() != k->sizes() || !fits(k->sizes())) return false;
    c->n_pages = (int)k->size(0), c->Hkv = (int)k->size(1), c->page = (int)k->size(2), c->D = (int)k->size(3);
    if (xs[3] != c->D) return false;
    c->k = k->data_ptr();
    c->v = v->data_ptr();
    if (!good(bt, at::kInt, c->at) || bt->dim() != 2 || bt->size(0) != c->B || bt->size(1) > INT_MAX) return false;
    if (!good(kl, at::kInt, c->at) || kl->dim() != 1 || kl->size(0) != c->B) return false;
    c->max_pages = (int)bt->size(1);
    c->table = static_cast<const int*>(bt->data_ptr());
    c->kv_lens = static_cast<const int*>(kl->data_ptr());
    if (lens != Py_None) {
        const Tensor* l = plain(lens);
        if (!good(l, at::kInt, c->at) || l->dim() != 1 || l->size(0) != c->B) return false;
        c->lens = static_cast<const int*>(l->data_ptr());
    }
    if (type == at::kFloat8_e4m3fn) {
        c->kind = ATTN_CACHE_E4M3;
        const Tensor *a = plain(k_scale), *b = plain(v_scale);
        for (const Tensor* s : {a, b})
            if (!good(s, at::kFloat, c->at) || s->dim() != 2 || s->size(0) != c->n_pages || s->size(1) != c->Hkv)
                return false;
        c->ks = static_cast<float*>(a->data_ptr());
        c->vs = static_cast<float*>(b->data_ptr());
    } else if (type != x->scalar_type() || k_scale != Py_None || v_scale != Py_None) {
        return false;
    }
    if (table != Py_None) {
        const Tensor* r = plain(table);
        if (!good(r, at::kFloat, c->at) || r->dim() != 3 || r->size(1) != c->D / 2 || r->size(2) != 2 || r->size(0) == 0 ||
            r->size(0) > INT_MAX)
            return false;
        c->rope = static_cast<const float*>(r->data_ptr());
        c->max_pos = (int)r->size(0);
    }
    return true;
}

// A window or a number of sinks: past a C int it means all keys. False for what
// is not a non-negative int.
bool count(PyObject* o, int* n) {
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (over < 0 || (over == 0 && x < 0)) return false;
    *n = over > 0 || x > INT_MAX ? INT_MAX : (int)x;
    return true;
}

bool scale_of(PyObject* o, float* s) {
    if (o == Py_None) {
        *s = NAN;
        return true;
    }
    if (!PyFloat_CheckExact(o)) return false;
    *s = (float)PyFloat_AS_DOUBLE(o);
    return true;
}

// The outputs of an attention over q: those given, or new ones.
bool outputs(const Tensor& q, int at, PyObject* out, PyObject* lse, Tensor* o, Tensor* l) {
    const int64_t B = q.size(0), S = q.size(1), H = q.size(2);
    if (out != Py_None) {
        const Tensor* t = plain(out);
        if (!good(t, q.scalar_type(), at) || t->sizes() != q.sizes()) return false;
        *o = *t;
    }
    if (lse != Py_None) {
        const Tensor* t = plain(lse);
        if (!good(t, at::kFloat, at) || t->dim() != 3 || t->size(0) != B || t->size(1) != H || t->size(2) != S) return false;
        *l = *t;
    }
    if (out == Py_None) *o = at::empty(q.sizes(), at::TensorOptions().dtype(q.scalar_type()).device(q.device()));
    if (lse == Py_None) *l = at::empty({B, H, S}, at::TensorOptions().dtype(at::kFloat).device(q.device()));
    return true;
}

PyObject* pair(PyObject* out, PyObject* lse, const Tensor& o, const Tensor& l) {
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, out != Py_None ? Py_NewRef(out) : THPVariable_Wrap(o));
    PyTuple_SET_ITEM(r, 1, lse != Py_None ? Py_NewRef(lse) : THPVariable_Wrap(l));
    return r;
}

// kv_append(k, v, k_cache, v_cache, block_table, kv_lens, new_lens, k_scale, v_scale, table)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 10) Py_RETURN_NONE;
    const Tensor *k = plain(a[0]), *v = plain(a[1]);
    Cache c;
    if (!open_cache(k, a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], &c)) Py_RETURN_NONE;
    if (!v || !v->defined() || !v->is_cuda() || v->device().index() != c.at || v->scalar_type() != k->scalar_type() ||
        v->sizes() != k->sizes() || c.H != c.Hkv)
        Py_RETURN_NONE;
    const long long ks = token_stride(*k), vs = token_stride(*v);
    if (ks < 0 || vs < 0) Py_RETURN_NONE;
    const void *kp = k->data_ptr(), *vp = v->data_ptr();
    const auto fn = k->scalar_type() == at::kBFloat16 ? attn_kv_append : attn_kv_append_f16;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(kp, vp, ks, vs, const_cast<void*>(c.k), const_cast<void*>(c.v), c.ks, c.vs, c.table, c.kv_lens, c.lens, c.B, c.S,
            c.Hkv, c.D, c.page, c.max_pages, c.n_pages, c.kind, c.rope, c.max_pos,
            reinterpret_cast<attn_stream_t>(c.stream));
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// attention_paged(q, k_cache, v_cache, block_table, kv_lens, q_lens, k_scale, v_scale, table, window, sinks, scale, out,
//                 lse, workspace, held, held_limit): (out, lse), a status, or None
// held: the thread's workspace for the default stream, or None; held_limit: what such a one may have at most.
PyObject* attention_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 17) Py_RETURN_NONE;
    const Tensor* q = plain(a[0]);
    Cache c;
    int window, sinks;
    float scale;
    if (!open_cache(q, a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], &c)) Py_RETURN_NONE;
    if (!count(a[9], &window) || !count(a[10], &sinks) || !scale_of(a[11], &scale)) Py_RETURN_NONE;
    const long long stride = token_stride(*q);
    if (stride < 0) Py_RETURN_NONE;
    Tensor ws;
    if (a[14] != Py_None) {
        const Tensor* t = plain(a[14]);
        if (!t || !t->defined() || !t->is_cuda() || t->device().index() != c.at || !t->is_contiguous()) Py_RETURN_NONE;
        ws = *t;
    } else {
        const size_t size = std::max<size_t>(
            1, attn_paged_workspace_bytes(c.B, c.H, c.Hkv, c.S, c.D, (long long)c.max_pages * c.page));
        if (c.stream == nullptr && size <= PyLong_AsSize_t(a[16])) {
            const Tensor* t = plain(a[15]);
            if (!t || (size_t)t->numel() < size) Py_RETURN_NONE;      // the wrapper makes a larger one
            ws = *t;
        } else {
            ws = at::empty({(int64_t)size}, at::TensorOptions().dtype(at::kByte).device(q->device()));
        }
    }
    Tensor o, l;
    if (!outputs(*q, c.at, a[12], a[13], &o, &l)) Py_RETURN_NONE;
    const void* qp = q->data_ptr();
    void *op = o.data_ptr(), *lp = l.data_ptr(), *wp = ws.data_ptr();
    const size_t bytes = ws.nbytes();
    const auto fn = q->scalar_type() == at::kBFloat16 ? attn_fwd_paged : attn_fwd_paged_f16;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(qp, stride, c.k, c.v, c.ks, c.vs, c.table, c.kv_lens, c.lens, op, static_cast<float*>(lp), c.B, c.H, c.Hkv, c.S,
            c.D, c.page, c.max_pages, c.n_pages, c.kind, scale, window, sinks, c.rope, c.max_pos, wp, bytes,
            reinterpret_cast<attn_stream_t>(c.stream));
    Py_END_ALLOW_THREADS
    return rc != ATTN_OK ? PyLong_FromLong(rc) : pair(a[12], a[13], o, l);
    END_HANDLE_TH_ERRORS
}

// attention_window(q, k, v, window, sinks, scale, out, lse): (out, lse), a status, or None
PyObject* attention_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) Py_RETURN_NONE;
    const Tensor *q = plain(a[0]), *k = plain(a[1]), *v = plain(a[2]);
    int at = -1, window, sinks;
    float scale;
    cudaStream_t stream;
    if (!begin(q, &at, &stream)) Py_RETURN_NONE;
    for (const Tensor* t : {q, k, v})
        if (!good(t, q->scalar_type(), at) || t->dim() != 4 || !fits(t->sizes())) Py_RETURN_NONE;
    if (k->size(0) != q->size(0) || k->size(3) != q->size(3) || v->sizes() != k->sizes()) Py_RETURN_NONE;
    if (!count(a[3], &window) || !count(a[4], &sinks) || !scale_of(a[5], &scale)) Py_RETURN_NONE;
    Tensor o, l;
    if (!outputs(*q, at, a[6], a[7], &o, &l)) Py_RETURN_NONE;
    const void *qp = q->data_ptr(), *kp = k->data_ptr(), *vp = v->data_ptr();
    void *op = o.data_ptr(), *lp = l.data_ptr();
    const int B = (int)q->size(0), Sq = (int)q->size(1), Hq = (int)q->size(2), D = (int)q->size(3);
    const int Sk = (int)k->size(1), Hkv = (int)k->size(2);
    const auto fn = q->scalar_type() == at::kBFloat16 ? attn_fwd_window : attn_fwd_window_f16;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(qp, kp, vp, op, static_cast<float*>(lp), B, Hq, Hkv, Sq, Sk, D, scale, window, sinks,
            reinterpret_cast<attn_stream_t>(stream));
    Py_END_ALLOW_THREADS
    return rc != ATTN_OK ? PyLong_FromLong(rc) : pair(a[6], a[7], o, l);
    END_HANDLE_TH_ERRORS
}

// A result of `like`'s shape and type on device `at`: the given one or a new one, and its token stride.
bool result(PyObject* o, const Tensor& like, int at, Tensor* t, long long* stride) {
    if (o == Py_None) {
        *t = at::empty(like.sizes(), at::TensorOptions().dtype(like.scalar_type()).device(like.device()));
    } else {
        const Tensor* g = plain(o);
        if (!g || !g->defined() || !g->is_cuda() || g->device().index() != at || g->scalar_type() != like.scalar_type() ||
            g->sizes() != like.sizes())
            return false;
        *t = *g;
    }
    return (*stride = token_stride(*t)) >= 0;
}

// A 4-D tensor of x's type and device with even tokens.
bool tokens(const Tensor* t, const Tensor& x, int at, long long* stride) {
    return t && t->defined() && t->is_cuda() && t->device().index() == at && t->scalar_type() == x.scalar_type() &&
           t->dim() == 4 && fits(t->sizes()) && (*stride = token_stride(*t)) >= 0;
}

PyObject* given(PyObject* o, const Tensor& t) { return o != Py_None ? Py_NewRef(o) : THPVariable_Wrap(t); }

// attention_backward(d_o, q, k, v, o, lse, causal, mask, window, sinks, scale, dq, dk, dv, workspace): (dq, dk, dv), a
// status, or None
PyObject* attention_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 15) Py_RETURN_NONE;
    const Tensor *g = plain(a[0]), *q = plain(a[1]), *k = plain(a[2]), *v = plain(a[3]), *o = plain(a[4]), *l = plain(a[5]);
    int at = -1, window, sinks;
    float scale;
    cudaStream_t stream;
    long long st[6];
    if (!begin(q, &at, &stream) || !tokens(q, *q, at, st) || !tokens(k, *q, at, st + 1) || !tokens(v, *q, at, st + 2))
        Py_RETURN_NONE;
    for (const Tensor* t : {g, o})
        if (!good(t, q->scalar_type(), at) || t->sizes() != q->sizes()) Py_RETURN_NONE;
    const int B = (int)q->size(0), Sq = (int)q->size(1), Hq = (int)q->size(2), D = (int)q->size(3);
    const int Sk = (int)k->size(1), Hkv = (int)k->size(2);
    if (k->size(0) != B || k->size(3) != D || v->sizes() != k->sizes()) Py_RETURN_NONE;
    if (!good(l, at::kFloat, at) || l->dim() != 3 || l->size(0) != B || l->size(1) != Hq || l->size(2) != Sq) Py_RETURN_NONE;
    if ((a[6] != Py_True && a[6] != Py_False) || !count(a[8], &window) || !count(a[9], &sinks) || !scale_of(a[10], &scale))
        Py_RETURN_NONE;
    const bool causal = a[6] == Py_True;
    const float* mask = nullptr;
    if (a[7] != Py_None) {
        const Tensor* m = plain(a[7]);
        if (!good(m, at::kFloat, at) || m->dim() != 3 || m->size(0) != B || m->size(1) != Sq || m->size(2) != Sk) Py_RETURN_NONE;
        mask = static_cast<const float*>(m->data_ptr());
    }
    if (window > 0 && (!causal || a[7] != Py_None)) Py_RETURN_NONE;
    const int kind = (causal ? ATTN_MASK_CAUSAL : ATTN_MASK_NONE) + (a[7] != Py_None ? ATTN_MASK_ADDITIVE : 0);
    Tensor ws;
    if (a[14] != Py_None) {
        const Tensor* t = plain(a[14]);
        if (!t || !t->defined() || !t->is_cuda() || t->device().index() != at || !t->is_contiguous()) Py_RETURN_NONE;
        ws = *t;
    }
    Tensor dq, dk, dv;
    if (!result(a[11], *q, at, &dq, st + 3) || !result(a[12], *k, at, &dk, st + 4) || !result(a[13], *k, at, &dv, st + 5))
        Py_RETURN_NONE;
    if (a[14] == Py_None) {
        const size_t size = std::max<size_t>(1, attn_bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, kind));
        ws = at::empty({(int64_t)size}, at::TensorOptions().dtype(at::kByte).device(q->device()));
    }
    const void *gp = g->data_ptr(), *qp = q->data_ptr(), *kp = k->data_ptr(), *vp = v->data_ptr(), *op = o->data_ptr();
    const float* lp = static_cast<const float*>(l->data_ptr());
    void *dqp = dq.data_ptr(), *dkp = dk.data_ptr(), *dvp = dv.data_ptr(), *wp = ws.data_ptr();
    const size_t bytes = ws.nbytes();
    const auto fn = q->scalar_type() == at::kBFloat16 ? attn_bwd : attn_bwd_f16;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(gp, qp, kp, vp, op, lp, dqp, dkp, dvp, st[0], st[1], st[2], st[3], st[4], st[5], B, Hq, Hkv, Sq, Sk, D, scale, kind,
            mask, window, sinks, wp, bytes, reinterpret_cast<attn_stream_t>(stream));
    Py_END_ALLOW_THREADS
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, given(a[11], dq));
    PyTuple_SET_ITEM(r, 1, given(a[12], dk));
    PyTuple_SET_ITEM(r, 2, given(a[13], dv));
    return r;
    END_HANDLE_TH_ERRORS
}

// rope_axes(q, k, table, positions, sections, inverse, q_out, k_out): (q_out, k_out), q_out without k, a status, or None
PyObject* rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8) Py_RETURN_NONE;
    const Tensor *q = plain(a[0]), *table = plain(a[2]), *pos = plain(a[3]);
    int at = -1, sections[4], axes = 0;
    cudaStream_t stream;
    long long qs, ks = 0, qos, kos = 0;
    if (!begin(q, &at, &stream) || !tokens(q, *q, at, &qs)) Py_RETURN_NONE;
    const int B = (int)q->size(0), S = (int)q->size(1), Hq = (int)q->size(2), D = (int)q->size(3);
    if (!PyTuple_CheckExact(a[4]) && !PyList_CheckExact(a[4])) Py_RETURN_NONE;
    const Py_ssize_t parts = PySequence_Fast_GET_SIZE(a[4]);
    long long pairs = 0;
    for (; axes < parts && axes < 4; ++axes) {
        if (!count(PySequence_Fast_GET_ITEM(a[4], axes), sections + axes) || sections[axes] > 512) Py_RETURN_NONE;
        pairs += sections[axes];
    }
    if (parts < 1 || parts > 4 || 2 * pairs != D) Py_RETURN_NONE;
    if (!good(pos, at::kInt, at) || pos->dim() != 3 || pos->size(0) != B || pos->size(1) != S || pos->size(2) != axes) Py_RETURN_NONE;
    if (!good(table, at::kFloat, at) || table->dim() != 3 || table->size(1) != D / 2 || table->size(2) != 2 ||
        table->size(0) == 0 || table->size(0) > INT_MAX || (a[5] != Py_True && a[5] != Py_False))
        Py_RETURN_NONE;
    const Tensor* k = nullptr;
    if (a[1] != Py_None) {
        k = plain(a[1]);
        if (!tokens(k, *q, at, &ks) || k->size(0) != B || k->size(1) != S || k->size(3) != D) Py_RETURN_NONE;
    } else if (a[7] != Py_None) {
        Py_RETURN_NONE;
    }
    Tensor qo, ko;
    if (!result(a[6], *q, at, &qo, &qos) || (k && !result(a[7], *k, at, &ko, &kos))) Py_RETURN_NONE;
    const void *qp = q->data_ptr(), *kp = k ? k->data_ptr() : nullptr;
    void *qop = qo.data_ptr(), *kop = k ? ko.data_ptr() : nullptr;
    const float* tp = static_cast<const float*>(table->data_ptr());
    const int *pp = static_cast<const int*>(pos->data_ptr()), max_pos = (int)table->size(0), Hkv = k ? (int)k->size(2) : 0;
    const auto fn = q->scalar_type() == at::kBFloat16 ? attn_rope_axes : attn_rope_axes_f16;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(qp, qop, qs, qos, kp, kop, ks, kos, B, S, Hq, Hkv, D, tp, max_pos, pp, sections, axes, a[5] == Py_True,
            reinterpret_cast<attn_stream_t>(stream));
    Py_END_ALLOW_THREADS
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    if (!k) return given(a[6], qo);
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, given(a[6], qo));
    PyTuple_SET_ITEM(r, 1, given(a[7], ko));
    return r;
    END_HANDLE_TH_ERRORS
}

// checkpoint_store(x, codes, scale): (codes, scale), a status, or None
PyObject* checkpoint_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 3) Py_RETURN_NONE;
    const Tensor* x = plain(a[0]);
    int at = -1;
    cudaStream_t stream;
    long long xs;
    if (!begin(x, &at, &stream) || !tokens(x, *x, at, &xs)) Py_RETURN_NONE;
    const int B = (int)x->size(0), S = (int)x->size(1), H = (int)x->size(2), D = (int)x->size(3);
    Tensor codes, scale;
    if (a[1] != Py_None) {
        const Tensor* t = plain(a[1]);
        if (!good(t, at::kFloat8_e4m3fn, at) || t->sizes() != x->sizes()) Py_RETURN_NONE;
        codes = *t;
    }
    if (a[2] != Py_None) {
        const Tensor* t = plain(a[2]);
        if (!good(t, at::kFloat, at) || t->dim() != 3 || t->size(0) != B || t->size(1) != S || t->size(2) != H) Py_RETURN_NONE;
        scale = *t;
    }
    if (a[1] == Py_None) codes = at::empty(x->sizes(), at::TensorOptions().dtype(at::kFloat8_e4m3fn).device(x->device()));
    if (a[2] == Py_None) scale = at::empty({B, S, H}, at::TensorOptions().dtype(at::kFloat).device(x->device()));
    const void* xp = x->data_ptr();
    void* cp = codes.data_ptr();
    float* sp = static_cast<float*>(scale.data_ptr());
    const auto fn = x->scalar_type() == at::kBFloat16 ? attn_checkpoint_store : attn_checkpoint_store_f16;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = fn(xp, xs, cp, sp, B, S, H, D, reinterpret_cast<attn_stream_t>(stream));
    Py_END_ALLOW_THREADS
    return rc != ATTN_OK ? PyLong_FromLong(rc) : pair(a[1], a[2], codes, scale);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"attention_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_paged)), METH_FASTCALL,
     nullptr},
    {"attention_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_window)), METH_FASTCALL,
     nullptr},
    {"attention_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_backward)), METH_FASTCALL,
     nullptr},
    {"rope_axes", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_axes)), METH_FASTCALL, nullptr},
    {"checkpoint_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(checkpoint_store)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
