// fastcall.cpp -- compiled argument marshalling for the entry points whose host time counts: a decode step's
// kernels take a few microseconds, the checks and allocations of a call from Python 12 to 20.
//
// Each function takes the arguments of the binding's function of that name, in order, and handles the
// ordinary call: tensors that pass the binding's checks, on the current device and its current stream.  It
// returns the result, or the library's status (an int) if that is not zero, or None for any call that it
// does not handle; the binding then goes through its own checks, which raise the errors.  The functions of
// the C ABI are handed over by address (bind), so this module holds no state of its own.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn_gb300.h"

namespace {

decltype(&paged_kv_append_rope) f_append;
decltype(&paged_kv_append_rope_fp8) f_append_fp8;
decltype(&attn_fwd_scoremod) f_fwd;
decltype(&attn_bwd_scoremod) f_bwd;
decltype(&attn_bwd_scoremod_workspace_size) f_bwd_ws;
decltype(&paged_attn_decode_scoremod) f_decode;
decltype(&paged_attn_decode_scoremod_fp8) f_decode_fp8;
decltype(&paged_attn_decode_scoremod_workspace_size) f_decode_ws;
decltype(&paged_attn_decode_shared) f_shared;
decltype(&paged_attn_decode_shared_fp8) f_shared_fp8;
decltype(&paged_attn_decode_shared_workspace_size) f_shared_ws;

// A call's tensors, all on one device; `ok` turns false at the first one that is not as it should be.
struct Call {
    bool ok = true;
    int device = -1;

    // A CUDA tensor of this type and number of dims on the call's device (any strides).
    const at::Tensor *strided(PyObject *o, at::ScalarType type, int dims) {
        if (!ok) return nullptr;
        ok = false;
        if (!THPVariable_Check(o)) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.defined() || t.key_set().has(c10::DispatchKey::Python) || !t.is_cuda() || t.scalar_type() != type ||
            t.dim() != dims)
            return nullptr;
        if (device < 0) device = t.device().index();
        ok = t.device().index() == device;
        return &t;
    }
    const at::Tensor *dense(PyObject *o, at::ScalarType type, int dims) {
        const at::Tensor *t = strided(o, type, dims);
        if (ok) ok = t->is_contiguous();
        return t;
    }
    // None, or such a tensor of this shape.
    const at::Tensor *optional(PyObject *o, at::ScalarType type, at::IntArrayRef shape) {
        if (!ok || o == Py_None) return nullptr;
        const at::Tensor *t = dense(o, type, (int)shape.size());
        if (ok) ok = t->sizes() == shape;
        return t;
    }
    void need(bool c) { ok = ok && c; }
    bool here() const { return ok && c10::cuda::current_device() == device; }
    attn_stream_t stream() const {
        return reinterpret_cast<attn_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    }
    // The output given, or a new one (made directly: a new tensor through the dispatcher costs 1.3 us, a call with
    // all of its outputs given 2.8).  The call's device is the current one here, and the memory belongs to its
    // current stream.
    at::Tensor output(const at::Tensor *given, at::IntArrayRef shape, at::ScalarType type) const {
        if (given) return *given;
        return at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                         c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
    }
};

// The workspace given (its size is the library's to check), or new memory of `need` bytes for the call: freed on
// the stream that it was made for, as a tensor's.
struct Workspace {
    c10::DataPtr own;
    void *data;
    size_t bytes;
    Workspace(const at::Tensor *given, size_t need) {
        if (given) {
            data = given->data_ptr();
            bytes = (size_t)given->numel();
        } else {
            bytes = need > 16 ? need : 16;
            own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
            data = own.get();
        }
    }
};

template <class T> T *ptr(const at::Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
int i32(int64_t x) { return x > INT_MAX ? INT_MAX : (int)x; }  // sizes past int are refused by the library

// A float argument; `none` where None may stand for it.
bool number(PyObject *o, double &x, double none = 0.0, bool may_be_none = false) {
    if (may_be_none && o == Py_None) {
        x = none;
        return true;
    }
    if (PyFloat_Check(o)) x = PyFloat_AS_DOUBLE(o);
    else if (PyLong_CheckExact(o)) x = PyLong_AsDouble(o);
    else return false;
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}
bool integer(PyObject *o, int &x) {
    if (!PyLong_Check(o)) return false;
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    x = (int)v;
    return v == x;
}
PyObject *none() { Py_RETURN_NONE; }
PyObject *pair(const at::Tensor &a, const at::Tensor *b) {
    PyObject *x = THPVariable_Wrap(a), *y;
    if (b) {
        y = THPVariable_Wrap(*b);
    } else {
        y = Py_None;
        Py_INCREF(y);
    }
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}
// Runs a body whose allocations may throw (before anything is launched): such a call is left to the binding,
// where torch raises its own error.
template <class F> PyObject *guarded(F &&body) {
    try {
        return body();
    } catch (const std::exception &) {
        return none();
    }
}
#define WITHOUT_GIL(call)        \
    do {                         \
        Py_BEGIN_ALLOW_THREADS;  \
        st = call;               \
        Py_END_ALLOW_THREADS;    \
    } while (0)

// Strides of a [B, heads, N, d] view with contiguous rows (those of dims of size one count as 0).
bool row_strides(const at::Tensor &t, int64_t (&s)[3]) {
    const auto size = t.sizes(), st = t.strides();
    if (st[3] != 1 && size[3] != 1) return false;
    for (int i = 0; i < 3; ++i) {
        s[i] = size[i] == 1 ? 0 : st[i];
        if (s[i] % 8 != 0) return false;
    }
    return true;
}

// (scales or None, q, k_new, v_new, k_pages, v_pages, cos_sin, page_table, start_pos, interleaved, new_lens, q_out)
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12 || !f_append || !f_append_fp8) return none();
    return guarded([&]() -> PyObject * {
        const bool fp8 = a[0] != Py_None;
        double ks = 1, vs = 1;
        if (fp8 && (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 2 || !number(PyTuple_GET_ITEM(a[0], 0), ks) ||
                    !number(PyTuple_GET_ITEM(a[0], 1), vs)))
            return none();
        Call c;
        const at::Tensor *k = c.strided(a[2], at::kBFloat16, 4), *v = c.strided(a[3], at::kBFloat16, 4);
        const at::ScalarType page = fp8 ? at::kByte : at::kBFloat16;
        const at::Tensor *kp = c.dense(a[4], page, 4), *vp = c.dense(a[5], page, 4);
        const at::Tensor *cs = c.dense(a[6], at::kFloat, 2);
        const at::Tensor *table = c.dense(a[7], at::kInt, 2), *start = c.dense(a[8], at::kInt, 1);
        const at::Tensor *q = a[1] == Py_None ? nullptr : c.strided(a[1], at::kBFloat16, 4);
        if (!c.ok) return none();
        const int64_t B = k->size(0), Hkv = k->size(1), N = k->size(2), d = k->size(3), H = q ? q->size(1) : 0;
        c.need(v->sizes() == k->sizes() && vp->sizes() == kp->sizes() && kp->size(1) == Hkv && kp->size(3) == d);
        c.need(table->size(0) == B && start->size(0) == B);
        const at::Tensor *lens = c.optional(a[10], at::kInt, {B});
        if (q) c.need(q->size(0) == B && q->size(2) == N && q->size(3) == d);
        else c.need(a[11] == Py_None);
        const at::Tensor *given = c.optional(a[11], at::kBFloat16, {B, H, N, d});
        int64_t qst[3] = {0, 0, 0}, kst[3], vst[3];
        if (!c.here() || !row_strides(*k, kst) || !row_strides(*v, vst) || (q && !row_strides(*q, qst))) return none();
        const int inter = PyObject_IsTrue(a[9]);
        if (inter < 0) return nullptr;
        at::Tensor out;
        if (q) out = c.output(given, {B, H, N, d}, at::kBFloat16);
        const attn_stream_t s = c.stream();
        void *qo = q ? out.data_ptr() : nullptr;
        int st;
        if (fp8)
            WITHOUT_GIL(f_append_fp8(ptr<void>(q), qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(),
                                     vp->data_ptr(), (float)ks, (float)vs, ptr<float>(cs), i32(cs->size(1)),
                                     i32(cs->size(0)), inter, ptr<int32_t>(table), ptr<int32_t>(start),
                                     ptr<int32_t>(lens), i32(kp->size(2)), i32(B), i32(H), i32(Hkv), i32(N), i32(d),
                                     i32(table->size(1)), i32(kp->size(0)), s));
        else
            WITHOUT_GIL(f_append(ptr<void>(q), qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(),
                                 vp->data_ptr(), ptr<float>(cs), i32(cs->size(1)), i32(cs->size(0)), inter,
                                 ptr<int32_t>(table), ptr<int32_t>(start), ptr<int32_t>(lens), i32(kp->size(2)), i32(B),
                                 i32(H), i32(Hkv), i32(N), i32(d), i32(table->size(1)), i32(kp->size(0)), s));
        if (st) return PyLong_FromLong(st);
        PyObject *r = a[11] != Py_None ? a[11] : nullptr;  // the caller's own tensor, not a second wrapper
        if (r) {
            Py_INCREF(r);
        } else if (q) {
            r = THPVariable_Wrap(out);
        } else {
            r = Py_False;  // done, and nothing to return
            Py_INCREF(r);
        }
        return r;
    });
}

// q [B, Hq, Nq, d] and k, v [B, Hkv, Nkv, d] with the modification's optional tensors at a[at ..].
struct Dense {
    const at::Tensor *q, *k, *v, *slopes, *begin, *end, *lens;
    int64_t B, Hq, Hkv, Nq, Nkv, d;
    bool get(Call &c, PyObject *const *a, int at) {
        q = c.dense(a[0], at::kBFloat16, 4);
        k = c.dense(a[1], at::kBFloat16, 4);
        v = c.dense(a[2], at::kBFloat16, 4);
        if (!c.ok) return false;
        B = q->size(0), Hq = q->size(1), Nq = q->size(2), d = q->size(3), Hkv = k->size(1), Nkv = k->size(2);
        c.need(k->size(0) == B && k->size(3) == d && v->sizes() == k->sizes());
        slopes = c.optional(a[at], at::kFloat, {Hq});
        begin = c.optional(a[at + 1], at::kInt, {B, Nq});
        end = c.optional(a[at + 2], at::kInt, {B, Nq});
        lens = c.optional(a[at + 3], at::kInt, {B});
        return c.ok;
    }
};

// (q, k, v, causal, scale, softcap, alibi_slopes, key_begin, key_end, kv_lens, out, lse, return_lse)
PyObject *fwd_scoremod(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || !f_fwd) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        Dense x;
        double scale, cap;
        if (!x.get(c, a, 6) || !number(a[4], scale, 1.0 / std::sqrt((double)x.d), true) || !number(a[5], cap)) return none();
        const at::Tensor *go = c.optional(a[10], at::kBFloat16, x.q->sizes());
        const at::Tensor *gl = c.optional(a[11], at::kFloat, {x.B, x.Hq, x.Nq});
        const int causal = PyObject_IsTrue(a[3]), want = PyObject_IsTrue(a[12]);
        if (causal < 0 || want < 0) return nullptr;
        if (!c.here()) return none();
        at::Tensor o = c.output(go, x.q->sizes(), at::kBFloat16), l;
        if (gl || want) l = c.output(gl, {x.B, x.Hq, x.Nq}, at::kFloat);
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_fwd(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), o.data_ptr(), l.defined() ? ptr<float>(&l) : nullptr,
                          i32(x.B), i32(x.Hq), i32(x.Hkv), i32(x.Nq), i32(x.Nkv), i32(x.d), causal, (float)scale, (float)cap,
                          ptr<float>(x.slopes), ptr<int32_t>(x.begin), ptr<int32_t>(x.end), ptr<int32_t>(x.lens), s));
        if (st) return PyLong_FromLong(st);
        return pair(o, l.defined() ? &l : nullptr);
    });
}

// (q, k, v, o, lse, dout, causal, scale, softcap, alibi_slopes, key_begin, key_end, kv_lens, dq, dk, dv, workspace)
PyObject *bwd_scoremod(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 17 || !f_bwd || !f_bwd_ws) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        Dense x;
        double scale, cap;
        if (!x.get(c, a, 9) || !number(a[7], scale, 1.0 / std::sqrt((double)x.d), true) || !number(a[8], cap)) return none();
        const at::Tensor *o = c.dense(a[3], at::kBFloat16, 4), *l = c.dense(a[4], at::kFloat, 3);
        const at::Tensor *g = c.dense(a[5], at::kBFloat16, 4);
        if (!c.ok) return none();
        c.need(o->sizes() == x.q->sizes() && g->sizes() == x.q->sizes() && l->sizes() == x.q->sizes().slice(0, 3));
        const at::Tensor *gq = c.optional(a[13], at::kBFloat16, x.q->sizes());
        const at::Tensor *gk = c.optional(a[14], at::kBFloat16, x.k->sizes());
        const at::Tensor *gv = c.optional(a[15], at::kBFloat16, x.k->sizes());
        const at::Tensor *gw = a[16] == Py_None ? nullptr : c.dense(a[16], at::kByte, 1);
        const int causal = PyObject_IsTrue(a[6]);
        if (causal < 0) return nullptr;
        if (!c.here()) return none();
        const int B = i32(x.B), Hq = i32(x.Hq), Hkv = i32(x.Hkv), Nq = i32(x.Nq), Nkv = i32(x.Nkv), d = i32(x.d);
        at::Tensor dq = c.output(gq, x.q->sizes(), at::kBFloat16), dk = c.output(gk, x.k->sizes(), at::kBFloat16);
        at::Tensor dv = c.output(gv, x.k->sizes(), at::kBFloat16);
        const Workspace w(gw, f_bwd_ws(B, Hq, Hkv, Nq, Nkv, d));
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_bwd(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), o->data_ptr(), ptr<float>(l), g->data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Nq, Nkv, d, causal, (float)scale,
                          (float)cap, ptr<float>(x.slopes), ptr<int32_t>(x.begin), ptr<int32_t>(x.end),
                          ptr<int32_t>(x.lens), w.data, w.bytes, s));
        if (st) return PyLong_FromLong(st);
        PyObject *p[3] = {THPVariable_Wrap(dq), THPVariable_Wrap(dk), THPVariable_Wrap(dv)};
        PyObject *r = p[0] && p[1] && p[2] ? PyTuple_Pack(3, p[0], p[1], p[2]) : nullptr;
        for (PyObject *y : p) Py_XDECREF(y);
        return r;
    });
}

// A decode batch over a paged cache: a[0] scales or None, then q, k_pages, v_pages, page_table, ctx_lens.
struct Paged {
    const at::Tensor *q, *k, *v, *table, *ctx;
    bool fp8;
    double ks = 1, vs = 1;
    int B, H, Hkv, d, max_pages, num_pages, page_size;
    bool get(Call &c, PyObject *const *a) {
        fp8 = a[0] != Py_None;
        if (fp8 && (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 2 || !number(PyTuple_GET_ITEM(a[0], 0), ks) ||
                    !number(PyTuple_GET_ITEM(a[0], 1), vs)))
            return false;
        const at::ScalarType page = fp8 ? at::kByte : at::kBFloat16;
        q = c.dense(a[1], at::kBFloat16, 3);
        k = c.dense(a[2], page, 4);
        v = c.dense(a[3], page, 4);
        table = c.dense(a[4], at::kInt, 2);
        ctx = c.dense(a[5], at::kInt, 1);
        if (!c.ok) return false;
        c.need(k->size(3) == q->size(2) && v->sizes() == k->sizes() && table->size(0) == q->size(0) &&
               ctx->size(0) == q->size(0));
        B = i32(q->size(0)), H = i32(q->size(1)), d = i32(q->size(2)), Hkv = i32(k->size(1));
        num_pages = i32(k->size(0)), page_size = i32(k->size(2)), max_pages = i32(table->size(1));
        return c.ok;
    }
};

// (scales, q, k_pages, v_pages, page_table, ctx_lens, scale, softcap, alibi_slopes, key_begin, out, lse, workspace,
//  return_lse)
PyObject *decode_scoremod(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 14 || !f_decode || !f_decode_fp8 || !f_decode_ws) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        Paged x;
        double scale, cap;
        if (!x.get(c, a) || !number(a[6], scale, 1.0 / std::sqrt((double)x.d), true) || !number(a[7], cap)) return none();
        const at::Tensor *slopes = c.optional(a[8], at::kFloat, {x.H}), *begin = c.optional(a[9], at::kInt, {x.B});
        const at::Tensor *go = c.optional(a[10], at::kBFloat16, x.q->sizes()), *gl = c.optional(a[11], at::kFloat, {x.B, x.H});
        const at::Tensor *gw = a[12] == Py_None ? nullptr : c.dense(a[12], at::kByte, 1);
        const int want = PyObject_IsTrue(a[13]);
        if (want < 0) return nullptr;
        if (!c.here()) return none();
        at::Tensor o = c.output(go, x.q->sizes(), at::kBFloat16), l;
        if (gl || want) l = c.output(gl, {x.B, x.H}, at::kFloat);
        const Workspace w(gw, f_decode_ws(x.B, x.H, x.Hkv, x.d, x.max_pages, x.page_size));
        float *lp = l.defined() ? ptr<float>(&l) : nullptr;
        const attn_stream_t s = c.stream();
        int st;
        if (x.fp8)
            WITHOUT_GIL(f_decode_fp8(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), (float)x.ks, (float)x.vs,
                                     ptr<int32_t>(x.table), ptr<int32_t>(x.ctx), x.page_size, o.data_ptr(), lp, x.B, x.H,
                                     x.Hkv, x.d, x.max_pages, x.num_pages, (float)scale, (float)cap, ptr<float>(slopes),
                                     ptr<int32_t>(begin), w.data, w.bytes, s));
        else
            WITHOUT_GIL(f_decode(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), ptr<int32_t>(x.table),
                                 ptr<int32_t>(x.ctx), x.page_size, o.data_ptr(), lp, x.B, x.H, x.Hkv, x.d, x.max_pages,
                                 x.num_pages, (float)scale, (float)cap, ptr<float>(slopes), ptr<int32_t>(begin),
                                 w.data, w.bytes, s));
        if (st) return PyLong_FromLong(st);
        return pair(o, l.defined() ? &l : nullptr);
    });
}

// (scales, q, k_pages, v_pages, page_table, ctx_lens, shared_pages, group_size, scale, out, lse, workspace, return_lse)
PyObject *decode_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || !f_shared || !f_shared_fp8 || !f_shared_ws) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        Paged x;
        double scale;
        int S;
        if (!x.get(c, a) || !integer(a[7], S) || S <= 0 || x.B % S != 0 ||
            !number(a[8], scale, 1.0 / std::sqrt((double)x.d), true))
            return none();
        const at::Tensor *shared = c.optional(a[6], at::kInt, {x.B / S});
        const at::Tensor *go = c.optional(a[9], at::kBFloat16, x.q->sizes()), *gl = c.optional(a[10], at::kFloat, {x.B, x.H});
        const at::Tensor *gw = a[11] == Py_None ? nullptr : c.dense(a[11], at::kByte, 1);
        const int want = PyObject_IsTrue(a[12]);
        if (want < 0) return nullptr;
        if (!shared || !c.here()) return none();
        at::Tensor o = c.output(go, x.q->sizes(), at::kBFloat16), l;
        if (gl || want) l = c.output(gl, {x.B, x.H}, at::kFloat);
        const Workspace w(gw, f_shared_ws(x.B, x.H, x.Hkv, x.d, x.max_pages, S, x.page_size));
        float *lp = l.defined() ? ptr<float>(&l) : nullptr;
        const attn_stream_t s = c.stream();
        int st;
        if (x.fp8)
            WITHOUT_GIL(f_shared_fp8(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), (float)x.ks, (float)x.vs,
                                     ptr<int32_t>(x.table), ptr<int32_t>(x.ctx), ptr<int32_t>(shared), S, x.page_size,
                                     o.data_ptr(), lp, x.B, x.H, x.Hkv, x.d, x.max_pages, x.num_pages, (float)scale,
                                     w.data, w.bytes, s));
        else
            WITHOUT_GIL(f_shared(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), ptr<int32_t>(x.table),
                                 ptr<int32_t>(x.ctx), ptr<int32_t>(shared), S, x.page_size, o.data_ptr(), lp, x.B, x.H,
                                 x.Hkv, x.d, x.max_pages, x.num_pages, (float)scale, w.data, w.bytes, s));
        if (st) return PyLong_FromLong(st);
        return pair(o, l.defined() ? &l : nullptr);
    });
}

// bind({name: address of the C ABI's function})
PyObject *bind(PyObject *, PyObject *table) {
    if (!PyDict_Check(table)) {
        PyErr_SetString(PyExc_TypeError, "a dict of addresses");
        return nullptr;
    }
    bool ok = true;
    auto take = [&](const char *name, auto &f) {
        PyObject *v = PyDict_GetItemString(table, name);
        void *p = v ? PyLong_AsVoidPtr(v) : nullptr;
        if (!p) ok = false;
        f = reinterpret_cast<std::decay_t<decltype(f)>>(p);
    };
    take("paged_kv_append_rope", f_append);
    take("paged_kv_append_rope_fp8", f_append_fp8);
    take("attn_fwd_scoremod", f_fwd);
    take("attn_bwd_scoremod", f_bwd);
    take("attn_bwd_scoremod_workspace_size", f_bwd_ws);
    take("paged_attn_decode_scoremod", f_decode);
    take("paged_attn_decode_scoremod_fp8", f_decode_fp8);
    take("paged_attn_decode_scoremod_workspace_size", f_decode_ws);
    take("paged_attn_decode_shared", f_shared);
    take("paged_attn_decode_shared_fp8", f_shared_fp8);
    take("paged_attn_decode_shared_workspace_size", f_shared_ws);
    if (PyErr_Occurred()) return nullptr;
    return PyBool_FromLong(ok);
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr}, FAST(append_rope),     FAST(fwd_scoremod),  FAST(bwd_scoremod),
                         FAST(decode_scoremod),           FAST(decode_shared),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
    PyObject *m = PyModule_Create(&module);
    // the torch (its full version) and the C++ ABI that this was compiled against; the binding uses the module with
    // those only
    if (m && (PyModule_AddStringConstant(m, "torch_version", ATTN_TORCH_VERSION) < 0 ||
              PyModule_AddIntConstant(m, "cxx11_abi", _GLIBCXX_USE_CXX11_ABI) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
