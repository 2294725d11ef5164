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

#include <vector>

#include "attn_gb300.h"

namespace {

decltype(&paged_kv_append_rope) f_append;
decltype(&paged_kv_append_rope_fp8) f_append_fp8;
decltype(&paged_kv_append_rope_axes) f_append_axes;
decltype(&paged_kv_append_rope_axes_fp8) f_append_axes_fp8;
decltype(&paged_kv_append_fp4) f_append_fp4;
decltype(&paged_kv_unpack_fp4) f_unpack;
decltype(&attn_rope_axes) f_rope;
decltype(&attn_rope_axes_bwd) f_rope_bwd;
decltype(&paged_attn_decode_fp4) f_decode4;
decltype(&paged_attn_decode_fp4_workspace_size) f_decode4_ws;
decltype(&paged_kv_fork) f_fork;
decltype(&paged_kv_reserve) f_reserve;
decltype(&paged_kv_reserve_workspace_size) f_reserve_ws;
decltype(&paged_kv_compact) f_compact;
decltype(&paged_kv_compact_workspace_size) f_compact_ws;
decltype(&paged_kv_copy_pages) f_copy_pages;
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

// Positions [axes, B, N] (`shared`: or [axes, 1, N]) and the bytes of the pairs' axes.
struct Axes {
    const at::Tensor *positions = nullptr;
    const uint8_t *axis = nullptr;
    bool get(Call &c, PyObject *pos, PyObject *pairs, int64_t B, int64_t N, int64_t rope, bool shared) {
        positions = c.dense(pos, at::kInt, 3);
        if (!c.ok || !PyBytes_CheckExact(pairs) || 2 * PyBytes_GET_SIZE(pairs) != rope) return c.ok = false;
        axis = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(pairs));
        c.need(positions->size(2) == N && (positions->size(1) == B || (shared && positions->size(1) == 1)));
        return c.ok;
    }
    int axes() const { return positions ? i32(positions->size(0)) : 0; }
};

// (scales or None, q, k_new, v_new, k_pages, v_pages, cos_sin, page_table, start_pos, interleaved, new_lens, q_out[,
//  positions, pair_axis]); fp4: into the 4-bit cache, where cos_sin and the last two may be None
PyObject *append_any(PyObject *const *a, Py_ssize_t n, bool fp4) {
    if ((n != 12 || fp4) && n != 14) return none();
    return guarded([&]() -> PyObject * {
        const bool fp8 = a[0] != Py_None;  // (or fp4: with scales)
        double ks = 1, vs = 1;
        if (fp8 && (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 2 || !number(PyTuple_GET_ITEM(a[0], 0), ks) ||
                    !number(PyTuple_GET_ITEM(a[0], 1), vs)))
            return none();
        Call c;
        const at::Tensor *k = c.strided(a[2], at::kBFloat16, 4), *v = c.strided(a[3], at::kBFloat16, 4);
        const at::ScalarType page = fp8 ? at::kByte : at::kBFloat16;
        const at::Tensor *kp = c.dense(a[4], page, fp4 ? 3 : 4), *vp = c.dense(a[5], page, fp4 ? 3 : 4);
        const at::Tensor *cs = fp4 && a[6] == Py_None ? nullptr : c.dense(a[6], at::kFloat, 2);
        const at::Tensor *table = c.dense(a[7], at::kInt, 2), *start = c.dense(a[8], at::kInt, 1);
        const at::Tensor *q = a[1] == Py_None ? nullptr : c.strided(a[1], at::kBFloat16, 4);
        if (!c.ok) return none();
        const int64_t B = k->size(0), Hkv = k->size(1), N = k->size(2), d = k->size(3), H = q ? q->size(1) : 0;
        c.need(v->sizes() == k->sizes() && vp->sizes() == kp->sizes() && kp->size(1) == Hkv);
        c.need(fp4 ? kp->size(2) == 9 * d : kp->size(3) == d);
        c.need(table->size(0) == B && start->size(0) == B);
        const at::Tensor *lens = c.optional(a[10], at::kInt, {B});
        if (q) c.need(cs && q->size(0) == B && q->size(2) == N && q->size(3) == d);
        else c.need(a[11] == Py_None);
        const at::Tensor *given = c.optional(a[11], at::kBFloat16, {B, H, N, d});
        const bool axes = n == 14 && (!fp4 || a[12] != Py_None);
        Axes x;
        if (axes && (!cs || !x.get(c, a[12], a[13], B, N, cs->size(1), false))) return none();
        if (n == 14 && !axes && a[13] != Py_None) return none();
        int64_t qst[3] = {0, 0, 0}, kst[3], vst[3];
        if (!c.here() || !row_strides(*k, kst) || !row_strides(*v, vst) || (q && !row_strides(*q, qst))) return none();
        const int inter = PyObject_IsTrue(a[9]);
        if (inter < 0) return nullptr;
        at::Tensor out;
        if (q) out = c.output(given, {B, H, N, d}, at::kBFloat16);
        const attn_stream_t s = c.stream();
        void *qo = q ? out.data_ptr() : nullptr;
        const void *qp = ptr<void>(q);
        float *csp = ptr<float>(cs);
        const int rope = cs ? i32(cs->size(1)) : 0, rows = cs ? i32(cs->size(0)) : 0;
        int32_t *pos = ptr<int32_t>(x.positions), *tp = ptr<int32_t>(table), *sp = ptr<int32_t>(start), *lp = ptr<int32_t>(lens);
        const int Bi = i32(B), Hi = i32(H), Hk = i32(Hkv), Ni = i32(N), di = i32(d), W = i32(table->size(1)), P = i32(kp->size(0));
        const int ps = fp4 ? 16 : i32(kp->size(2));
        const float kf = (float)ks, vf = (float)vs;
        int st;
        if (fp4)
            WITHOUT_GIL(f_append_fp4(qp, qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(), vp->data_ptr(), kf,
                                     vf, csp, rope, rows, inter, pos, x.axes(), x.axis, tp, sp, lp, ps, Bi, Hi, Hk, Ni, di, W,
                                     P, s));
        else if (axes && fp8)
            WITHOUT_GIL(f_append_axes_fp8(qp, qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(), vp->data_ptr(),
                                          kf, vf, csp, rope, rows, inter, pos, x.axes(), x.axis, tp, sp, lp, ps, Bi, Hi, Hk,
                                          Ni, di, W, P, s));
        else if (axes)
            WITHOUT_GIL(f_append_axes(qp, qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(), vp->data_ptr(), csp,
                                      rope, rows, inter, pos, x.axes(), x.axis, tp, sp, lp, ps, Bi, Hi, Hk, Ni, di, W, P, s));
        else if (fp8)
            WITHOUT_GIL(f_append_fp8(qp, qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(), vp->data_ptr(), kf,
                                     vf, csp, rope, rows, inter, tp, sp, lp, ps, Bi, Hi, Hk, Ni, di, W, P, s));
        else
            WITHOUT_GIL(f_append(qp, qst, k->data_ptr(), kst, v->data_ptr(), vst, qo, kp->data_ptr(), vp->data_ptr(), csp,
                                 rope, rows, inter, tp, sp, lp, ps, Bi, Hi, Hk, Ni, di, W, P, s));
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
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return f_append && f_append_fp8 && f_append_axes && f_append_axes_fp8 ? append_any(a, n, false) : none();
}
PyObject *append_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) { return f_append_fp4 ? append_any(a, n, true) : none(); }

// An output: the caller's own object, or a new tensor's.
PyObject *own_or_new(PyObject *given, const at::Tensor &t) {
    if (given == Py_None) return THPVariable_Wrap(t);
    Py_INCREF(given);
    return given;
}
// A tuple of new references (null: the failure of one of them).
template <size_t N> PyObject *tuple_of(PyObject *(&p)[N]) {
    PyObject *r = PyTuple_New(N);
    bool ok = r != nullptr;
    for (PyObject *x : p) ok = ok && x;
    if (!ok) {
        Py_XDECREF(r);
        for (PyObject *x : p) Py_XDECREF(x);
        return nullptr;
    }
    for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(r, (Py_ssize_t)i, p[i]);
    return r;
}

// ((k_scale, v_scale), k_pages, v_pages, page_ids, k_out, v_out)
PyObject *unpack_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6 || !f_unpack) return none();
    return guarded([&]() -> PyObject * {
        double ks, vs;
        if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 2 || !number(PyTuple_GET_ITEM(a[0], 0), ks) ||
            !number(PyTuple_GET_ITEM(a[0], 1), vs))
            return none();
        Call c;
        const at::Tensor *k = c.dense(a[1], at::kByte, 3), *v = c.dense(a[2], at::kByte, 3), *ids = c.dense(a[3], at::kInt, 1);
        if (!c.ok) return none();
        const int64_t m = ids->size(0), Hkv = k->size(1), d = k->size(2) / 9;
        c.need(k->size(2) == 9 * d && v->sizes() == k->sizes());
        const at::Tensor *gk = c.optional(a[4], at::kBFloat16, {m, Hkv, 16, d}), *gv = c.optional(a[5], at::kBFloat16, {m, Hkv, 16, d});
        if (!c.here()) return none();
        at::Tensor ko = c.output(gk, {m, Hkv, 16, d}, at::kBFloat16), vo = c.output(gv, {m, Hkv, 16, d}, at::kBFloat16);
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_unpack(k->data_ptr(), v->data_ptr(), (float)ks, (float)vs, ptr<int32_t>(ids), i32(m), ko.data_ptr(),
                             vo.data_ptr(), 16, i32(Hkv), i32(d), i32(k->size(0)), s));
        if (st) return PyLong_FromLong(st);
        PyObject *p[2] = {own_or_new(a[4], ko), own_or_new(a[5], vo)};
        return tuple_of(p);
    });
}

// (backward, q, k, cos_sin, positions, pair_axis, interleaved, q_out, k_out)
PyObject *rope_axes(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || !f_rope || !f_rope_bwd) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const at::Tensor *q = c.strided(a[1], at::kBFloat16, 4);
        const at::Tensor *k = a[2] == Py_None ? nullptr : c.strided(a[2], at::kBFloat16, 4);
        const at::Tensor *cs = c.dense(a[3], at::kFloat, 2);
        if (!c.ok) return none();
        const int64_t B = q->size(0), H = q->size(1), N = q->size(2), d = q->size(3), Hkv = k ? k->size(1) : 0;
        if (k) c.need(k->size(0) == B && k->size(2) == N && k->size(3) == d);
        else c.need(a[8] == Py_None);
        Axes x;
        if (!x.get(c, a[4], a[5], B, N, cs->size(1), true)) return none();
        const at::Tensor *gq = a[7] == Py_None ? nullptr : c.strided(a[7], at::kBFloat16, 4);
        const at::Tensor *gk = a[8] == Py_None ? nullptr : c.strided(a[8], at::kBFloat16, 4);
        if (!c.ok) return none();
        if (gq) c.need(gq->sizes() == q->sizes());
        if (gk) c.need(gk->sizes() == k->sizes());
        const int back = PyObject_IsTrue(a[0]), inter = PyObject_IsTrue(a[6]);
        if (back < 0 || inter < 0) return nullptr;
        if (!c.here()) return none();
        at::Tensor qo = c.output(gq, {B, H, N, d}, at::kBFloat16), ko;
        if (k) ko = c.output(gk, {B, Hkv, N, d}, at::kBFloat16);
        int64_t qst[3], kst[3] = {0, 0, 0}, qos[3], kos[3] = {0, 0, 0};
        if (!row_strides(*q, qst) || !row_strides(qo, qos) || (k && (!row_strides(*k, kst) || !row_strides(ko, kos)))) return none();
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL((back ? f_rope_bwd : f_rope)(q->data_ptr(), qst, ptr<void>(k), kst, ptr<float>(cs), i32(cs->size(1)),
                                                 i32(cs->size(0)), inter, ptr<int32_t>(x.positions), x.axes(),
                                                 i32(x.positions->size(1)), x.axis, qo.data_ptr(), qos,
                                                 k ? ko.data_ptr() : nullptr, kos, i32(B), i32(H), i32(Hkv), i32(N), i32(d), s));
        if (st) return PyLong_FromLong(st);
        PyObject *none_ref = Py_None;
        if (!k) Py_INCREF(none_ref);
        PyObject *p[2] = {own_or_new(a[7], qo), k ? own_or_new(a[8], ko) : none_ref};
        return tuple_of(p);
    });
}

// (page_table, ctx_lens, parents, ref_counts, page_table_out, ctx_lens_out, ref_counts_out)
PyObject *kv_fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7 || !f_fork) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const at::Tensor *t = c.dense(a[0], at::kInt, 2), *par = c.dense(a[2], at::kInt, 1), *ref = c.dense(a[3], at::kInt, 1);
        if (!c.ok) return none();
        const int64_t B = t->size(0), W = t->size(1), Bo = par->size(0), P = ref->size(0);
        const at::Tensor *ctx = c.optional(a[1], at::kInt, {B}), *gt = c.optional(a[4], at::kInt, {Bo, W});
        const at::Tensor *gc = c.optional(a[5], at::kInt, {Bo}), *gr = c.optional(a[6], at::kInt, {P});
        if (!ctx || !c.here()) return none();
        at::Tensor to = c.output(gt, {Bo, W}, at::kInt), co = c.output(gc, {Bo}, at::kInt), ro = c.output(gr, {P}, at::kInt);
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_fork(ptr<int32_t>(t), ptr<int32_t>(ctx), ptr<int32_t>(par), ptr<int32_t>(ref), ptr<int32_t>(&to),
                           ptr<int32_t>(&co), ptr<int32_t>(&ro), 16, i32(B), i32(Bo), i32(W), i32(P), s));
        if (st) return PyLong_FromLong(st);
        PyObject *p[3] = {own_or_new(a[4], to), own_or_new(a[5], co), own_or_new(a[6], ro)};
        return tuple_of(p);
    });
}

// (page_table, ctx_lens, new_lens, ref_counts, page_table_out, ref_counts_out, reserved, src_pages, dst_pages, workspace)
PyObject *kv_reserve(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10 || !f_reserve || !f_reserve_ws) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const at::Tensor *t = c.dense(a[0], at::kInt, 2), *ref = c.dense(a[3], at::kInt, 1);
        if (!c.ok) return none();
        const int64_t B = t->size(0), W = t->size(1), P = ref->size(0);
        const at::Tensor *ctx = c.optional(a[1], at::kInt, {B}), *add = c.optional(a[2], at::kInt, {B});
        const at::Tensor *gt = c.optional(a[4], at::kInt, {B, W}), *gr = c.optional(a[5], at::kInt, {P});
        const at::Tensor *g[3];
        for (int i = 0; i < 3; ++i) g[i] = c.optional(a[6 + i], at::kInt, {B});
        const at::Tensor *gw = a[9] == Py_None ? nullptr : c.dense(a[9], at::kByte, 1);
        if (!ctx || !add || !c.here()) return none();
        at::Tensor to = c.output(gt, {B, W}, at::kInt), ro = c.output(gr, {P}, at::kInt), o[3];
        for (int i = 0; i < 3; ++i) o[i] = c.output(g[i], {B}, at::kInt);
        const Workspace w(gw, f_reserve_ws(i32(B), i32(P)));
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_reserve(ptr<int32_t>(t), ptr<int32_t>(ctx), ptr<int32_t>(add), ptr<int32_t>(ref), ptr<int32_t>(&to),
                              ptr<int32_t>(&ro), ptr<int32_t>(&o[0]), ptr<int32_t>(&o[1]), ptr<int32_t>(&o[2]), 16, i32(B),
                              i32(W), i32(P), w.data, w.bytes, s));
        if (st) return PyLong_FromLong(st);
        PyObject *p[5] = {own_or_new(a[4], to), own_or_new(a[5], ro), own_or_new(a[6], o[0]), own_or_new(a[7], o[1]),
                          own_or_new(a[8], o[2])};
        return tuple_of(p);
    });
}

// (page_table, ref_counts, page_table_out, ref_counts_out, src_pages, dst_pages, count, workspace)
PyObject *kv_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 8 || !f_compact || !f_compact_ws) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const at::Tensor *t = c.dense(a[0], at::kInt, 2), *ref = c.dense(a[1], at::kInt, 1);
        if (!c.ok) return none();
        const int64_t B = t->size(0), W = t->size(1), P = ref->size(0);
        const at::Tensor *gt = c.optional(a[2], at::kInt, {B, W});
        const at::Tensor *g[3];
        for (int i = 0; i < 3; ++i) g[i] = c.optional(a[3 + i], at::kInt, {P});
        const at::Tensor *gc = c.optional(a[6], at::kInt, {1});
        const at::Tensor *gw = a[7] == Py_None ? nullptr : c.dense(a[7], at::kByte, 1);
        if (!c.here()) return none();
        at::Tensor to = c.output(gt, {B, W}, at::kInt), o[3], co = c.output(gc, {1}, at::kInt);
        for (int i = 0; i < 3; ++i) o[i] = c.output(g[i], {P}, at::kInt);
        const Workspace w(gw, f_compact_ws(i32(P)));
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_compact(ptr<int32_t>(t), ptr<int32_t>(ref), ptr<int32_t>(&to), ptr<int32_t>(&o[0]), ptr<int32_t>(&o[1]),
                              ptr<int32_t>(&o[2]), ptr<int32_t>(&co), i32(B), i32(W), i32(P), w.data, w.bytes, s));
        if (st) return PyLong_FromLong(st);
        PyObject *p[5] = {own_or_new(a[2], to), own_or_new(a[3], o[0]), own_or_new(a[4], o[1]), own_or_new(a[5], o[2]),
                          own_or_new(a[6], co)};
        return tuple_of(p);
    });
}

// (pools, src_pages, dst_pages, count)
PyObject *kv_copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4 || !f_copy_pages || !(PyList_CheckExact(a[0]) || PyTuple_CheckExact(a[0]))) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        const at::Tensor *src = c.dense(a[1], at::kInt, 1);
        if (!c.ok) return none();
        const at::Tensor *dst = c.optional(a[2], at::kInt, {src->size(0)}), *count = c.optional(a[3], at::kInt, {1});
        const Py_ssize_t pools = PySequence_Fast_GET_SIZE(a[0]);
        PyObject **items = PySequence_Fast_ITEMS(a[0]);
        if (!dst || !c.ok || pools == 0 || pools > INT_MAX) return none();
        std::vector<void *> at_(pools);
        int64_t P = 0, bytes = 0;
        for (Py_ssize_t i = 0; i < pools; ++i) {
            if (!THPVariable_Check(items[i])) return none();
            const at::Tensor &t = THPVariable_Unpack(items[i]);
            if (!t.defined() || t.key_set().has(c10::DispatchKey::Python) || !t.is_cuda() || t.dim() < 1 ||
                t.device().index() != c.device || !t.is_contiguous() || t.numel() == 0)
                return none();
            const int64_t each = t.numel() / t.size(0) * (int64_t)t.element_size();
            if (i == 0) P = t.size(0), bytes = each;
            if (t.size(0) != P || each != bytes) return none();
            at_[i] = t.data_ptr();
        }
        if (!c.here()) return none();
        const attn_stream_t s = c.stream();
        int st;
        WITHOUT_GIL(f_copy_pages(at_.data(), (int)pools, (size_t)bytes, ptr<int32_t>(src), ptr<int32_t>(dst), ptr<int32_t>(count),
                                 i32(src->size(0)), i32(P), s));
        return PyLong_FromLong(st);
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
    bool get(Call &c, PyObject *const *a, bool fp4 = false) {
        fp8 = a[0] != Py_None;
        if (fp8 && (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 2 || !number(PyTuple_GET_ITEM(a[0], 0), ks) ||
                    !number(PyTuple_GET_ITEM(a[0], 1), vs)))
            return false;
        const at::ScalarType page = fp8 ? at::kByte : at::kBFloat16;
        q = c.dense(a[1], at::kBFloat16, 3);
        k = c.dense(a[2], page, fp4 ? 3 : 4);
        v = c.dense(a[3], page, fp4 ? 3 : 4);
        table = c.dense(a[4], at::kInt, 2);
        ctx = c.dense(a[5], at::kInt, 1);
        if (!c.ok) return false;
        c.need((fp4 ? k->size(2) == 9 * q->size(2) : k->size(3) == q->size(2)) && v->sizes() == k->sizes() && table->size(0) == q->size(0) &&
               ctx->size(0) == q->size(0));
        B = i32(q->size(0)), H = i32(q->size(1)), d = i32(q->size(2)), Hkv = i32(k->size(1));
        num_pages = i32(k->size(0)), page_size = fp4 ? 16 : i32(k->size(2)), max_pages = i32(table->size(1));
        return c.ok;
    }
};

// (scales, q, k_pages, v_pages, page_table, ctx_lens, scale, softcap, alibi_slopes, key_begin, out, lse, workspace,
//  return_lse)
PyObject *decode_modified(PyObject *const *a, Py_ssize_t n, bool fp4) {
    if (n != 14) return none();
    return guarded([&]() -> PyObject * {
        Call c;
        Paged x;
        double scale, cap;
        if (!x.get(c, a, fp4) || (fp4 && !x.fp8) || !number(a[6], scale, 1.0 / std::sqrt((double)x.d), true) || !number(a[7], cap)) return none();
        const at::Tensor *slopes = c.optional(a[8], at::kFloat, {x.H}), *begin = c.optional(a[9], at::kInt, {x.B});
        const at::Tensor *go = c.optional(a[10], at::kBFloat16, x.q->sizes()), *gl = c.optional(a[11], at::kFloat, {x.B, x.H});
        const at::Tensor *gw = a[12] == Py_None ? nullptr : c.dense(a[12], at::kByte, 1);
        const int want = PyObject_IsTrue(a[13]);
        if (want < 0) return nullptr;
        if (!c.here()) return none();
        at::Tensor o = c.output(go, x.q->sizes(), at::kBFloat16), l;
        if (gl || want) l = c.output(gl, {x.B, x.H}, at::kFloat);
        const Workspace w(gw, (fp4 ? f_decode4_ws : f_decode_ws)(x.B, x.H, x.Hkv, x.d, x.max_pages, x.page_size));
        float *lp = l.defined() ? ptr<float>(&l) : nullptr;
        const attn_stream_t s = c.stream();
        int st;
        if (x.fp8)
            WITHOUT_GIL((fp4 ? f_decode4 : f_decode_fp8)(
                x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), (float)x.ks, (float)x.vs, ptr<int32_t>(x.table),
                ptr<int32_t>(x.ctx), x.page_size, o.data_ptr(), lp, x.B, x.H, x.Hkv, x.d, x.max_pages, x.num_pages, (float)scale,
                (float)cap, ptr<float>(slopes), ptr<int32_t>(begin), w.data, w.bytes, s));
        else
            WITHOUT_GIL(f_decode(x.q->data_ptr(), x.k->data_ptr(), x.v->data_ptr(), ptr<int32_t>(x.table),
                                 ptr<int32_t>(x.ctx), x.page_size, o.data_ptr(), lp, x.B, x.H, x.Hkv, x.d, x.max_pages,
                                 x.num_pages, (float)scale, (float)cap, ptr<float>(slopes), ptr<int32_t>(begin),
                                 w.data, w.bytes, s));
        if (st) return PyLong_FromLong(st);
        return pair(o, l.defined() ? &l : nullptr);
    });
}

PyObject *decode_scoremod(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return f_decode && f_decode_fp8 && f_decode_ws ? decode_modified(a, n, false) : none();
}
PyObject *decode_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return f_decode4 && f_decode4_ws ? decode_modified(a, n, true) : none();
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
    take("paged_kv_append_rope_axes", f_append_axes);
    take("paged_kv_append_rope_axes_fp8", f_append_axes_fp8);
    take("paged_kv_append_fp4", f_append_fp4);
    take("paged_kv_unpack_fp4", f_unpack);
    take("attn_rope_axes", f_rope);
    take("attn_rope_axes_bwd", f_rope_bwd);
    take("paged_attn_decode_fp4", f_decode4);
    take("paged_attn_decode_fp4_workspace_size", f_decode4_ws);
    take("paged_kv_fork", f_fork);
    take("paged_kv_reserve", f_reserve);
    take("paged_kv_reserve_workspace_size", f_reserve_ws);
    take("paged_kv_compact", f_compact);
    take("paged_kv_compact_workspace_size", f_compact_ws);
    take("paged_kv_copy_pages", f_copy_pages);
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
                         FAST(decode_scoremod),           FAST(decode_shared),   FAST(decode_fp4),    FAST(append_fp4),
                         FAST(unpack_fp4),                FAST(rope_axes),       FAST(kv_fork),       FAST(kv_reserve),
                         FAST(kv_compact),                FAST(kv_copy_pages),   {nullptr, nullptr, 0, nullptr}};
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
