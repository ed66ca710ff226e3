// marshal.cpp -- the common case of the binding's calls on queries, keys and
// values, in native code.
//
// A call for one token of a sequence is a few microseconds of kernel; read in
// Python, a dozen arguments take longer than that (a key's norm and rotation
// of eight tokens: 26 us in Python, 6.5 to 9 here).  Each function below takes the
// arguments of the api.py function of its name, and either does the whole call
// (outputs made, launched on the device's current stream) or returns None,
// having done nothing, where an argument is not a contiguous tensor on the current
// CUDA device, of the expected type and shape; api.py then takes it apart itself,
// pitches, other devices and messages included.  An error of the call comes back as its status, an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "s5.h"

namespace {
using at::Tensor;

const at::ScalarType F32 = at::kFloat, BF16 = at::kBFloat16;

// The arguments; `ok` stays true while all are what the common case takes.
struct Reader {
    PyObject *const *args;
    bool ok = true;
    c10::DeviceIndex device = -1;

    const Tensor *tensor(int i) {
        if (!ok || !THPVariable_CheckExact(args[i])) return ok = false, nullptr;
        const Tensor &t = THPVariable_Unpack(args[i]);
        if (!t.is_cuda() || !t.is_contiguous() || t.numel() == 0) return ok = false, nullptr;
        if (device < 0) {
            device = t.get_device();
            if (device != c10::cuda::current_device()) return ok = false, nullptr;   // launches go to that one
        }
        if (t.get_device() != device) return ok = false, nullptr;
        return &t;
    }
    bool none(int i) const { return args[i] == Py_None; }
    // q or v: float32 or bfloat16 of `dims` axes (at least three if 0)
    const Tensor *rows(int i, int dims) {
        const Tensor *t = tensor(i);
        if (ok && ((t->scalar_type() != F32 && t->scalar_type() != BF16) || (dims ? t->dim() != dims : t->dim() < 3))) ok = false;
        return t;
    }
    const Tensor *like(int i, at::ScalarType type, at::IntArrayRef shape) {
        const Tensor *t = tensor(i);
        if (ok && (t->scalar_type() != type || t->sizes() != shape)) ok = false;
        return t;
    }
    const Tensor *maybe(int i, at::ScalarType type, at::IntArrayRef shape) {
        return none(i) ? nullptr : like(i, type, shape);
    }
    const Tensor *bytes(int i) {
        const Tensor *t = tensor(i);
        if (ok && t->scalar_type() != at::kByte) ok = false;
        return t;
    }
    double number(int i) {
        if (PyFloat_Check(args[i])) return PyFloat_AS_DOUBLE(args[i]);
        return ok = false, 0.0;
    }
    int code(int i) {
        if (PyLong_Check(args[i])) return (int)PyLong_AsLong(args[i]);
        return ok = false, 0;
    }
    float scale(int i, int64_t head) { return none(i) ? (float)std::pow((double)head, -0.5) : (float)number(i); }
    s5_stream_t stream() const { return (s5_stream_t)c10::cuda::getCurrentCUDAStream(device).stream(); }
};

s5_dtype dtype(const Tensor &t) { return t.scalar_type() == BF16 ? S5_BF16 : S5_F32; }
Tensor make(at::IntArrayRef shape, const Tensor &like) { return at::empty(shape, like.options()); }
Tensor make(at::IntArrayRef shape, const Tensor &like, at::ScalarType type) { return at::empty(shape, like.options().dtype(type)); }
template <typename T = float> T *data(const Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
bool fits(std::initializer_list<int64_t> sizes) {
    for (int64_t n : sizes)
        if (n > INT32_MAX) return false;
    return true;
}

PyObject *result(s5_status code, const Tensor &t) {
    return code == S5_OK ? THPVariable_Wrap(t) : PyLong_FromLong(code);
}
PyObject *result(s5_status code, const Tensor &a, const Tensor &b) {
    if (code != S5_OK) return PyLong_FromLong(code);
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(b));
    return pair;
}
bool put(PyObject *dict, const char *name, const Tensor &t) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    const bool done = o && PyDict_SetItemString(dict, name, o) == 0;
    Py_XDECREF(o);
    return done;
}

// Every entry takes a fixed number of positional arguments.
#define ENTRY(name, count)                                                            \
    PyObject *name##_call(Reader r);                                                  \
    PyObject *name(PyObject *, PyObject *const *args, Py_ssize_t n) {                 \
        HANDLE_TH_ERRORS                                                              \
        if (n != count) return PyErr_Format(PyExc_TypeError, #name ": %zd arguments", n); \
        return name##_call(Reader{args});                                             \
        END_HANDLE_TH_ERRORS                                                          \
    }                                                                                 \
    PyObject *name##_call(Reader r)

// q, k, v, g, beta, state, scale, o
ENTRY(delta_step, 8) {
    const Tensor *q = r.rows(0, 3), *v = r.rows(2, 3);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = q->size(0), Hk = q->size(1), Dk = q->size(2), Hv = v->size(1), Dv = v->size(2);
    const at::ScalarType type = q->scalar_type();
    const Tensor *k = r.like(1, type, q->sizes());
    const Tensor *g = r.like(3, F32, {B, Hv}), *beta = r.like(4, F32, {B, Hv});
    const Tensor *state = r.like(5, F32, {B, Hv, Dk, Dv}), *given = r.maybe(7, type, v->sizes());
    const float scale = r.scale(6, Dk);
    if (!r.ok || v->scalar_type() != type || v->size(0) != B || !fits({B, Hk, Dk, Hv, Dv})) Py_RETURN_NONE;
    const Tensor o = given ? *given : make(v->sizes(), *v);
    return result(s5_delta_step(q->data_ptr(), k->data_ptr(), v->data_ptr(), dtype(*q), data(g), data(beta), scale, (int)B,
                                (int)Hk, (int)Hv, (int)Dk, (int)Dv, data(state), o.data_ptr(), r.stream()),
                  o);
}

// Sizes of q [B,L,Hk,Dk] and v [B,L,Hv,Dv].
struct Sizes {
    int64_t B, L, Hk, Dk, Hv, Dv;
    Sizes(const Tensor &q, const Tensor &v)
        : B(q.size(0)), L(q.size(1)), Hk(q.size(2)), Dk(q.size(3)), Hv(v.size(2)), Dv(v.size(3)) {}
    bool ok(const Tensor &q, const Tensor &v) const {
        return v.scalar_type() == q.scalar_type() && v.size(0) == B && v.size(1) == L && fits({B, L, Hk, Dk, Hv, Dv});
    }
    size_t workspace(bool backward) const {
        return s5_delta_workspace_size((int)B, (int)L, (int)Hv, (int)Dk, (int)Dv, backward);
    }
};

// q, k, v, g, beta, scale, s0, s_last, o, saved, workspace
ENTRY(delta_forward, 11) {
    const Tensor *q = r.rows(0, 4), *v = r.rows(2, 4);
    if (!r.ok) Py_RETURN_NONE;
    const Sizes n(*q, *v);
    const at::ScalarType type = q->scalar_type();
    const Tensor *k = r.like(1, type, q->sizes());
    const Tensor *g = r.like(3, F32, {n.B, n.L, n.Hv}), *beta = r.like(4, F32, {n.B, n.L, n.Hv});
    const int64_t states[4] = {n.B, n.Hv, n.Dk, n.Dv};
    const float scale = r.scale(5, n.Dk);
    const Tensor *s0 = r.maybe(6, F32, states);
    const bool ends = r.args[7] == Py_True;
    const Tensor *last = ends ? nullptr : r.maybe(7, F32, states);
    const Tensor *given = r.maybe(8, type, v->sizes()), *saved = r.none(9) ? nullptr : r.bytes(9);
    const Tensor *work = r.none(10) ? nullptr : r.bytes(10);
    if (!r.ok || !n.ok(*q, *v)) Py_RETURN_NONE;
    const size_t need = work ? (size_t)work->numel() : n.workspace(false);
    if (need == 0) Py_RETURN_NONE;
    const Tensor o = given ? *given : make(v->sizes(), *v), s = ends ? make(states, *q, F32) : last ? *last : Tensor();
    const Tensor w = work ? *work : make({(int64_t)need}, *q, at::kByte);
    const s5_status code = s5_delta_forward(
        q->data_ptr(), n.Hk * n.Dk, k->data_ptr(), n.Hk * n.Dk, v->data_ptr(), n.Hv * n.Dv, dtype(*q), data(g), data(beta),
        data(s0), scale, (int)n.B, (int)n.L, (int)n.Hk, (int)n.Hv, (int)n.Dk, (int)n.Dv, o.data_ptr(), n.Hv * n.Dv,
        s.defined() ? data(&s) : nullptr, data<void>(saved), saved ? saved->numel() : 0, w.data_ptr(), need, r.stream());
    return s.defined() ? result(code, o, s) : result(code, o);
}

// q, k, v, g, beta, do, saved, scale, s0, ds_last, workspace
ENTRY(delta_backward, 11) {
    const Tensor *q = r.rows(0, 4), *v = r.rows(2, 4);
    if (!r.ok) Py_RETURN_NONE;
    const Sizes n(*q, *v);
    const at::ScalarType type = q->scalar_type();
    const int64_t gates[3] = {n.B, n.L, n.Hv}, states[4] = {n.B, n.Hv, n.Dk, n.Dv};
    const Tensor *k = r.like(1, type, q->sizes()), *g = r.like(3, F32, gates), *beta = r.like(4, F32, gates);
    const Tensor *dout = r.like(5, type, v->sizes()), *saved = r.bytes(6);
    const float scale = r.scale(7, n.Dk);
    const Tensor *s0 = r.maybe(8, F32, states), *last = r.maybe(9, F32, states);
    const Tensor *work = r.none(10) ? nullptr : r.bytes(10);
    if (!r.ok || !n.ok(*q, *v)) Py_RETURN_NONE;
    const size_t need = work ? (size_t)work->numel() : n.workspace(true);
    if (need == 0) Py_RETURN_NONE;
    const Tensor dq = make(q->sizes(), *q), dk = make(q->sizes(), *q), dv = make(v->sizes(), *v);
    const Tensor dg = make(gates, *q, F32), dbeta = make(gates, *q, F32), ds0 = s0 ? make(states, *q, F32) : Tensor();
    const Tensor w = work ? *work : make({(int64_t)need}, *q, at::kByte);
    const s5_status code = s5_delta_backward(
        q->data_ptr(), n.Hk * n.Dk, k->data_ptr(), n.Hk * n.Dk, v->data_ptr(), n.Hv * n.Dv, dtype(*q), data(g), data(beta),
        data(s0), scale, (int)n.B, (int)n.L, (int)n.Hk, (int)n.Hv, (int)n.Dk, (int)n.Dv, dout->data_ptr(), n.Hv * n.Dv,
        data(last), saved->data_ptr(), saved->numel(), dq.data_ptr(), n.Hk * n.Dk, dk.data_ptr(), n.Hk * n.Dk, dv.data_ptr(),
        n.Hv * n.Dv, data(&dg), data(&dbeta), ds0.defined() ? data(&ds0) : nullptr, w.data_ptr(), need, r.stream());
    if (code != S5_OK) return PyLong_FromLong(code);
    PyObject *out = PyDict_New();
    if (out && put(out, "dq", dq) && put(out, "dk", dk) && put(out, "dv", dv) && put(out, "dg", dg) &&
        put(out, "dbeta", dbeta) && put(out, "ds0", ds0))
        return out;
    Py_XDECREF(out);
    return nullptr;
}

// x [..., H, D], its positions [...] and frequencies.
struct Turn {
    const Tensor *positions = nullptr, *freq = nullptr;
    int64_t T = 0, H = 0, D = 0;
    int rot = 0;
    Turn(Reader &r, const Tensor &x, int at) {
        const at::IntArrayRef shape = x.sizes();
        H = shape[shape.size() - 2], D = shape[shape.size() - 1], T = x.numel() / (H * D);
        if (r.none(at + 1)) return;
        positions = r.like(at, at::kLong, shape.slice(0, shape.size() - 2));
        freq = r.tensor(at + 1);
        if (!r.ok || freq->scalar_type() != at::kDouble || freq->dim() != 1 || !fits({H, D, 2 * freq->numel()})) {
            r.ok = false;
            return;
        }
        rot = (int)(2 * freq->numel());
    }
    const long long *pos() const { return data<long long>(positions); }
};

// x, positions, freq, layout, amplitude, inverse, out
ENTRY(rotary, 7) {
    const Tensor *x = r.rows(0, 0);
    if (!r.ok) Py_RETURN_NONE;
    const Turn t(r, *x, 1);
    const int layout = r.code(3), inverse = r.code(5);
    const double amplitude = r.number(4);
    const Tensor *given = r.maybe(6, x->scalar_type(), x->sizes());
    if (!r.ok) Py_RETURN_NONE;
    const Tensor out = given ? *given : make(x->sizes(), *x);
    const long long ld = t.H * t.D;
    return result(s5_rotary(x->data_ptr(), ld, dtype(*x), t.pos(), data<double>(t.freq), t.rot, (s5_rotary_layout)layout,
                            (float)amplitude, inverse, t.T, (int)t.H, (int)t.D, out.data_ptr(), ld, r.stream()),
                  out);
}

// q, k, positions, freq, norm, eps, q_weight, k_weight, layout, amplitude, q_out, k_out
ENTRY(qk_norm_rotary, 12) {
    const Tensor *q = r.rows(0, 0), *k = r.rows(1, 0);
    if (!r.ok || k->dim() != q->dim()) Py_RETURN_NONE;
    const Turn t(r, *q, 2);
    const at::ScalarType type = q->scalar_type();
    const int64_t Hk = k->size(-2), tokens = q->dim() - 2;
    const int norm = r.code(4), layout = r.code(8);
    const double eps = r.number(5), amplitude = r.number(9);
    const Tensor *wq = r.maybe(6, F32, {t.D}), *wk = r.maybe(7, F32, {t.D});
    const Tensor *gq = r.maybe(10, type, q->sizes()), *gk = r.maybe(11, type, k->sizes());
    if (!r.ok || k->scalar_type() != type || k->size(-1) != t.D || !fits({Hk}) ||
        k->sizes().slice(0, tokens) != q->sizes().slice(0, tokens))
        Py_RETURN_NONE;
    const Tensor qo = gq ? *gq : make(q->sizes(), *q), ko = gk ? *gk : make(k->sizes(), *k);
    const long long lq = t.H * t.D, lk = Hk * t.D;
    return result(s5_qk_norm_rotary(q->data_ptr(), lq, k->data_ptr(), lk, dtype(*q), data(wq), data(wk), (s5_norm)norm,
                                    (float)eps, t.pos(), data<double>(t.freq), t.rot, (s5_rotary_layout)layout,
                                    (float)amplitude, t.T, (int)t.H, (int)Hk, (int)t.D, qo.data_ptr(), lq, ko.data_ptr(), lk,
                                    r.stream()),
                  qo, ko);
}

// q, k, dq_out, dk_out, positions, freq, norm, eps, q_weight, k_weight, layout, amplitude, workspace
ENTRY(qk_norm_rotary_backward, 13) {
    const Tensor *q = r.rows(0, 0), *k = r.rows(1, 0);
    if (!r.ok || k->dim() != q->dim()) Py_RETURN_NONE;
    const Turn t(r, *q, 4);
    const at::ScalarType type = q->scalar_type();
    const int64_t Hk = k->size(-2), tokens = q->dim() - 2;
    const Tensor *gq = r.like(2, type, q->sizes()), *gk = r.like(3, type, k->sizes());
    const int norm = r.code(6), layout = r.code(10);
    const double eps = r.number(7), amplitude = r.number(11);
    const Tensor *wq = r.maybe(8, F32, {t.D}), *wk = r.maybe(9, F32, {t.D});
    const Tensor *work = r.none(12) ? nullptr : r.bytes(12);
    if (!r.ok || k->scalar_type() != type || k->size(-1) != t.D || !fits({Hk}) ||
        k->sizes().slice(0, tokens) != q->sizes().slice(0, tokens))
        Py_RETURN_NONE;
    const bool weights = wq || wk;
    const size_t need = work ? (size_t)work->numel() : weights ? s5_qk_norm_rotary_workspace_size((int)t.D) : 0;
    if (weights && need == 0) Py_RETURN_NONE;
    const Tensor dq = make(q->sizes(), *q), dk = make(k->sizes(), *k);
    const Tensor dwq = wq ? make({t.D}, *q, F32) : Tensor(), dwk = wk ? make({t.D}, *q, F32) : Tensor();
    const Tensor w = work ? *work : weights ? make({(int64_t)need}, *q, at::kByte) : Tensor();
    const long long lq = t.H * t.D, lk = Hk * t.D;
    const s5_status code = s5_qk_norm_rotary_backward(
        q->data_ptr(), lq, k->data_ptr(), lk, dtype(*q), data(wq), data(wk), (s5_norm)norm, (float)eps, t.pos(),
        data<double>(t.freq), t.rot, (s5_rotary_layout)layout, (float)amplitude, t.T, (int)t.H, (int)Hk, (int)t.D,
        gq->data_ptr(), lq, gk->data_ptr(), lk, dq.data_ptr(), lq, dk.data_ptr(), lk, dwq.defined() ? data(&dwq) : nullptr,
        dwk.defined() ? data(&dwk) : nullptr, w.defined() ? w.data_ptr() : nullptr, need, r.stream());
    if (code != S5_OK) return PyLong_FromLong(code);
    PyObject *out = PyDict_New();
    if (out && put(out, "dq", dq) && put(out, "dk", dk) && put(out, "dwq", dwq) && put(out, "dwk", dwk)) return out;
    Py_XDECREF(out);
    return nullptr;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(delta_step), METHOD(delta_forward), METHOD(delta_backward), METHOD(rotary),
                         METHOD(qk_norm_rotary), METHOD(qk_norm_rotary_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "The common case of the binding's calls.", -1, methods};
}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
