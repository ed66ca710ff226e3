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

#include <ATen/Context.h>
#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDACachingAllocator.h>
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
    int bare = -1;                       // whether memory is all that a new array takes; -1: not asked yet

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
    // at::empty on the current CUDA device, which is `like`'s.  Its way there takes as long as a small kernel, so it is
    // called only where something on that way would do more than allocate: a dispatch mode, a transform or a tracer, which
    // add a dispatch key of theirs; an observer of operators, as a profiler; filling of what is not written yet.
    Tensor make(at::IntArrayRef shape, const Tensor &like, at::ScalarType type) {
        if (bare < 0)
            bare = (c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() &&
                   !at::getStepCallbacksUnlessEmpty(at::RecordScope::FUNCTION).has_value() && !at::globalContext().deterministicAlgorithms();
        if (!bare) return at::empty(shape, like.options().dtype(type));
        return Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                type, std::nullopt));
    }
    Tensor make(at::IntArrayRef shape, const Tensor &like) { return make(shape, like, like.scalar_type()); }
    s5_stream_t stream() const { return (s5_stream_t)c10::cuda::getCurrentCUDAStream(device).stream(); }
};

s5_dtype dtype(const Tensor &t) { return t.scalar_type() == BF16 ? S5_BF16 : S5_F32; }
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
    const Tensor o = given ? *given : r.make(v->sizes(), *v);
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
    const Tensor o = given ? *given : r.make(v->sizes(), *v), s = ends ? r.make(states, *q, F32) : last ? *last : Tensor();
    const Tensor w = work ? *work : r.make({(int64_t)need}, *q, at::kByte);
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
    const Tensor dq = r.make(q->sizes(), *q), dk = r.make(q->sizes(), *q), dv = r.make(v->sizes(), *v);
    const Tensor dg = r.make(gates, *q, F32), dbeta = r.make(gates, *q, F32), ds0 = s0 ? r.make(states, *q, F32) : Tensor();
    const Tensor w = work ? *work : r.make({(int64_t)need}, *q, at::kByte);
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
    const Tensor out = given ? *given : r.make(x->sizes(), *x);
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
    const Tensor qo = gq ? *gq : r.make(q->sizes(), *q), ko = gk ? *gk : r.make(k->sizes(), *k);
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
    const Tensor dq = r.make(q->sizes(), *q), dk = r.make(k->sizes(), *k);
    const Tensor dwq = wq ? r.make({t.D}, *q, F32) : Tensor(), dwk = wk ? r.make({t.D}, *q, F32) : Tensor();
    const Tensor w = work ? *work : weights ? r.make({(int64_t)need}, *q, at::kByte) : Tensor();
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

// ------------------------------------------------------------------ gated recurrence, short convolution, layer norm
struct Marks {
    const Tensor *reset = nullptr, *lengths = nullptr;
    Marks(Reader &r, int at, int64_t B, int64_t L) {
        if (!r.none(at)) {
            reset = r.tensor(at);
            if (r.ok && ((reset->scalar_type() != at::kBool && reset->scalar_type() != at::kByte) || reset->sizes() != at::IntArrayRef({B, L})))
                r.ok = false;
        }
        lengths = r.maybe(at + 1, at::kInt, {B});
    }
    const unsigned char *bytes() const { return data<unsigned char>(reset); }
    const int *ints() const { return data<int>(lengths); }
};
bool flag(Reader &r, int i) {
    if (r.args[i] != Py_True && r.args[i] != Py_False) r.ok = false;
    return r.args[i] == Py_True;
}
const Tensor *channels(Reader &r, int i, int dims) {
    const Tensor *t = r.tensor(i);
    if (r.ok && ((t->scalar_type() != F32 && t->scalar_type() != BF16) || (dims ? t->dim() != dims : t->dim() < 1))) r.ok = false;
    return t;
}
Tensor given_or(Reader &r, const Tensor *t, const Tensor &like) { return t ? *t : r.make(like.sizes(), like); }
template <typename T = float> T *at_or_null(const Tensor &t) { return t.defined() ? data<T>(&t) : nullptr; }

// x: the buffer that the forward call fills
ENTRY(gated_scan_saved, 1) {
    const Tensor *x = channels(r, 0, 3);
    if (!r.ok || !fits({x->size(0), x->size(1), x->size(2)})) Py_RETURN_NONE;
    const size_t n = s5_gated_scan_saved_size((int)x->size(0), (int)x->size(1), (int)x->size(2));
    if (n == 0) Py_RETURN_NONE;
    return THPVariable_Wrap(r.make({(int64_t)n}, *x, at::kByte));
}
ENTRY(layernorm_saved, 1) {
    const Tensor *x = channels(r, 0, 0);
    if (!r.ok) Py_RETURN_NONE;
    return THPVariable_Wrap(r.make({x->numel() / x->size(-1), 2}, *x, F32));
}

// x, gate_a, gate_x, rate, h0, h_last, reset, lengths, normalize, h, saved
ENTRY(gated_scan_forward, 11) {
    const Tensor *x = channels(r, 0, 3);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = x->size(0), L = x->size(1), C = x->size(2);
    const at::ScalarType type = x->scalar_type();
    const Tensor *ga = r.like(1, type, x->sizes()), *gx = r.maybe(2, type, x->sizes()), *rate = r.like(3, F32, {C});
    const Tensor *h0 = r.maybe(4, F32, {B, C});
    const bool ends = r.args[5] == Py_True;
    const Tensor *last = ends ? nullptr : r.maybe(5, F32, {B, C});
    const Marks m(r, 6, B, L);
    const bool normalize = flag(r, 8);
    const Tensor *given = r.maybe(9, type, x->sizes()), *saved = r.none(10) ? nullptr : r.bytes(10);
    if (!r.ok || !fits({B, L, C})) Py_RETURN_NONE;
    const Tensor h = given_or(r, given, *x), s = ends ? r.make({B, C}, *x, F32) : last ? *last : Tensor();
    const s5_status code =
        s5_gated_scan_forward(x->data_ptr(), C, ga->data_ptr(), C, data<void>(gx), C, dtype(*x), data(rate), data(h0), m.bytes(),
                              m.ints(), normalize, (int)B, (int)L, (int)C, h.data_ptr(), C, at_or_null(s), data<void>(saved),
                              saved ? saved->numel() : 0, r.stream());
    return s.defined() ? result(code, h, s) : result(code, h);
}

// x, gate_a, gate_x, rate, dh, saved, h0, dh_last, reset, lengths, normalize, workspace
ENTRY(gated_scan_backward, 12) {
    const Tensor *x = channels(r, 0, 3);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = x->size(0), L = x->size(1), C = x->size(2);
    const at::ScalarType type = x->scalar_type();
    const Tensor *ga = r.like(1, type, x->sizes()), *gx = r.maybe(2, type, x->sizes()), *rate = r.like(3, F32, {C});
    const Tensor *dh = r.like(4, type, x->sizes()), *saved = r.bytes(5);
    const Tensor *h0 = r.maybe(6, F32, {B, C}), *last = r.maybe(7, F32, {B, C});
    const Marks m(r, 8, B, L);
    const bool normalize = flag(r, 10);
    const Tensor *work = r.none(11) ? nullptr : r.bytes(11);
    if (!r.ok || !fits({B, L, C})) Py_RETURN_NONE;
    const size_t need = work ? (size_t)work->numel() : s5_gated_scan_workspace_size((int)B, (int)L, (int)C);
    if (need == 0) Py_RETURN_NONE;
    const Tensor dx = r.make(x->sizes(), *x), dga = r.make(x->sizes(), *x), dgx = gx ? r.make(x->sizes(), *x) : Tensor();
    const Tensor drate = r.make({C}, *x, F32), dh0 = h0 ? r.make({B, C}, *x, F32) : Tensor();
    const Tensor w = work ? *work : r.make({(int64_t)need}, *x, at::kByte);
    const s5_status code = s5_gated_scan_backward(
        x->data_ptr(), C, ga->data_ptr(), C, data<void>(gx), C, dtype(*x), data(rate), m.bytes(), m.ints(), normalize, (int)B, (int)L,
        (int)C, dh->data_ptr(), C, data(last), saved->data_ptr(), saved->numel(), dx.data_ptr(), C, dga.data_ptr(), C,
        at_or_null<void>(dgx), C, data(&drate), at_or_null(dh0), w.data_ptr(), need, r.stream());
    if (code != S5_OK) return PyLong_FromLong(code);
    PyObject *out = PyDict_New();
    if (out && put(out, "dx", dx) && put(out, "dgate_a", dga) && put(out, "dgate_x", dgx) && put(out, "drate", drate) &&
        put(out, "dh0", dh0))
        return out;
    Py_XDECREF(out);
    return nullptr;
}

// x, gate_a, gate_x, rate, state, normalize, h
ENTRY(gated_scan_step, 7) {
    const Tensor *x = channels(r, 0, 2);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = x->size(0), C = x->size(1);
    const at::ScalarType type = x->scalar_type();
    const Tensor *ga = r.like(1, type, x->sizes()), *gx = r.maybe(2, type, x->sizes()), *rate = r.like(3, F32, {C});
    const Tensor *state = r.like(4, F32, x->sizes());
    const bool normalize = flag(r, 5);
    const Tensor *given = r.maybe(6, type, x->sizes());
    if (!r.ok || !fits({B, C})) Py_RETURN_NONE;
    const Tensor h = given_or(r, given, *x);
    return result(s5_gated_scan_step(x->data_ptr(), ga->data_ptr(), data<void>(gx), dtype(*x), data(rate), normalize, (int)B, (int)C,
                                     data(state), h.data_ptr(), r.stream()),
                  h);
}

// The weight [C,K] of x's channels; its taps.
int64_t taps(Reader &r, int i, int64_t C) {
    const Tensor *w = r.tensor(i);
    if (r.ok && (w->scalar_type() != F32 || w->dim() != 2 || w->size(0) != C || w->size(1) < 2)) r.ok = false;
    return r.ok ? w->size(1) : 0;
}

// x, weight, bias, activation, past, past_out, reset, lengths, y
ENTRY(short_conv_forward, 9) {
    const Tensor *x = channels(r, 0, 3);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = x->size(0), L = x->size(1), C = x->size(2), K = taps(r, 1, C);
    const at::ScalarType type = x->scalar_type();
    const Tensor *w = r.tensor(1), *bias = r.maybe(2, F32, {C});
    const int act = r.code(3);
    const Tensor *past = r.maybe(4, type, {B, K - 1, C});
    const bool ends = r.args[5] == Py_True;
    const Tensor *last = ends ? nullptr : r.maybe(5, type, {B, K - 1, C});
    const Marks m(r, 6, B, L);
    const Tensor *given = r.maybe(8, type, x->sizes());
    if (!r.ok || !fits({B, L, C, K})) Py_RETURN_NONE;
    const Tensor y = given_or(r, given, *x), s = ends ? r.make({B, K - 1, C}, *x) : last ? *last : Tensor();
    const s5_status code = s5_short_conv_forward(x->data_ptr(), C, dtype(*x), data(w), data(bias), (s5_activation)act, data<void>(past),
                                                 m.bytes(), m.ints(), (int)B, (int)L, (int)C, (int)K, y.data_ptr(), C,
                                                 at_or_null<void>(s), r.stream());
    return s.defined() ? result(code, y, s) : result(code, y);
}

// x, weight, dy, bias, activation, past, dpast_out, reset, lengths, workspace
ENTRY(short_conv_backward, 10) {
    const Tensor *x = channels(r, 0, 3);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = x->size(0), L = x->size(1), C = x->size(2), K = taps(r, 1, C);
    const at::ScalarType type = x->scalar_type();
    const Tensor *w = r.tensor(1), *dy = r.like(2, type, x->sizes()), *bias = r.maybe(3, F32, {C});
    const int act = r.code(4);
    const Tensor *past = r.maybe(5, type, {B, K - 1, C}), *last = r.maybe(6, type, {B, K - 1, C});
    const Marks m(r, 7, B, L);
    const Tensor *work = r.none(9) ? nullptr : r.bytes(9);
    if (!r.ok || !fits({B, L, C, K})) Py_RETURN_NONE;
    const size_t need = work ? (size_t)work->numel() : s5_short_conv_workspace_size((int)C, (int)K);
    if (need == 0) Py_RETURN_NONE;
    const Tensor dx = r.make(x->sizes(), *x), dw = r.make({C, K}, *x, F32), db = bias ? r.make({C}, *x, F32) : Tensor();
    const Tensor dpast = past ? r.make({B, K - 1, C}, *x) : Tensor();
    const Tensor ws = work ? *work : r.make({(int64_t)need}, *x, at::kByte);
    const s5_status code = s5_short_conv_backward(
        x->data_ptr(), C, dtype(*x), data(w), data(bias), (s5_activation)act, data<void>(past), m.bytes(), m.ints(), (int)B, (int)L,
        (int)C, (int)K, dy->data_ptr(), C, data<void>(last), dx.data_ptr(), C, data(&dw), at_or_null(db), at_or_null<void>(dpast),
        ws.data_ptr(), need, r.stream());
    if (code != S5_OK) return PyLong_FromLong(code);
    PyObject *out = PyDict_New();
    if (out && put(out, "dx", dx) && put(out, "dweight", dw) && put(out, "dbias", db) && put(out, "dpast", dpast)) return out;
    Py_XDECREF(out);
    return nullptr;
}

// x, weight, state, bias, activation, y
ENTRY(short_conv_step, 6) {
    const Tensor *x = channels(r, 0, 2);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t B = x->size(0), C = x->size(1), K = taps(r, 1, C);
    const at::ScalarType type = x->scalar_type();
    const Tensor *w = r.tensor(1), *state = r.like(2, type, {B, K - 1, C}), *bias = r.maybe(3, F32, {C});
    const int act = r.code(4);
    const Tensor *given = r.maybe(5, type, x->sizes());
    if (!r.ok || !fits({B, C, K})) Py_RETURN_NONE;
    const Tensor y = given_or(r, given, *x);
    return result(s5_short_conv_step(x->data_ptr(), dtype(*x), data(w), data(bias), (s5_activation)act, (int)B, (int)C, (int)K,
                                     state->data_ptr(), y.data_ptr(), r.stream()),
                  y);
}

// x, weight, bias, residual, eps, y, total, saved
ENTRY(add_layernorm, 8) {
    const Tensor *x = channels(r, 0, 0);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t H = x->size(-1), N = x->numel() / H;
    const at::ScalarType type = x->scalar_type();
    const Tensor *w = r.maybe(1, F32, {H}), *bias = r.maybe(2, F32, {H}), *residual = r.maybe(3, type, x->sizes());
    const double eps = r.number(4);
    const Tensor *gy = r.maybe(5, type, x->sizes()), *gt = r.maybe(6, type, x->sizes()), *saved = r.maybe(7, F32, {N, 2});
    if (!r.ok || !fits({H}) || (gt && !residual)) Py_RETURN_NONE;
    const Tensor y = given_or(r, gy, *x), total = residual ? given_or(r, gt, *x) : Tensor();
    const s5_status code =
        s5_add_layernorm(x->data_ptr(), H, data<void>(residual), H, dtype(*x), data(w), data(bias), (float)eps, N, (int)H, y.data_ptr(),
                         H, at_or_null<void>(total), H, data(saved), r.stream());
    return residual ? result(code, y, total) : result(code, y);
}

// x, dy, saved, weight, bias, residual, dtotal, workspace
ENTRY(add_layernorm_backward, 8) {
    const Tensor *x = channels(r, 0, 0);
    if (!r.ok) Py_RETURN_NONE;
    const int64_t H = x->size(-1), N = x->numel() / H;
    const at::ScalarType type = x->scalar_type();
    const Tensor *dy = r.like(1, type, x->sizes()), *saved = r.like(2, F32, {N, 2});
    const Tensor *w = r.maybe(3, F32, {H}), *bias = r.maybe(4, F32, {H});
    const Tensor *residual = r.maybe(5, type, x->sizes()), *dt = r.maybe(6, type, x->sizes());
    const Tensor *work = r.none(7) ? nullptr : r.bytes(7);
    if (!r.ok || !fits({H})) Py_RETURN_NONE;
    const size_t need = work ? (size_t)work->numel() : w || bias ? s5_add_layernorm_workspace_size((int)H) : 0;
    if ((w || bias) && need == 0) Py_RETURN_NONE;
    const Tensor dx = r.make(x->sizes(), *x), dw = w ? r.make({H}, *x, F32) : Tensor(), db = bias ? r.make({H}, *x, F32) : Tensor();
    const Tensor ws = work ? *work : need ? r.make({(int64_t)need}, *x, at::kByte) : Tensor();
    const s5_status code = s5_add_layernorm_backward(x->data_ptr(), H, data<void>(residual), H, dy->data_ptr(), H, data<void>(dt), H,
                                                     dtype(*x), data(w), data(saved), N, (int)H, dx.data_ptr(), H, at_or_null(dw),
                                                     at_or_null(db), at_or_null<void>(ws), need, r.stream());
    if (code != S5_OK) return PyLong_FromLong(code);
    PyObject *out = PyDict_New();
    if (out && put(out, "dx", dx) && put(out, "dweight", dw) && put(out, "dbias", db)) return out;
    Py_XDECREF(out);
    return nullptr;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(delta_step), METHOD(delta_forward), METHOD(delta_backward), METHOD(rotary),
                         METHOD(qk_norm_rotary), METHOD(qk_norm_rotary_backward),
                         METHOD(gated_scan_forward), METHOD(gated_scan_backward), METHOD(gated_scan_step),
                         METHOD(short_conv_forward), METHOD(short_conv_backward), METHOD(short_conv_step),
                         METHOD(add_layernorm), METHOD(add_layernorm_backward),
                         METHOD(gated_scan_saved), METHOD(layernorm_saved), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "The common case of the binding's calls.", -1, methods};
}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
