// binding.cpp -- the torch side of the causal mixer's and beam search's entry
// points and of those beside them (causal.py, beam.py, gated.py, norm.py and loss.py
// hold their names, defaults and documentation):
// checks of the arguments, allocation of the outputs and the call of the C
// ABI. A single-token call's kernels take 2 to 6 us; checked argument by
// argument in Python such a call cost the host 9 us.
//
// Every function takes its arguments by position, as Python's wrappers pass
// them. TypeError and ValueError name the argument; a negative status raises
// ScanError through the callable given to bind(). The library's functions come
// in by address, so this module does not depend on where it was loaded from.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include <cstdarg>
#include <initializer_list>
#include <memory>
#include <string>
#include <unordered_set>
#include <vector>

#include "vimscan.h"

namespace {

#define VS_BOUND(X)                                                                                   \
    X(s6_workspace_bytes) X(s6_causal_conv) X(s6_causal_conv_grad) X(s6_conv_step) X(s6_causal_scan)  \
    X(s6_causal_scan_saved) X(s6_causal_scan_grad) X(s6_scan_step) X(beam_workspace_bytes)            \
    X(beam_select) X(beam_reorder)                                                                    \
    X(gated_workspace_bytes) X(gated_scan) X(gated_scan_saved) X(gated_scan_grad) X(gated_scan_step)   \
    X(norm_workspace_bytes) X(rms_norm) X(rms_norm_grad)                                              \
    X(vocab_workspace_bytes) X(vocab_loss) X(vocab_loss_grad)

struct Abi {
#define VS_MEMBER(f) decltype(&::f) f;
    VS_BOUND(VS_MEMBER)
#undef VS_MEMBER
} abi;
PyObject* check_status;              // _native.check(name, code)

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
    va_list v;
    va_start(v, format);
    PyErr_FormatV(type, format, v);
    va_end(v);
    throw python_error();
}

using Dims = std::initializer_list<int64_t>;
using Maybe = const at::Tensor*;     // NULL: None

std::string shape(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + (v.size() == 1 ? ",)" : ")");
}
PyObject* dtype_name(at::ScalarType t) { return reinterpret_cast<PyObject*>(torch::getTHPDtype(t)); }

Maybe maybe(const char* name, PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}
const at::Tensor& need(const char* name, PyObject* o) {
    Maybe t = maybe(name, o);
    if (!t) raise(PyExc_ValueError, "%s is required", name);
    return *t;
}
bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}

float number(const char* name, PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        raise(PyExc_TypeError, "%s must be a number, not %s", name, Py_TYPE(o)->tp_name);
    }
    return static_cast<float>(v);
}

void axes(const char* name, const at::Tensor& t, int64_t n) {
    if (t.dim() != n) raise(PyExc_ValueError, "%s must have %d axes, got shape %s", name, static_cast<int>(n), shape(t.sizes()).c_str());
}

// The caller's tensors that a call writes in place: the pools, and whatever was
// given for an output, a buffer or a state to reorder. The write is no part of
// a graph, so none of them may require a gradient while gradients are recorded;
// and after the call each gets a new version, so that a backward pass that
// saved its former values is refused. Inference tensors have no version, and
// nothing can save them.
class Written {
    const at::Tensor* t[4];
    int n = 0;

public:
    void add(const char* name, Maybe v) {
        if (!v) return;
        if (v->requires_grad() && at::GradMode::is_enabled())
            raise(PyExc_ValueError, "%s is written in place, but requires a gradient: detach it, or call under torch.no_grad()", name);
        t[n++] = v;
    }
    void changed() const {
        for (int i = 0; i < n; ++i)
            if (!t[i]->is_inference()) t[i]->unsafeGetTensorImpl()->bump_version();
    }
};

// dtype and device of a call, from its first argument
struct Call {
    at::ScalarType dt;
    at::Device dev;
    int dtype;                       // the ABI's
    mutable Written written;

    Call(const char* name, const at::Tensor& t, int64_t ndim) : dt(t.scalar_type()), dev(t.device()) {
        if (dt != at::kFloat && dt != at::kBFloat16) raise(PyExc_TypeError, "unsupported dtype %S", dtype_name(dt));
        axes(name, t, ndim);
        if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be on the GPU", name);
        dtype = dt == at::kBFloat16 ? VS_BF16 : VS_F32;
    }
    void* stream() const { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }
    void expect(const char* name, const at::Tensor& t, Dims dims, at::ScalarType want) const {
        if (t.scalar_type() != want)
            raise(PyExc_TypeError, "%s has dtype %S, expected %S", name, dtype_name(t.scalar_type()), dtype_name(want));
        if (t.sizes() != at::IntArrayRef(dims.begin(), dims.size()))
            raise(PyExc_ValueError, "%s has shape %s, expected %s", name, shape(t.sizes()).c_str(),
                  shape(at::IntArrayRef(dims.begin(), dims.size())).c_str());
        if (t.device() != dev)
            raise(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
    }
    // a contiguous tensor's memory, or NULL
    void* dense(const char* name, Maybe t, Dims dims, at::ScalarType want) const {
        if (!t) return nullptr;
        expect(name, *t, dims, want);
        if (!t->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
        return t->data_ptr();
    }
    template <typename T>
    T* dense(const char* name, Maybe t, Dims dims) const {
        return static_cast<T*>(dense(name, t, dims, std::is_same_v<T, float> ? at::kFloat : at::kInt));
    }
    // an activation's: contiguous along its last axis, other strides free
    const void* input(const char* name, Maybe t, Dims dims) const {
        if (!t) return nullptr;
        expect(name, *t, dims, dt);
        if (t->size(-1) > 1 && t->stride(-1) != 1) raise(PyExc_ValueError, "%s must be contiguous along its last axis", name);
        return t->data_ptr();
    }
    at::Tensor fresh(Dims dims, at::ScalarType type) const {
        return at::empty(at::IntArrayRef(dims.begin(), dims.size()), at::TensorOptions().dtype(type).device(dev));
    }
    // a given output, or a new one
    at::Tensor out(const char* name, PyObject* given, Dims dims, at::ScalarType type) const {
        Maybe t = maybe(name, given);
        if (!t) return fresh(dims, type);
        dense(name, t, dims, type);
        written.add(name, t);
        return *t;
    }
};

// the batch and channel strides of a call's activations; NULL when all are contiguous
struct Strides {
    int64_t v[12];
    const int64_t* p;
    explicit Strides(std::initializer_list<Maybe> ts) : p(nullptr) {
        for (Maybe t : ts)
            if (t && !t->is_contiguous()) p = v;
        int64_t* o = v;
        if (p)
            for (Maybe t : ts) {
                *o++ = t ? t->stride(0) : 0;
                *o++ = t ? t->stride(1) : 0;
            }
    }
};

// a workspace or saved buffer of at least `need` bytes: the given one (which the call writes, or only reads) or a new one
struct Buffer {
    at::Tensor t;
    void* p = nullptr;
    size_t bytes;
    Buffer(const char* name, size_t need, const Call& c, PyObject* given, bool writes = true) : bytes(need) {
        if (Maybe g = maybe(name, given)) {
            bytes = static_cast<size_t>(g->numel()) * g->element_size();
            if (bytes < need || !g->is_contiguous() || g->device() != c.dev)
                raise(PyExc_ValueError, "%s needs %zu contiguous bytes on %s", name, need, c.dev.str().c_str());
            if (writes) c.written.add(name, g);
            t = *g;
        } else if (need > 0) {
            t = c.fresh({static_cast<int64_t>(need)}, at::kByte);
        }
        if (t.defined()) p = t.data_ptr();
    }
};

// the call itself, on the tensors' device and without the interpreter's lock; a status becomes an exception
template <typename F>
void run(const char* name, const at::Device& dev, const Written& written, F&& f) {
    c10::OptionalDeviceGuard guard;
    if (c10::hip::current_device() != dev.index()) guard.reset_device(dev);
    int code;
    Py_BEGIN_ALLOW_THREADS
    code = f();
    Py_END_ALLOW_THREADS
    if (code == 0) return written.changed();
    PyObject* r = PyObject_CallFunction(check_status, "si", name, code);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed (%d)", name, code);
    throw python_error();
}

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}
struct Named { const char* name; at::Tensor t; };
PyObject* dict(std::initializer_list<Named> ts) {
    PyObject* r = PyDict_New();
    if (!r) throw python_error();
    for (const Named& n : ts) {
        PyObject* v = wrap(n.t);
        PyDict_SetItemString(r, n.name, v);
        Py_XDECREF(v);
    }
    return r;
}
void* at_or_null(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* f32(const at::Tensor& t) { return static_cast<float*>(at_or_null(t)); }

// ------------------------------------------------------------- convolution
// x, w, bias, window, lengths, silu, out, window_out
PyObject* conv(PyObject* const* a) {
    const at::Tensor& x = need("x", a[0]);
    const Call c("x", x, 3);
    const int64_t batch = x.size(0), dim = x.size(1), L = x.size(2);
    const at::Tensor& w = need("w", a[1]);
    axes("w", w, 2);
    const int64_t width = w.size(1);
    const void* xp = c.input("x", &x, {batch, dim, L});
    const float* wp = c.dense<float>("w", &w, {dim, width});
    const float* bp = c.dense<float>("bias", maybe("bias", a[2]), {dim});
    const void* win = c.dense("window", maybe("window", a[3]), {batch, dim, width - 1}, c.dt);
    const int32_t* len = c.dense<int32_t>("lengths", maybe("lengths", a[4]), {batch});
    const at::Tensor y = c.out("out", a[6], {batch, dim, L}, c.dt);
    const at::Tensor wo = c.out("window_out", a[7], {batch, dim, width - 1}, c.dt);
    const Strides st({&x});
    const int flags = truth(a[5]) ? VS_CONV_SILU : 0;
    run("s6_causal_conv", c.dev, c.written, [&] {
        return abi.s6_causal_conv(batch, dim, width, L, c.dtype, flags, xp, st.p, wp, bp, win, len, y.data_ptr(), wo.data_ptr(), c.stream());
    });
    return tuple({y, wo});
}

// x, w, bias, dy, window, dwindow, lengths, silu, workspace
PyObject* conv_grad(PyObject* const* a) {
    const at::Tensor &x = need("x", a[0]), &dy = need("dy", a[3]);
    const Call c("x", x, 3);
    const int64_t batch = x.size(0), dim = x.size(1), L = x.size(2);
    const at::Tensor& w = need("w", a[1]);
    axes("w", w, 2);
    const int64_t width = w.size(1);
    const void *xp = c.input("x", &x, {batch, dim, L}), *dyp = c.input("dy", &dy, {batch, dim, L});
    const float* wp = c.dense<float>("w", &w, {dim, width});
    const float* bp = c.dense<float>("bias", maybe("bias", a[2]), {dim});
    const void* win = c.dense("window", maybe("window", a[4]), {batch, dim, width - 1}, c.dt);
    const void* dwo = c.dense("dwindow", maybe("dwindow", a[5]), {batch, dim, width - 1}, c.dt);
    const int32_t* len = c.dense<int32_t>("lengths", maybe("lengths", a[6]), {batch});
    const Buffer ws("workspace", abi.s6_workspace_bytes(VS_S6_CONV_GRAD, batch, dim, width, L), c, a[8]);
    const at::Tensor dx = c.fresh({batch, dim, L}, c.dt), dw = c.fresh({dim, width}, at::kFloat), db = c.fresh({dim}, at::kFloat);
    at::Tensor dwin;
    if (win) dwin = c.fresh({batch, dim, width - 1}, c.dt);
    const Strides st({&x, &dy});
    const int flags = truth(a[7]) ? VS_CONV_SILU : 0;
    run("s6_causal_conv_grad", c.dev, c.written, [&] {
        return abi.s6_causal_conv_grad(batch, dim, width, L, c.dtype, flags, xp, dyp, st.p, wp, bp, win, len, dwo, dx.data_ptr(),
                                       f32(dw), f32(db), at_or_null(dwin), ws.p, ws.bytes, c.stream());
    });
    return dict({{"dx", dx}, {"dw", dw}, {"dbias", db}, {"dwindow", dwin}});
}

// x, w, bias, window, slot_in, slot_out, silu, out
PyObject* conv_step(PyObject* const* a) {
    at::Tensor x = need("x", a[0]);
    const Call c("x", x, 2);
    const int64_t batch = x.size(0), dim = x.size(1);
    const at::Tensor &w = need("w", a[1]), &window = need("window", a[3]);
    axes("w", w, 2);
    axes("window", window, 3);
    const int64_t width = w.size(1), slots = window.size(0);
    c.input("x", &x, {batch, dim});
    if (batch > 1 && x.stride(0) == 0) x = x.contiguous();   // one row for all: the ABI's stride 0 means dense rows
    const float* wp = c.dense<float>("w", &w, {dim, width});
    const float* bp = c.dense<float>("bias", maybe("bias", a[2]), {dim});
    void* pool = c.dense("window", &window, {slots, dim, width - 1}, c.dt);
    c.written.add("window", &window);
    const int32_t* si = c.dense<int32_t>("slot_in", maybe("slot_in", a[4]), {batch});
    const int32_t* so = c.dense<int32_t>("slot_out", maybe("slot_out", a[5]), {batch});
    const at::Tensor y = c.out("out", a[7], {batch, dim}, c.dt);
    const int64_t stride = batch > 1 ? x.stride(0) : 0;
    const int flags = truth(a[6]) ? VS_CONV_SILU : 0;
    run("s6_conv_step", c.dev, c.written, [&] {
        return abi.s6_conv_step(batch, dim, width, c.dtype, flags, x.data_ptr(), stride, wp, bp, pool, slots, si, so, y.data_ptr(), c.stream());
    });
    return wrap(y);
}

// -------------------------------------------------------------------- scan
// what the three forms over prompts share: u, delta, z, B, C, A, Dskip, dt_bias and lengths
struct ScanIn {
    const at::Tensor &tu, &td, &tB, &tC, &tA;
    Maybe tz;
    Call c;
    int64_t batch, dim, L, N;
    const void *u, *delta, *z, *B, *C;
    const float *A, *Dskip, *dt_bias;
    const int32_t* lengths;

    ScanIn(PyObject* const* a, PyObject* lens)
        : tu(need("u", a[0])), td(need("delta", a[1])), tB(need("B", a[3])), tC(need("C", a[4])), tA(need("A", a[5])),
          tz(maybe("z", a[2])), c("u", tu, 3), batch(tu.size(0)), dim(tu.size(1)), L(tu.size(2)) {
        axes("A", tA, 2);
        N = tA.size(1);
        u = c.input("u", &tu, {batch, dim, L});
        delta = c.input("delta", &td, {batch, dim, L});
        z = c.input("z", tz, {batch, dim, L});
        B = c.input("B", &tB, {batch, N, L});
        C = c.input("C", &tC, {batch, N, L});
        A = c.dense<float>("A", &tA, {dim, N});
        Dskip = c.dense<float>("Dskip", maybe("Dskip", a[6]), {dim});
        dt_bias = c.dense<float>("dt_bias", maybe("dt_bias", a[7]), {dim});
        lengths = c.dense<int32_t>("lengths", maybe("lengths", lens), {batch});
    }
    size_t bytes(int op) const { return abi.s6_workspace_bytes(op, batch, dim, N, L); }
};

// u, delta, z, B, C, A, Dskip, dt_bias, h0, lengths, delta_softplus, out, h_out, workspace[, saved]
PyObject* scan_call(PyObject* const* a, bool saves) {
    const ScanIn s(a, a[9]);
    const Call& c = s.c;
    const float* h0 = c.dense<float>("h0", maybe("h0", a[8]), {s.batch, s.dim, s.N});
    const at::Tensor y = c.out("out", a[11], {s.batch, s.dim, s.L}, c.dt);
    const at::Tensor h = c.out("h_out", a[12], {s.batch, s.dim, s.N}, at::kFloat);
    const Strides st({&s.tu, &s.td, s.tz, &s.tB, &s.tC});
    const int flags = truth(a[10]) ? VS_FLAG_SOFTPLUS : 0;
    if (!saves) {
        const Buffer ws("workspace", s.bytes(VS_S6_SCAN), c, a[13]);
        run("s6_causal_scan", c.dev, c.written, [&] {
            return abi.s6_causal_scan(s.batch, s.dim, s.N, s.L, c.dtype, flags, s.u, s.delta, s.z, s.B, s.C, st.p, s.A, s.Dskip, s.dt_bias,
                                      h0, s.lengths, y.data_ptr(), f32(h), ws.p, ws.bytes, c.stream());
        });
        return tuple({y, h});
    }
    const Buffer saved("saved", s.bytes(VS_S6_SAVED), c, a[14]), ws("workspace", s.bytes(VS_S6_SCAN), c, a[13]);
    run("s6_causal_scan_saved", c.dev, c.written, [&] {
        return abi.s6_causal_scan_saved(s.batch, s.dim, s.N, s.L, c.dtype, flags, s.u, s.delta, s.z, s.B, s.C, st.p, s.A, s.Dskip,
                                        s.dt_bias, h0, s.lengths, y.data_ptr(), f32(h), saved.p, saved.bytes, ws.p, ws.bytes, c.stream());
    });
    return tuple({y, h, saved.t});
}
PyObject* scan(PyObject* const* a) { return scan_call(a, false); }
PyObject* scan_saved(PyObject* const* a) { return scan_call(a, true); }

// u, delta, z, B, C, A, Dskip, dt_bias, saved, dy, dh, h0, lengths, delta_softplus, workspace
PyObject* scan_grad(PyObject* const* a) {
    const ScanIn s(a, a[12]);
    const Call& c = s.c;
    const at::Tensor& tdy = need("dy", a[9]);
    const void* dy = c.input("dy", &tdy, {s.batch, s.dim, s.L});
    const float* dh = c.dense<float>("dh", maybe("dh", a[10]), {s.batch, s.dim, s.N});
    const float* h0 = c.dense<float>("h0", maybe("h0", a[11]), {s.batch, s.dim, s.N});
    need("saved", a[8]);
    const Buffer saved("saved", s.bytes(VS_S6_SAVED), c, a[8], false), ws("workspace", s.bytes(VS_S6_GRAD), c, a[14]);
    const auto act = [&] { return c.fresh({s.batch, s.dim, s.L}, c.dt); };
    const auto fp = [&](Dims d) { return c.fresh(d, at::kFloat); };
    const at::Tensor du = act(), dd = act();
    at::Tensor dz, dh0;
    if (s.tz) dz = act();
    if (h0) dh0 = fp({s.batch, s.dim, s.N});
    const at::Tensor dB = fp({s.batch, s.N, s.L}), dC = fp({s.batch, s.N, s.L}), dA = fp({s.dim, s.N}), dD = fp({s.dim}), db = fp({s.dim});
    const Strides st({&s.tu, &s.td, s.tz, &s.tB, &s.tC, &tdy});
    const int flags = truth(a[13]) ? VS_FLAG_SOFTPLUS : 0;
    run("s6_causal_scan_grad", c.dev, c.written, [&] {
        return abi.s6_causal_scan_grad(s.batch, s.dim, s.N, s.L, c.dtype, flags, s.u, s.delta, s.z, s.B, s.C, dy, st.p, s.A, s.Dskip,
                                       s.dt_bias, s.lengths, saved.p, saved.bytes, dh, du.data_ptr(), dd.data_ptr(), at_or_null(dz),
                                       f32(dB), f32(dC), f32(dA), f32(dD), f32(db), f32(dh0), ws.p, ws.bytes, c.stream());
    });
    return dict({{"du", du}, {"ddelta", dd}, {"dz", dz}, {"dB", dB}, {"dC", dC}, {"dA", dA}, {"dD", dD}, {"ddt_bias", db}, {"dh0", dh0}});
}

// u, delta, z, B, C, A, Dskip, dt_bias, h, slot_in, slot_out, delta_softplus, out
PyObject* scan_step(PyObject* const* a) {
    const at::Tensor &u = need("u", a[0]), &delta = need("delta", a[1]), &B = need("B", a[3]), &C = need("C", a[4]);
    const at::Tensor &A = need("A", a[5]), &h = need("h", a[8]);
    Maybe z = maybe("z", a[2]);
    const Call c("u", u, 2);
    axes("A", A, 2);
    axes("h", h, 3);
    const int64_t batch = u.size(0), dim = u.size(1), N = A.size(1), slots = h.size(0);
    const void *up = c.input("u", &u, {batch, dim}), *dp = c.input("delta", &delta, {batch, dim}), *zp = c.input("z", z, {batch, dim});
    const void *Bp = c.input("B", &B, {batch, N}), *Cp = c.input("C", &C, {batch, N});
    const float* Ap = c.dense<float>("A", &A, {dim, N});
    const float* Dp = c.dense<float>("Dskip", maybe("Dskip", a[6]), {dim});
    const float* bias = c.dense<float>("dt_bias", maybe("dt_bias", a[7]), {dim});
    float* hp = c.dense<float>("h", &h, {slots, dim, N});
    c.written.add("h", &h);
    const int32_t* si = c.dense<int32_t>("slot_in", maybe("slot_in", a[9]), {batch});
    const int32_t* so = c.dense<int32_t>("slot_out", maybe("slot_out", a[10]), {batch});
    const at::Tensor y = c.out("out", a[12], {batch, dim}, c.dt);
    int64_t st[5];
    const int64_t* stp = nullptr;
    int k = 0;
    for (Maybe t : {&u, &delta, z, &B, &C}) {
        if (batch > 1 && t && !t->is_contiguous()) stp = st;
        st[k++] = t ? t->stride(0) : 0;
    }
    const int flags = truth(a[11]) ? VS_FLAG_SOFTPLUS : 0;
    run("s6_scan_step", c.dev, c.written, [&] {
        return abi.s6_scan_step(batch, dim, N, c.dtype, flags, up, dp, zp, Bp, Cp, stp, Ap, Dp, bias, hp, slots, si, so, y.data_ptr(), c.stream());
    });
    return wrap(y);
}

// ------------------------------------------------- gated linear recurrence
// what the forms over prompts share: x, r, i, lam, z, lengths and rate
struct GatedIn {
    const at::Tensor &tx, &tr, &ti;
    Maybe tz;
    Call c;
    int64_t batch, dim, L;
    const void *x, *r, *i, *z;
    const float* lam;
    const int32_t* lengths;
    float rate;

    GatedIn(PyObject* const* a, PyObject* zed, PyObject* lens, PyObject* rt)
        : tx(need("x", a[0])), tr(need("r", a[1])), ti(need("i", a[2])), tz(maybe("z", zed)), c("x", tx, 3), batch(tx.size(0)),
          dim(tx.size(1)), L(tx.size(2)) {
        x = c.input("x", &tx, {batch, dim, L});
        r = c.input("r", &tr, {batch, dim, L});
        i = c.input("i", &ti, {batch, dim, L});
        z = c.input("z", tz, {batch, dim, L});
        lam = c.dense<float>("lam", &need("lam", a[3]), {dim});
        lengths = c.dense<int32_t>("lengths", maybe("lengths", lens), {batch});
        rate = number("rate", rt);
    }
    size_t bytes(int op) const { return abi.gated_workspace_bytes(op, batch, dim, L); }
};

// x, r, i, lam, z, h0, lengths, rate, out, h_out[, saved]
PyObject* gated_call(PyObject* const* a, bool saves) {
    const GatedIn s(a, a[4], a[6], a[7]);
    const Call& c = s.c;
    const float* h0 = c.dense<float>("h0", maybe("h0", a[5]), {s.batch, s.dim});
    const at::Tensor y = c.out("out", a[8], {s.batch, s.dim, s.L}, c.dt), h = c.out("h_out", a[9], {s.batch, s.dim}, at::kFloat);
    const Strides st({&s.tx, &s.tr, &s.ti, s.tz});
    if (!saves) {
        run("gated_scan", c.dev, c.written, [&] {
            return abi.gated_scan(s.batch, s.dim, s.L, c.dtype, s.x, s.r, s.i, s.z, st.p, s.lam, s.rate, h0, s.lengths, y.data_ptr(), f32(h),
                                  c.stream());
        });
        return tuple({y, h});
    }
    const Buffer saved("saved", s.bytes(VS_GATED_SAVED), c, a[10]);
    run("gated_scan_saved", c.dev, c.written, [&] {
        return abi.gated_scan_saved(s.batch, s.dim, s.L, c.dtype, s.x, s.r, s.i, s.z, st.p, s.lam, s.rate, h0, s.lengths, y.data_ptr(),
                                    f32(h), saved.p, saved.bytes, c.stream());
    });
    return tuple({y, h, saved.t});
}
PyObject* gated(PyObject* const* a) { return gated_call(a, false); }
PyObject* gated_saved(PyObject* const* a) { return gated_call(a, true); }

// x, r, i, lam, saved, dy, z, dh, h0, lengths, rate, workspace
PyObject* gated_grad(PyObject* const* a) {
    const GatedIn s(a, a[6], a[9], a[10]);
    const Call& c = s.c;
    const at::Tensor& tdy = need("dy", a[5]);
    const void* dy = c.input("dy", &tdy, {s.batch, s.dim, s.L});
    const float* dh = c.dense<float>("dh", maybe("dh", a[7]), {s.batch, s.dim});
    const float* h0 = c.dense<float>("h0", maybe("h0", a[8]), {s.batch, s.dim});
    need("saved", a[4]);
    const Buffer saved("saved", s.bytes(VS_GATED_SAVED), c, a[4], false), ws("workspace", s.bytes(VS_GATED_GRAD), c, a[11]);
    const auto act = [&] { return c.fresh({s.batch, s.dim, s.L}, c.dt); };
    const at::Tensor dx = act(), dr = act(), di = act(), dlam = c.fresh({s.dim}, at::kFloat);
    at::Tensor dz, dh0;
    if (s.tz) dz = act();
    if (h0) dh0 = c.fresh({s.batch, s.dim}, at::kFloat);
    const Strides st({&s.tx, &s.tr, &s.ti, s.tz, &tdy});
    run("gated_scan_grad", c.dev, c.written, [&] {
        return abi.gated_scan_grad(s.batch, s.dim, s.L, c.dtype, s.x, s.r, s.i, s.z, dy, st.p, s.lam, s.rate, s.lengths, saved.p, saved.bytes,
                                   dh, dx.data_ptr(), dr.data_ptr(), di.data_ptr(), at_or_null(dz), f32(dlam), f32(dh0), ws.p, ws.bytes,
                                   c.stream());
    });
    return dict({{"dx", dx}, {"dr", dr}, {"di", di}, {"dz", dz}, {"dlam", dlam}, {"dh0", dh0}});
}

// x, r, i, lam, h, z, slot_in, slot_out, rate, out
PyObject* gated_step(PyObject* const* a) {
    const at::Tensor &x = need("x", a[0]), &r = need("r", a[1]), &i = need("i", a[2]), &lam = need("lam", a[3]), &h = need("h", a[4]);
    Maybe z = maybe("z", a[5]);
    const Call c("x", x, 2);
    axes("h", h, 2);
    const int64_t batch = x.size(0), dim = x.size(1), slots = h.size(0);
    const void *xp = c.input("x", &x, {batch, dim}), *rp = c.input("r", &r, {batch, dim}), *ip = c.input("i", &i, {batch, dim});
    const void* zp = c.input("z", z, {batch, dim});
    const float* lp = c.dense<float>("lam", &lam, {dim});
    float* hp = c.dense<float>("h", &h, {slots, dim});
    c.written.add("h", &h);
    const int32_t* si = c.dense<int32_t>("slot_in", maybe("slot_in", a[6]), {batch});
    const int32_t* so = c.dense<int32_t>("slot_out", maybe("slot_out", a[7]), {batch});
    const float rate = number("rate", a[8]);
    const at::Tensor y = c.out("out", a[9], {batch, dim}, c.dt);
    int64_t st[4] = {};                                      // one row has no stride
    if (batch > 1) {
        int k = 0;
        for (Maybe t : {&x, &r, &i, z}) st[k++] = t ? t->stride(0) : 0;
    }
    run("gated_scan_step", c.dev, c.written, [&] {
        return abi.gated_scan_step(batch, dim, c.dtype, xp, rp, ip, zp, st, lp, rate, hp, slots, si, so, y.data_ptr(), c.stream());
    });
    return wrap(y);
}

// -------------------------------------------------------------------- norm
// A row form [rows, dim] is the channel-major form's [rows, dim, 1] with
// channel stride 1.
struct NormIn {
    Call c;
    int64_t batch, dim, L;
    bool rows;
    int64_t st[6];

    NormIn(const char* name, const at::Tensor& t) : c(name, t, t.dim() == 2 ? 2 : 3), batch(t.size(0)), dim(t.size(1)), L(t.dim() == 2 ? 1 : t.size(2)), rows(t.dim() == 2) {}
    const void* input(const char* name, Maybe t, int k) {
        st[2 * k] = st[2 * k + 1] = 0;
        if (!t) return nullptr;
        const void* p = rows ? c.input(name, t, {batch, dim}) : c.input(name, t, {batch, dim, L});
        st[2 * k] = batch > 1 ? t->stride(0) : 0;
        st[2 * k + 1] = dim > 1 ? t->stride(1) : 1;
        return p;
    }
    at::Tensor out(const char* name, PyObject* given) const {
        return rows ? c.out(name, given, {batch, dim}, c.dt) : c.out(name, given, {batch, dim, L}, c.dt);
    }
    const float* weight(PyObject* o) const { return c.dense<float>("w", maybe("w", o), {dim}); }
    const int32_t* lengths(PyObject* o) const { return c.dense<int32_t>("lengths", maybe("lengths", o), {batch}); }
};

// x, w, residual, eps, lengths, out, sum_out
PyObject* norm(PyObject* const* a) {
    const at::Tensor& x = need("x", a[0]);
    NormIn n("x", x);
    Maybe res = maybe("residual", a[2]);
    const void *xp = n.input("x", &x, 0), *rp = n.input("residual", res, 1);
    const float* w = n.weight(a[1]);
    const float eps = number("eps", a[3]);
    const int32_t* len = n.lengths(a[4]);
    const at::Tensor y = n.out("out", a[5]);
    at::Tensor sum;
    if (res) sum = n.out("sum_out", a[6]);
    else if (a[6] != Py_None) raise(PyExc_ValueError, "sum_out needs a residual");
    run("rms_norm", n.c.dev, n.c.written, [&] {
        return abi.rms_norm(n.batch, n.dim, n.L, n.c.dtype, xp, rp, n.st, w, eps, len, y.data_ptr(), at_or_null(sum), n.c.stream());
    });
    return tuple({y, sum});
}

// s, w, dy, dsum, eps, lengths, workspace
PyObject* norm_grad(PyObject* const* a) {
    const at::Tensor &s = need("s", a[0]), &dy = need("dy", a[2]);
    NormIn n("s", s);
    const void *sp = n.input("s", &s, 0), *yp = n.input("dy", &dy, 1), *dp = n.input("dsum", maybe("dsum", a[3]), 2);
    const float* w = n.weight(a[1]);
    const float eps = number("eps", a[4]);
    const int32_t* len = n.lengths(a[5]);
    const at::Tensor ds = n.out("ds", Py_None);
    at::Tensor dw;
    if (w) dw = n.c.fresh({n.dim}, at::kFloat);
    const Buffer ws("workspace", w ? abi.norm_workspace_bytes(n.batch, n.dim, n.L) : 0, n.c, a[6]);
    run("rms_norm_grad", n.c.dev, n.c.written, [&] {
        return abi.rms_norm_grad(n.batch, n.dim, n.L, n.c.dtype, sp, yp, dp, n.st, w, eps, len, ds.data_ptr(), f32(dw), ws.p, ws.bytes,
                                 n.c.stream());
    });
    return dict({{"dx", ds}, {"dw", dw}});
}

// --------------------------------------------------------- vocabulary loss
// x, W, target
struct VocabIn {
    const at::Tensor &tx, &tW, &tt;
    Call c;
    int64_t tokens, dim, vocab, stride;
    const void *x, *W, *target;
    int bits;

    explicit VocabIn(PyObject* const* a) : tx(need("x", a[0])), tW(need("W", a[1])), tt(need("target", a[2])), c("x", tx, 2), tokens(tx.size(0)), dim(tx.size(1)) {
        axes("W", tW, 2);
        vocab = tW.size(0);
        x = c.input("x", &tx, {tokens, dim});
        stride = tokens > 1 ? tx.stride(0) : dim;
        W = c.dense("W", &tW, {vocab, dim}, c.dt);
        bits = tt.scalar_type() == at::kInt ? 32 : 64;
        target = c.dense("target", &tt, {tokens}, bits == 32 ? at::kInt : at::kLong);
    }
    size_t bytes(int op) const { return abi.vocab_workspace_bytes(op, tokens, dim, vocab, c.dtype); }
};

// x, W, target, workspace
PyObject* vocab_forward(PyObject* const* a) {
    VocabIn v(a);
    const Call& c = v.c;
    at::Tensor x = v.tx;
    if (v.tokens > 1 && v.stride < v.dim) {                  // one row for all, or overlapping rows
        x = v.tx.contiguous();
        v.stride = v.dim;
    }
    const Buffer ws("workspace", v.bytes(VS_VOCAB_LOSS), c, a[3]);
    const at::Tensor loss = c.fresh({v.tokens}, at::kFloat), lse = c.fresh({v.tokens}, at::kFloat);
    run("vocab_loss", c.dev, c.written, [&] {
        return abi.vocab_loss(v.tokens, v.dim, v.vocab, c.dtype, x.data_ptr(), v.stride, v.W, v.target, v.bits, f32(loss), f32(lse), ws.p,
                              ws.bytes, c.stream());
    });
    return tuple({loss, lse});
}

// x, W, target, lse, dloss, workspace
PyObject* vocab_grad(PyObject* const* a) {
    VocabIn v(a);
    const Call& c = v.c;
    at::Tensor x = v.tx;
    if (v.tokens > 1 && v.stride < v.dim) {
        x = v.tx.contiguous();
        v.stride = v.dim;
    }
    const float* lse = c.dense<float>("lse", &need("lse", a[3]), {v.tokens});
    const float* dloss = c.dense<float>("dloss", &need("dloss", a[4]), {v.tokens});
    const Buffer ws("workspace", v.bytes(VS_VOCAB_GRAD), c, a[5]);
    const at::Tensor dx = c.fresh({v.tokens, v.dim}, c.dt), dW = c.fresh({v.vocab, v.dim}, c.dt);
    run("vocab_loss_grad", c.dev, c.written, [&] {
        return abi.vocab_loss_grad(v.tokens, v.dim, v.vocab, c.dtype, x.data_ptr(), v.stride, v.W, v.target, v.bits, lse, dloss,
                                   dx.data_ptr(), dW.data_ptr(), ws.p, ws.bytes, c.stream());
    });
    return dict({{"dx", dx}, {"dW", dW}});
}

// ------------------------------------------------------------- beam search
// logits, scores, done, eos, workspace, out[0], out[1], out[2]
PyObject* select(PyObject* const* a) {
    const at::Tensor &logits = need("logits", a[0]), &scores = need("scores", a[1]);
    const Call c("logits", logits, 3);
    const int64_t batch = logits.size(0), beams = logits.size(1), vocab = logits.size(2);
    const void* lp = c.input("logits", &logits, {batch, beams, vocab});
    const float* sp = c.dense<float>("scores", &scores, {batch, beams});
    const void* done = c.dense("done", maybe("done", a[2]), {batch, beams}, at::kBool);
    if (done && a[3] == Py_None) raise(PyExc_ValueError, "eos is required where done is given");
    int64_t eos = 0;
    if (a[3] != Py_None) {
        PyObject* v = PyNumber_Long(a[3]);
        if (!v) throw python_error();
        eos = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (eos == -1 && PyErr_Occurred()) throw python_error();
    }
    const at::Tensor s = c.out("out[0]", a[5], {batch, beams}, at::kFloat), p = c.out("out[1]", a[6], {batch, beams}, at::kInt);
    const at::Tensor t = c.out("out[2]", a[7], {batch, beams}, at::kInt);
    const Strides st({&logits});
    const Buffer ws("workspace", abi.beam_workspace_bytes(batch, beams, vocab), c, a[4]);
    run("beam_select", c.dev, c.written, [&] {
        return abi.beam_select(batch, beams, vocab, c.dtype, lp, st.p, sp, static_cast<const uint8_t*>(done), eos, f32(s),
                               static_cast<int32_t*>(p.data_ptr()), static_cast<int32_t*>(t.data_ptr()), ws.p, ws.bytes, c.stream());
    });
    return tuple({s, p, t});
}

// state, parent, out
PyObject* reorder(PyObject* const* a) {
    const at::Tensor &state = need("state", a[0]), &parent = need("parent", a[1]);
    Maybe given = maybe("out", a[2]);
    const at::Tensor& out = given ? *given : state;
    if (!state.is_cuda()) raise(PyExc_ValueError, "state must be on the GPU");
    if (parent.dim() != 2 || state.dim() < 2 || state.size(1) != parent.size(0) * parent.size(1))
        raise(PyExc_ValueError, "state must be [layers, batch * beams, ...] for a parent of [batch, beams]");
    if (parent.scalar_type() != at::kInt) raise(PyExc_TypeError, "parent has dtype %S, expected %S", dtype_name(parent.scalar_type()), dtype_name(at::kInt));
    if (parent.device() != state.device() || !parent.is_contiguous())
        raise(PyExc_ValueError, "parent must be contiguous and on %s", state.device().str().c_str());
    if (state.numel() == 0) raise(PyExc_ValueError, "state is empty: %s", shape(state.sizes()).c_str());
    const int64_t layers = state.size(0), rows = state.size(1), layer = state.numel() / layers;
    int64_t dense = 1;                                      // strides of a layer's contiguous rows, from the last axis on
    bool ok = layers == 1 || state.stride(0) >= layer;
    for (int64_t d = state.dim() - 1; d > 0; --d) {
        ok = ok && (state.size(d) == 1 || state.stride(d) == dense);
        dense *= state.size(d);
    }
    if (!ok) raise(PyExc_ValueError, "each layer of state must be contiguous and apart from the others");
    if (out.scalar_type() != state.scalar_type() || out.sizes() != state.sizes() || out.strides() != state.strides() ||
        out.device() != state.device())
        raise(PyExc_ValueError, "out must have state's dtype, shape, strides and device");
    Written written;
    written.add(given ? "out" : "state", &out);
    const int64_t es = static_cast<int64_t>(state.element_size());
    const int64_t row_bytes = layer / rows * es, layer_bytes = layers > 1 ? state.stride(0) * es : 0;
    run("beam_reorder", state.device(), written, [&] {
        return abi.beam_reorder(layers, parent.size(0), parent.size(1), row_bytes, layer_bytes, state.data_ptr(),
                                static_cast<const int32_t*>(parent.data_ptr()), out.data_ptr(),
                                c10::hip::getCurrentHIPStream(state.device().index()).stream());
    });
    PyObject* r = given ? a[2] : a[0];
    Py_INCREF(r);
    return r;
}

// ---------------------------------------------------------------- autograd
// whether a node was made on a stream that is neither the current one nor being captured with it
bool elsewhere(const c10::Stream& made) {
    if (made.id() == c10::hip::getCurrentHIPStream(made.device_index()).unwrap().id()) return false;
    const hipStream_t s = c10::hip::HIPStream(c10::hip::HIPStream::UNCHECKED, made).stream();
    if (!s) return true;                                     // the null stream cannot be captured
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &status) != hipSuccess) (void)hipGetLastError();
    return status == hipStreamCaptureStatusNone;
}

// A differentiable call's arguments, before it is made. Where their stream is
// capturing and gradients are recorded, no graph that leads to one of them may have
// a node of an eager graph that is still alive, a leaf's among them: that node
// belongs to the stream it was made on, and the captured backward pass would
// make that stream wait inside the capture, which ends the process.
PyObject* capture_ready(PyObject* const* a) {
    using torch::autograd::Node;
    if (!PyTuple_Check(a[0])) raise(PyExc_TypeError, "expected a tuple of arguments");
    if (!at::GradMode::is_enabled()) Py_RETURN_NONE;
    std::vector<std::shared_ptr<Node>> todo;
    bool capturing = false;
    for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(a[0]); ++k) {
        PyObject* o = PyTuple_GET_ITEM(a[0], k);
        if (!THPVariable_Check(o)) continue;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || !t.requires_grad()) continue;
        if (!capturing) {
            const c10::DeviceGuard guard(t.device());
            if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) Py_RETURN_NONE;
            capturing = true;
        }
        todo.push_back(t.is_leaf() ? torch::autograd::impl::try_get_grad_accumulator(t) : t.grad_fn());
    }
    std::unordered_set<const Node*> seen;
    while (!todo.empty()) {
        const std::shared_ptr<Node> node = std::move(todo.back());
        todo.pop_back();
        if (!node || !seen.insert(node.get()).second) continue;
        const auto made = node->stream();
        if (made && elsewhere(*made))
            raise(PyExc_RuntimeError, "an eager graph that is still alive leads to this call or shares a leaf with it: free it (its outputs and losses) "
                                      "before its backward pass is captured");
        for (const auto& edge : node->next_edges()) todo.push_back(edge.function);
    }
    Py_RETURN_NONE;
}

// ------------------------------------------------------------------ module
// addresses of the library's functions by name, and what turns a status into an
// exception; where one is missing, those bound before stay
PyObject* bind(PyObject*, PyObject* args) {
    PyObject *table, *check;
    if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &table, &check)) return nullptr;
    Abi found;
#define VS_FIND(f)                                                                          \
    {                                                                                       \
        PyObject* v = PyDict_GetItemString(table, #f);                                      \
        void* p = v ? PyLong_AsVoidPtr(v) : nullptr;                                        \
        if (!p) {                                                                           \
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no address of " #f);  \
            return nullptr;                                                                 \
        }                                                                                   \
        found.f = reinterpret_cast<decltype(found.f)>(p);                                   \
    }
    VS_BOUND(VS_FIND)
#undef VS_FIND
    abi = found;
    Py_INCREF(check);
    Py_XSETREF(check_status, check);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) raise(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    if (!check_status) raise(PyExc_RuntimeError, "bind() was not called");
    return F(a);
    END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    method<conv, 8>("s6_causal_conv"), method<conv_grad, 9>("s6_causal_conv_grad"), method<conv_step, 8>("s6_conv_step"),
    method<scan, 14>("s6_causal_scan"), method<scan_saved, 15>("s6_causal_scan_saved"), method<scan_grad, 15>("s6_causal_scan_grad"),
    method<scan_step, 13>("s6_scan_step"), method<select, 8>("beam_select"), method<reorder, 3>("beam_reorder"),
    method<gated, 10>("gated_scan"), method<gated_saved, 11>("gated_scan_saved"), method<gated_grad, 12>("gated_scan_grad"),
    method<gated_step, 10>("gated_scan_step"), method<norm, 7>("rms_norm"), method<norm_grad, 7>("rms_norm_grad"),
    method<vocab_forward, 4>("vocab_loss"), method<vocab_grad, 6>("vocab_loss_grad"),
    method<capture_ready, 1>("capture_ready"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
