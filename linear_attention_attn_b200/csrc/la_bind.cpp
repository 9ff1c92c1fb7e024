// la_bind.cpp -- CPython module behind the binding's operators around the token mixers: checks the
// tensors, takes their addresses, finds the stream and the workspace, and calls the C entry point.
//
// Everything here also works through ctypes; a single-token call then spends about 10 us on the host
// (2 of them in the launch), most of it in argument conversion, while its kernel runs for 2 to 5 us.
// Functions take positional arguments only (the package wraps them) and return the la_status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/la.h"

namespace {

struct Refused {};                       // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw Refused{};
}

const at::Tensor &as_tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch tensor");
    return THPVariable_Unpack(o);
}

// One call: its first tensor fixes device and dtype, the others are held against them.
class Call {
public:
    Call(PyObject *first, const char *name, int dims) : x_(as_tensor(first, name)) {
        if (!x_.is_cuda() || x_.dim() != dims || !x_.is_contiguous())
            refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor of " + std::to_string(dims) +
                                         " dimensions");
        switch (x_.scalar_type()) {
        case at::kFloat: code = LA_F32; break;
        case at::kHalf: code = LA_F16; break;
        case at::kBFloat16: code = LA_BF16; break;
        default: refuse(PyExc_TypeError, std::string("unsupported dtype ") + at::toString(x_.scalar_type()));
        }
    }
    int size(int d) const { return fit(x_.size(d)); }
    static int fit(int64_t n) {
        if (n > 2147483647) refuse(PyExc_ValueError, "a dimension exceeds 2^31 - 1");
        return (int)n;
    }
    at::IntArrayRef sizes() const { return x_.sizes(); }
    void *data() const { return x_.data_ptr(); }
    // Address of a tensor of this shape (null for None): of the call's dtype, or of `type`.
    void *like(PyObject *o, const char *name) const { return at(o, name, x_.sizes(), x_.scalar_type()); }
    void *same(PyObject *o, const char *name, at::IntArrayRef shape) const { return at(o, name, shape, x_.scalar_type()); }
    float *f32(PyObject *o, const char *name, at::IntArrayRef shape) const {
        return (float *)at(o, name, shape, at::kFloat);
    }
    void *at(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type) const {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = as_tensor(o, name);
        if (t.scalar_type() != type || t.sizes() != shape || t.device() != x_.device() || !t.is_contiguous()) {
            std::string s;
            for (int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
            refuse(PyExc_ValueError, std::string(name) + " must be a contiguous " + at::toString(type) + " tensor [" + s +
                                         "] on " + x_.device().str());
        }
        return t.data_ptr();
    }
    const int *lengths(PyObject *o, int B) const { return (const int *)at(o, "lengths", {B}, at::kInt); }

    // The stream to launch on: None for torch's current one, else the handle as an int.
    void on(PyObject *stream) {
        guard_.emplace(x_.device());
        if (stream == Py_None) {
            stream_ = c10::cuda::getCurrentCUDAStream(x_.device().index()).stream();
        } else {
            stream_ = (cudaStream_t)PyLong_AsVoidPtr(stream);
            if (PyErr_Occurred()) throw Refused{};
            given_ = true;
        }
    }
    void *stream() const { return (void *)stream_; }

    // Workspace: the caller's tensor, or memory from the pool of the stream that the kernels run on,
    // whose earlier users are done there.
    void workspace(PyObject *o, size_t need) {
        if (o != Py_None) {
            const at::Tensor &t = as_tensor(o, "workspace");
            if (t.device() != x_.device() || !t.is_contiguous())
                refuse(PyExc_ValueError, "workspace must be a contiguous tensor on " + x_.device().str());
            ws = t.data_ptr();
            ws_bytes = t.nbytes();
        } else if (need) {
            std::optional<c10::cuda::CUDAStreamGuard> g;
            if (given_) g.emplace(c10::cuda::getStreamFromExternal(stream_, x_.device().index()));
            mem_ = at::empty({(int64_t)need}, x_.options().dtype(at::kByte));
            ws = mem_.data_ptr();
            ws_bytes = need;
        }
    }
    la_dtype code;
    void *ws = nullptr;
    size_t ws_bytes = 0;

private:
    const at::Tensor &x_;
    at::Tensor mem_;
    std::optional<c10::cuda::CUDAGuard> guard_;
    cudaStream_t stream_ = nullptr;
    bool given_ = false;
};

long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}

using Body = la_status (*)(PyObject *const *);
template <int N, Body body>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        if (n != N) refuse(PyExc_TypeError, "wrong number of arguments");
        return PyLong_FromLong(body(args));
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// back, q, k, oq, ok, freqs, positions, start, layout, magnitude, stream
la_status rotary(PyObject *const *a) {
    const bool back = integer(a[0]) != 0;
    Call c(a[1], back ? "doq" : "q", 4);
    const int B = c.size(0), H = c.size(1), T = c.size(2), D = c.size(3);
    if ((a[2] == Py_None) != (a[4] == Py_None)) refuse(PyExc_ValueError, "k and its output must be given together");
    int Hk = 0;
    if (a[2] != Py_None) {
        const at::Tensor &k = as_tensor(a[2], "k");
        if (k.dim() != 4) refuse(PyExc_ValueError, "k must be a [B, Hk, T, D] tensor");
        Hk = Call::fit(k.size(1));
    }
    const int64_t ks[4] = {B, Hk, T, D};
    const int64_t pairs = as_tensor(a[5], "freqs").numel();
    if (pairs > 512) refuse(PyExc_ValueError, "freqs has more than 512 entries");
    int per_batch = 0;
    const long long *pos = nullptr;
    if (a[6] != Py_None) {
        per_batch = as_tensor(a[6], "positions").dim() == 2;
        const int64_t two[2] = {B, T};
        pos = (const long long *)c.at(a[6], "positions", per_batch ? at::IntArrayRef(two, 2) : at::IntArrayRef(two + 1, 1),
                                      at::kLong);
    }
    void *k = c.same(a[2], "k", ks), *oq = c.like(a[3], "the first output"), *ok = c.same(a[4], "the second output", ks);
    float *freqs = c.f32(a[5], "freqs", {pairs});
    const long long start = integer(a[7]);
    const la_rotary_layout layout = (la_rotary_layout)integer(a[8]);
    const float magnitude = number(a[9]);
    c.on(a[10]);
    return (back ? la_rotary_bwd : la_rotary_fwd)(c.data(), k, oq, ok, freqs, pos, per_batch, start, layout, magnitude, B,
                                                  H, Hk, T, D, (int)(2 * pairs), c.code, c.stream());
}

int taps(PyObject *w) {
    const at::Tensor &t = as_tensor(w, "w");
    if (t.dim() != 2) refuse(PyExc_ValueError, "w must be a [C, W] tensor");
    return Call::fit(t.size(1));
}

// x, w, bias, state_in, y, state_out, lengths, act, stream
la_status conv_fwd(PyObject *const *a) {
    Call c(a[0], "x", 3);
    const int B = c.size(0), T = c.size(1), C = c.size(2), W = taps(a[1]);
    const int64_t st[3] = {B, W - 1, C};
    float *w = c.f32(a[1], "w", {C, W}), *bias = c.f32(a[2], "bias", {C});
    void *si = c.same(a[3], "state_in", st), *y = c.like(a[4], "y"), *so = c.same(a[5], "state_out", st);
    const int *len = c.lengths(a[6], B);
    const la_activation act = (la_activation)integer(a[7]);
    c.on(a[8]);
    return la_short_conv_fwd(c.data(), w, bias, si, y, so, len, act, B, T, C, W, c.code, c.stream());
}

// x, w, bias, state_in, y, state_out, act, stream
la_status conv_step(PyObject *const *a) {
    Call c(a[0], "x", 2);
    const int B = c.size(0), C = c.size(1), W = taps(a[1]);
    const int64_t st[3] = {B, W - 1, C};
    float *w = c.f32(a[1], "w", {C, W}), *bias = c.f32(a[2], "bias", {C});
    void *si = c.same(a[3], "state_in", st), *y = c.like(a[4], "y"), *so = c.same(a[5], "state_out", st);
    const la_activation act = (la_activation)integer(a[6]);
    c.on(a[7]);
    return la_short_conv_step(c.data(), w, bias, si, y, so, act, B, C, W, c.code, c.stream());
}

// x, w, bias, state_in, dy, dstate_in, dx, dw, dbias, dstate_out, lengths, act, workspace, stream
la_status conv_bwd(PyObject *const *a) {
    Call c(a[0], "x", 3);
    const int B = c.size(0), T = c.size(1), C = c.size(2), W = taps(a[1]);
    const int64_t st[3] = {B, W - 1, C};
    float *w = c.f32(a[1], "w", {C, W}), *bias = c.f32(a[2], "bias", {C});
    void *si = c.same(a[3], "state_in", st), *dy = c.like(a[4], "dy"), *di = c.same(a[5], "dstate_in", st);
    void *dx = c.like(a[6], "dx");
    float *dw = c.f32(a[7], "dw", {C, W}), *db = c.f32(a[8], "dbias", {C});
    void *dso = c.same(a[9], "dstate_out", st);
    const int *len = c.lengths(a[10], B);
    const la_activation act = (la_activation)integer(a[11]);
    c.on(a[13]);
    c.workspace(a[12], la_mixer_workspace_size(LA_OP_SHORT_CONV_BWD, B, T, C, 1, W, c.code));
    return la_short_conv_bwd(c.data(), w, bias, si, dy, di, dx, dw, db, dso, len, act, B, T, C, W, c.code, c.ws,
                             c.ws_bytes, c.stream());
}

// The inputs that every form of the scan takes, at a[0..8]: x, dt, A, Bm, Cm, D, z, dt_bias, state_in.
struct ScanIn {
    ScanIn(const Call &c, PyObject *const *a, int lead) {
        const at::Tensor &b = as_tensor(a[3], "Bm");
        if (b.dim() != lead + 2)
            refuse(PyExc_ValueError, "Bm must be a tensor of " + std::to_string(lead + 2) + " dimensions ending in [G, N]");
        B = c.size(0);
        T = lead == 2 ? c.size(1) : 1;
        C = c.size(lead);
        G = Call::fit(b.size(lead));
        N = Call::fit(b.size(lead + 1));
        const int64_t full[4] = {B, T, G, N}, step[3] = {B, G, N};
        const at::IntArrayRef bc = lead == 2 ? at::IntArrayRef(full, 4) : at::IntArrayRef(step, 3);
        dt = c.like(a[1], "dt");
        A = c.f32(a[2], "A", {C, N});
        Bm = c.same(a[3], "Bm", bc);
        Cm = c.same(a[4], "Cm", bc);
        D = c.f32(a[5], "D", {C});
        z = c.like(a[6], "z");
        bias = c.f32(a[7], "dt_bias", {C});
        si = c.f32(a[8], "state_in", {B, C, N});
    }
    int B, T, C, G, N;
    void *dt, *Bm, *Cm, *z;
    float *A, *D, *bias, *si;
};

// a[0..8], y, state_out, lengths, softplus, workspace, stream
la_status scan_fwd(PyObject *const *a) {
    Call c(a[0], "x", 3);
    const ScanIn s(c, a, 2);
    void *y = c.like(a[9], "y");
    float *so = c.f32(a[10], "state_out", {s.B, s.C, s.N});
    const int *len = c.lengths(a[11], s.B);
    const int sp = integer(a[12]) != 0;
    c.on(a[14]);
    c.workspace(a[13], la_mixer_workspace_size(LA_OP_SELECTIVE_SCAN_FWD, s.B, s.T, s.C, s.G, s.N, c.code));
    return la_selective_scan_fwd(c.data(), s.dt, s.A, s.Bm, s.Cm, s.D, s.z, s.bias, s.si, y, so, len, sp, s.B, s.T, s.C,
                                 s.G, s.N, c.code, c.ws, c.ws_bytes, c.stream());
}

// a[0..8], y, state_out, softplus, stream
la_status scan_step(PyObject *const *a) {
    Call c(a[0], "x", 2);
    const ScanIn s(c, a, 1);
    void *y = c.like(a[9], "y");
    float *so = c.f32(a[10], "state_out", {s.B, s.C, s.N});
    const int sp = integer(a[11]) != 0;
    c.on(a[12]);
    return la_selective_scan_step(c.data(), s.dt, s.A, s.Bm, s.Cm, s.D, s.z, s.bias, s.si, y, so, sp, s.B, s.C, s.G, s.N,
                                  c.code, c.stream());
}

// a[0..8], dy, dstate_in, dx, ddt, dA, dBm, dCm, dD, dz, ddt_bias, dstate_out, lengths, softplus, workspace, stream
la_status scan_bwd(PyObject *const *a) {
    Call c(a[0], "x", 3);
    const ScanIn s(c, a, 2);
    const int64_t bc[4] = {s.B, s.T, s.G, s.N};
    const int64_t st[3] = {s.B, s.C, s.N};
    void *dy = c.like(a[9], "dy");
    float *di = c.f32(a[10], "dstate_in", st);
    void *dx = c.like(a[11], "dx"), *ddt = c.like(a[12], "ddt");
    float *dA = c.f32(a[13], "dA", {s.C, s.N});
    void *dB = c.same(a[14], "dBm", bc), *dC = c.same(a[15], "dCm", bc);
    float *dD = c.f32(a[16], "dD", {s.C});
    void *dz = c.like(a[17], "dz");
    float *db = c.f32(a[18], "ddt_bias", {s.C}), *dso = c.f32(a[19], "dstate_out", st);
    const int *len = c.lengths(a[20], s.B);
    const int sp = integer(a[21]) != 0;
    c.on(a[23]);
    c.workspace(a[22], la_mixer_workspace_size(LA_OP_SELECTIVE_SCAN_BWD, s.B, s.T, s.C, s.G, s.N, c.code));
    return la_selective_scan_bwd(c.data(), s.dt, s.A, s.Bm, s.Cm, s.D, s.z, s.bias, s.si, dy, di, dx, ddt, dA, dB, dC, dD,
                                 dz, db, dso, len, sp, s.B, s.T, s.C, s.G, s.N, c.code, c.ws, c.ws_bytes, c.stream());
}

// x, y, groups, gamma, beta, eps, act, mean, rstd, workspace, stream
la_status norm_fwd(PyObject *const *a) {
    Call c(a[0], "x", 3);
    const int B = c.size(0), T = c.size(1), C = c.size(2), G = Call::fit(integer(a[2]));
    const int64_t bg[2] = {B, G};
    void *y = c.like(a[1], "y");
    float *ga = c.f32(a[3], "gamma", {C}), *be = c.f32(a[4], "beta", {C});
    const float eps = number(a[5]);
    const la_activation act = (la_activation)integer(a[6]);
    float *m = c.f32(a[7], "mean", bg), *r = c.f32(a[8], "rstd", bg);
    c.on(a[10]);
    c.workspace(a[9], la_mixer_workspace_size(LA_OP_GROUP_NORM_FWD, B, T, C, G, 1, c.code));
    return la_group_norm_fwd(c.data(), ga, be, y, m, r, eps, act, B, T, C, G, c.code, c.ws, c.ws_bytes, c.stream());
}

// x, dy, dx, groups, mean, rstd, gamma, beta, dgamma, dbeta, act, workspace, stream
la_status norm_bwd(PyObject *const *a) {
    Call c(a[0], "x", 3);
    const int B = c.size(0), T = c.size(1), C = c.size(2), G = Call::fit(integer(a[3]));
    const int64_t bg[2] = {B, G};
    void *dy = c.like(a[1], "dy"), *dx = c.like(a[2], "dx");
    float *m = c.f32(a[4], "mean", bg), *r = c.f32(a[5], "rstd", bg);
    float *ga = c.f32(a[6], "gamma", {C}), *be = c.f32(a[7], "beta", {C});
    float *dga = c.f32(a[8], "dgamma", {C}), *dbe = c.f32(a[9], "dbeta", {C});
    const la_activation act = (la_activation)integer(a[10]);
    c.on(a[12]);
    c.workspace(a[11], la_mixer_workspace_size(LA_OP_GROUP_NORM_BWD, B, T, C, G, 1, c.code));
    return la_group_norm_bwd(c.data(), dy, m, r, ga, be, dx, dga, dbe, act, B, T, C, G, c.code, c.ws, c.ws_bytes,
                             c.stream());
}

#define LA_ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<n, name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LA_ENTRY(rotary, 11),    LA_ENTRY(conv_fwd, 9),   LA_ENTRY(conv_step, 8),
                         LA_ENTRY(conv_bwd, 14),  LA_ENTRY(scan_fwd, 15),  LA_ENTRY(scan_step, 13),
                         LA_ENTRY(scan_bwd, 24),  LA_ENTRY(norm_fwd, 11),  LA_ENTRY(norm_bwd, 13),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_la_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__la_bind(void) { return PyModule_Create(&module); }
