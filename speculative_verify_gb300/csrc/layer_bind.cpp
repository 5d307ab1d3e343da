// layer_bind.cpp -- Python binding of the calls between the weight reads
// (the second half of specverify.h), on torch tensors.
//
// A decode step makes several of these calls, each a few microseconds of GPU
// time, so their checks and allocations are done here rather than in Python:
// a call costs little more than its launch and its outputs' allocations.
// Python (layer.py) holds the signatures and their documentation.
//
// Wrong types raise TypeError, wrong shapes, strides and devices ValueError,
// tensors that require a gradient RuntimeError (outside torch.no_grad()), and
// a status of the library the package's SpecVerifyError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "specverify.h"

namespace {

struct PyFail {};                               // a Python error has been set

[[noreturn]] void fail(PyObject *type, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw PyFail{};
}

PyObject *g_status_error = nullptr;             // SpecVerifyError(function, status)

void check_status(const char *fn, int rc)
{
    if (rc == SV_OK) return;
    PyObject *e = PyObject_CallFunction(g_status_error, "si", fn, rc);
    if (e) {
        PyErr_SetObject(g_status_error, e);
        Py_DECREF(e);
    }
    throw PyFail{};
}

constexpr auto BF16 = at::kBFloat16;
constexpr auto F32 = at::kFloat;

// The device of a call's tensors: the first one's.  The calls have no
// gradients, so a tensor that wants one is refused rather than its lost.
struct Where {
    int device = -1;

    const at::Tensor &operator()(const at::Tensor &t, const char *name)
    {
        if (t.requires_grad() && c10::GradMode::is_enabled())
            fail(PyExc_RuntimeError, "%s requires a gradient, which this call does not compute (use torch.no_grad())", name);
        if (device < 0) device = t.get_device();
        if (t.get_device() != device)
            fail(PyExc_ValueError, "%s is on device %d, the call's first tensor on device %d", name,
                 static_cast<int>(t.get_device()), device);
        return t;
    }
};

// A CUDA tensor of that type.
const at::Tensor &tensor(PyObject *o, const char *name, at::ScalarType type, Where &on)
{
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda()) fail(PyExc_TypeError, "%s must be a %s CUDA tensor", name, c10::toString(type));
    return on(t, name);
}

bool same(at::IntArrayRef a, std::initializer_list<int64_t> b)
{
    return a.size() == b.size() && std::equal(a.begin(), a.end(), b.begin());
}

// The row distance of t, whose first `lead` dimensions number rows one after
// another and whose other dimensions must be dense.
long long row_distance(const at::Tensor &t, size_t lead, std::initializer_list<int64_t> shape, const char *name)
{
    const at::IntArrayRef size = t.sizes(), stride = t.strides();
    if (!same(size, shape)) {
        char want[96];
        int at = 0;
        for (int64_t n : shape) at += std::snprintf(want + at, sizeof want - at, "[%lld]", static_cast<long long>(n));
        fail(PyExc_ValueError, "%s must be %s", name, want);
    }
    int64_t dense = 1;
    for (size_t d = size.size(); d-- > lead;) {
        if (size[d] > 1 && stride[d] != dense) fail(PyExc_ValueError, "the rows of %s must be dense", name);
        dense *= size[d];
    }
    int64_t ld = -1, span = 1;                  // span: rows that one step of dimension d passes over
    for (size_t d = lead; d-- > 0;) {
        if (size[d] == 0) return dense;         // no rows
        if (size[d] > 1) {
            if (ld < 0 ? stride[d] % span != 0 : stride[d] != ld * span)
                fail(PyExc_ValueError, "the rows of %s must be equally far apart", name);
            if (ld < 0) ld = stride[d] / span;
        }
        span *= size[d];
    }
    return ld < 0 ? dense : ld;
}

template <class T>
T *ptr(const at::Tensor &t)
{
    return static_cast<T *>(t.data_ptr());
}

const int32_t *indices(PyObject *o, const char *name, Where &on, int64_t n = -1)
{
    const at::Tensor &t = tensor(o, name, at::kInt, on);
    if (!t.is_contiguous()) fail(PyExc_TypeError, "%s must be contiguous", name);
    if (n >= 0 && t.numel() != n) fail(PyExc_ValueError, "%s must have one entry per sequence", name);
    return ptr<const int32_t>(t);
}

// A device made the current one, and the one before it again at the end.
struct Device {
    c10::DeviceIndex before = -1;               // -1: it was the current one already

    explicit Device(c10::DeviceIndex d)
    {
        if (d == c10::cuda::current_device()) return;
        before = c10::cuda::ExchangeDevice(d);
    }
    Device(const Device &) = delete;
    ~Device()
    {
        if (before >= 0) C10_CUDA_CHECK_WARN(c10::cuda::SetDevice(before));
    }
};

// The stream of a call: the given stream object's, or the current one of the
// tensor's device.  That device is the current one meanwhile (the library, and
// a launch on the default stream, go by it), and outputs allocated meanwhile
// belong to that stream.
struct Stream {
    sv_stream raw;
    Device device;
    c10::cuda::OptionalCUDAStreamGuard guard;

    Stream(PyObject *o, const at::Tensor &t) : device(t.get_device())
    {
        if (o == Py_None) {
            raw = reinterpret_cast<sv_stream>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
            return;
        }
        PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
        if (!v) throw PyFail{};
        void *p = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (PyErr_Occurred()) throw PyFail{};
        raw = reinterpret_cast<sv_stream>(p);
        guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), t.get_device()));
    }
};

at::Tensor make(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

bool truth(PyObject *o)
{
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw PyFail{};
    return r != 0;
}

double real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyFail{};
    return v;
}

int count(int64_t n, const char *what)
{
    if (n > 0x7FFFFFFF) fail(PyExc_ValueError, "too many %s", what);
    return static_cast<int>(n);
}

// A given output, or a new one.
at::Tensor output(PyObject *o, const char *name, at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type, Where &on)
{
    return o == Py_None ? make(shape, like, type) : tensor(o, name, type, on);
}

PyObject *wrap(PyObject *given, const at::Tensor &t)
{
    if (given == Py_None) return THPVariable_Wrap(t);
    Py_INCREF(given);
    return given;
}

void arguments(const char *fn, Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) fail(PyExc_TypeError, "%s takes %zd arguments", fn, want);
}

// ------------------------------------------------------------------- norm

struct NormArgs {
    const at::Tensor *x, *w, *r;
    at::Tensor ro;
    int64_t T, D;
    long long ldx, ldr = 0, ldro = 0;

    Where on;

    NormArgs(PyObject *x_, PyObject *w_, PyObject *r_) : x(nullptr), w(nullptr), r(nullptr)
    {
        x = &tensor(x_, "x", BF16, on);
        w = &tensor(w_, "weight", BF16, on);
        if (x->dim() != 2) fail(PyExc_TypeError, "x must be [T][D]");
        T = x->size(0);
        D = x->size(1);
        ldx = row_distance(*x, 1, {T, D}, "x");
        if (w->dim() != 1 || w->size(0) != D || !w->is_contiguous())
            fail(PyExc_ValueError, "weight must be contiguous with %lld entries", static_cast<long long>(D));
        if (r_ != Py_None) {
            r = &tensor(r_, "residual", BF16, on);
            ldr = row_distance(*r, 1, {T, D}, "residual");
        }
    }
    void out(PyObject *ro_)
    {
        if (!r) {
            if (ro_ != Py_None) fail(PyExc_ValueError, "residual_out without a residual");
            return;
        }
        ro = output(ro_, "residual_out", {T, D}, *x, BF16, on);
        ldro = row_distance(ro, 1, {T, D}, "residual_out");
    }
    PyObject *wrapped(PyObject *ro_) const
    {
        if (r) return wrap(ro_, ro);
        Py_RETURN_NONE;
    }
};

// (x, weight, residual, eps, unit_offset, y, residual_out, stream)
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("rmsnorm", n, 8);
        NormArgs s(a[0], a[1], a[2]);
        const Stream stream(a[7], *s.x);
        s.out(a[6]);
        const at::Tensor y = output(a[5], "y", {s.T, s.D}, *s.x, BF16, s.on);
        const long long ldy = row_distance(y, 1, {s.T, s.D}, "y");
        check_status("rmsnorm_residual",
                     rmsnorm_residual(ptr<const sv_bf16>(*s.x), s.ldx, s.r ? ptr<const sv_bf16>(*s.r) : nullptr, s.ldr,
                                      ptr<const sv_bf16>(*s.w), count(s.T, "rows"), count(s.D, "columns"),
                                      static_cast<float>(real(a[3])), truth(a[4]) ? SV_NORM_UNIT_OFFSET : 0,
                                      s.r ? ptr<sv_bf16>(s.ro) : nullptr, s.ldro, ptr<sv_bf16>(y), ldy, stream.raw));
        return Py_BuildValue("(NN)", wrap(a[5], y), s.wrapped(a[6]));
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (x, weight, residual, eps, unit_offset, group, y, scales, residual_out, stream)
PyObject *rmsnorm_fp8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("rmsnorm_fp8", n, 10);
        NormArgs s(a[0], a[1], a[2]);
        const long group = PyLong_AsLong(a[5]);
        if (group == -1 && PyErr_Occurred()) throw PyFail{};
        if (group != 0 && group != 128) fail(PyExc_ValueError, "group must be 0 or 128");
        const int64_t ns = group ? (s.D + group - 1) / group : 1;
        const Stream stream(a[9], *s.x);
        s.out(a[8]);
        const at::Tensor y = output(a[6], "y", {s.T, s.D}, *s.x, at::kFloat8_e4m3fn, s.on);
        const at::Tensor sc = output(a[7], "scales", {s.T, ns}, *s.x, F32, s.on);
        const long long ldy = row_distance(y, 1, {s.T, s.D}, "y"), lds = row_distance(sc, 1, {s.T, ns}, "scales");
        check_status("rmsnorm_residual_fp8",
                     rmsnorm_residual_fp8(ptr<const sv_bf16>(*s.x), s.ldx, s.r ? ptr<const sv_bf16>(*s.r) : nullptr,
                                          s.ldr, ptr<const sv_bf16>(*s.w), count(s.T, "rows"), count(s.D, "columns"),
                                          static_cast<float>(real(a[3])), truth(a[4]) ? SV_NORM_UNIT_OFFSET : 0,
                                          static_cast<int>(group), s.r ? ptr<sv_bf16>(s.ro) : nullptr, s.ldro,
                                          ptr<uint8_t>(y), ldy, ptr<float>(sc), lds, stream.raw));
        return Py_BuildValue("(NNN)", wrap(a[6], y), wrap(a[7], sc), s.wrapped(a[8]));
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------ gated delta rule

struct State {
    const at::Tensor *t;
    int64_t slots, Hv, dv, dk;

    State(PyObject *o, int64_t dk_, Where &on) : t(&tensor(o, "state", F32, on)), dk(dk_)
    {
        if (t->dim() != 4 || !t->is_contiguous()) fail(PyExc_TypeError, "state must be contiguous [slots][Hv][dv][dk]");
        slots = t->size(0);
        Hv = t->size(1);
        dv = t->size(2);
        if (t->size(3) != dk) fail(PyExc_ValueError, "state must be [slots][Hv][dv][%lld]", static_cast<long long>(dk));
    }
};

// sv_delta_rows of B x T rows (lead 2) or T rows (lead 1); q may be null.
sv_delta_rows delta_rows(PyObject *q, PyObject *k, PyObject *v, PyObject *g, PyObject *beta, size_t lead, int64_t B,
                         int64_t T, int64_t Hk, const State &s, Where &on)
{
    sv_delta_rows r{};
    auto take = [&](PyObject *o, const char *name, at::ScalarType type, int64_t heads, int64_t d, long long *ld) {
        const at::Tensor &t = tensor(o, name, type, on);
        if (lead == 2)
            *ld = d ? row_distance(t, 2, {B, T, heads, d}, name) : row_distance(t, 2, {B, T, heads}, name);
        else
            *ld = d ? row_distance(t, 1, {T, heads, d}, name) : row_distance(t, 1, {T, heads}, name);
        return t.data_ptr();
    };
    if (q) r.q = static_cast<const sv_bf16 *>(take(q, "q", BF16, Hk, s.dk, &r.ldq));
    r.k = static_cast<const sv_bf16 *>(take(k, "k", BF16, Hk, s.dk, &r.ldk));
    r.v = static_cast<const sv_bf16 *>(take(v, "v", BF16, s.Hv, s.dv, &r.ldv));
    long long ldb = 0;
    r.g = static_cast<const float *>(take(g, "g", F32, s.Hv, 0, &r.ldg));
    r.beta = static_cast<const float *>(take(beta, "beta", F32, s.Hv, 0, &ldb));
    if (ldb != r.ldg) fail(PyExc_ValueError, "g and beta must have the same row distance");
    return r;
}

sv_delta_shape delta_shape(int64_t Hk, const State &s, PyObject *scale, int flags)
{
    sv_delta_shape d{};
    d.Hk = count(Hk, "heads");
    d.Hv = count(s.Hv, "heads");
    d.dk = count(s.dk, "columns");
    d.dv = count(s.dv, "columns");
    d.scale = static_cast<float>(scale == Py_None ? 1.0 / std::sqrt(static_cast<double>(s.dk)) : real(scale));
    d.flags = flags;
    return d;
}

// (q, k, v, g, beta, state, state_idx, prev, accept_len, commit, scale, l2norm, o, stream)
PyObject *gated_delta_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("gated_delta_step", n, 14);
        Where on;
        const at::Tensor &k = tensor(a[1], "k", BF16, on);
        if (k.dim() != 4) fail(PyExc_TypeError, "k must be [B][T][Hk][dk]");
        const int64_t B = k.size(0), T = k.size(1), Hk = k.size(2);
        const State s(a[5], k.size(3), on);
        const sv_delta_rows rows = delta_rows(a[0], a[1], a[2], a[3], a[4], 2, B, T, Hk, s, on);
        sv_delta_rows prev{};
        int64_t P = 0;
        // the sequence that prev gave, held until the launch: an iterator's
        // tensors may have no other owner, and `o` is allocated before it
        struct Held {
            PyObject *p = nullptr;
            ~Held() { Py_XDECREF(p); }
        } held;
        if (a[7] != Py_None) {
            PyObject *f = held.p = PySequence_Fast(a[7], "prev must be (k, v, g, beta)");
            if (!f) throw PyFail{};
            if (PySequence_Fast_GET_SIZE(f) != 4) fail(PyExc_ValueError, "prev must be (k, v, g, beta)");
            PyObject **i = PySequence_Fast_ITEMS(f);
            const at::Tensor &pk = tensor(i[0], "k of prev", BF16, on);
            if (pk.dim() != 4) fail(PyExc_ValueError, "prev must be rows of the same sequences");
            P = pk.size(1);
            prev = delta_rows(nullptr, i[0], i[1], i[2], i[3], 2, B, P, Hk, s, on);
        }
        if (a[8] != Py_None && a[7] == Py_None) fail(PyExc_ValueError, "accept_len needs prev");
        const int32_t *accept = a[8] == Py_None ? nullptr : indices(a[8], "accept_len", on, B);
        const int32_t *idx = a[6] == Py_None ? nullptr : indices(a[6], "state_idx", on, B);
        const sv_delta_shape shape = delta_shape(Hk, s, a[10], (truth(a[11]) ? SV_DELTA_L2NORM : 0) | (truth(a[9]) ? SV_DELTA_COMMIT : 0));
        const Stream stream(a[13], k);
        const at::Tensor o = output(a[12], "o", {B, T, s.Hv, s.dv}, k, BF16, on);
        const long long ldo = row_distance(o, 2, {B, T, s.Hv, s.dv}, "o");
        if (B)
            check_status("gated_delta_step",
                         ::gated_delta_step(&rows, count(T, "rows"), &prev, count(P, "rows"), accept, count(B, "sequences"),
                                            &shape, ptr<float>(*s.t), idx, count(s.slots, "slots"), ptr<sv_bf16>(o), ldo,
                                            stream.raw));
        return wrap(a[12], o);
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (q, k, v, g, beta, cu_seqlens, state, state_idx, zero_init, scale, l2norm, o, workspace, stream)
PyObject *gated_delta_chunk(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("gated_delta_chunk", n, 14);
        Where on;
        const at::Tensor &k = tensor(a[1], "k", BF16, on);
        if (k.dim() != 3) fail(PyExc_TypeError, "k must be [R][Hk][dk]");
        const int64_t R = k.size(0), Hk = k.size(1);
        const State s(a[6], k.size(2), on);
        const sv_delta_rows rows = delta_rows(a[0], a[1], a[2], a[3], a[4], 1, 1, R, Hk, s, on);
        const int32_t *cu = indices(a[5], "cu_seqlens", on);
        const int64_t B = THPVariable_Unpack(a[5]).numel() - 1;
        if (B < 0) fail(PyExc_ValueError, "cu_seqlens must have B + 1 entries");
        const int32_t *idx = a[7] == Py_None ? nullptr : indices(a[7], "state_idx", on, B);
        const sv_delta_shape shape = delta_shape(Hk, s, a[9], (truth(a[10]) ? SV_DELTA_L2NORM : 0) | (truth(a[8]) ? SV_DELTA_ZERO_INIT : 0));
        const Stream stream(a[13], k);
        const at::Tensor o = output(a[11], "o", {R, s.Hv, s.dv}, k, BF16, on);
        const long long ldo = row_distance(o, 1, {R, s.Hv, s.dv}, "o");
        if (B) {
            const int r = count(R, "rows"), b = count(B, "sequences");
            at::Tensor ws;
            if (a[12] == Py_None) {
                const size_t need = gated_delta_chunk_bytes(r, b, &shape);
                ws = make({static_cast<int64_t>(need < 16 ? 16 : need)}, k, at::kByte);
            } else {
                ws = tensor(a[12], "workspace", at::kByte, on);
                if (!ws.is_contiguous()) fail(PyExc_TypeError, "workspace must be contiguous");
            }
            check_status("gated_delta_chunk",
                         ::gated_delta_chunk(&rows, r, cu, b, &shape, ptr<float>(*s.t), idx, count(s.slots, "slots"),
                                             ptr<sv_bf16>(o), ldo, ws.data_ptr(), static_cast<size_t>(ws.numel()), stream.raw));
        }
        return wrap(a[11], o);
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------- gated feed-forward

// A contiguous CUDA tensor of one of the types that hold such bits.
const at::Tensor &bits(PyObject *o, const char *name, std::initializer_list<at::ScalarType> types, Where &on)
{
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (std::find(types.begin(), types.end(), t.scalar_type()) == types.end())
        fail(PyExc_TypeError, "%s must not be %s", name, c10::toString(t.scalar_type()));
    if (!t.is_cuda() || !t.is_contiguous()) fail(PyExc_ValueError, "%s must be a contiguous CUDA tensor", name);
    return on(t, name);
}

// (x, Wq, scales, act, h, stream); act is SV_ACT_*
PyObject *w4a16_gate_up(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("w4a16_gate_up", n, 6);
        const auto b16 = {BF16, at::kShort, at::kUInt16};
        Where on;
        const at::Tensor &x = bits(a[0], "x", b16, on), &W = bits(a[1], "Wq", {at::kInt, at::kUInt32}, on),
                         &sc = bits(a[2], "scales", b16, on);
        const long act = PyLong_AsLong(a[3]);
        if (act == -1 && PyErr_Occurred()) throw PyFail{};
        if (x.dim() != 2 || W.dim() != 2) fail(PyExc_ValueError, "x must be [T][K] and Wq [2F][K/8]");
        const int64_t T = x.size(0), K = x.size(1), N = W.size(0), F = N / 2;
        if (N % 2 || W.size(1) * 8 != K || !same(sc.sizes(), {N, K / 128}))
            fail(PyExc_ValueError, "shape mismatch between x, Wq and scales");
        const Stream stream(a[5], x);
        const at::Tensor h = output(a[4], "h", {T, F}, x, BF16, on);
        if (!same(h.sizes(), {T, F}) || !h.is_contiguous()) fail(PyExc_ValueError, "h must be contiguous [T][F]");
        check_status("w4a16_gate_up",
                     ::w4a16_gate_up(ptr<const sv_bf16>(x), ptr<const uint32_t>(W), ptr<const sv_bf16>(sc), count(T, "rows"),
                                     count(K, "columns"), count(F, "columns"), static_cast<int>(act), ptr<sv_bf16>(h), stream.raw));
        return wrap(a[4], h);
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------- attention layers

// Rows of heads, [T][H][d] or [B][T][H][d]: their number and distance.
struct HeadRows {
    int64_t rows = 0, heads = 0, d = 0;
    long long ld = 0;
    const at::Tensor *t = nullptr;

    HeadRows() = default;
    HeadRows(const at::Tensor &x, const char *name) : t(&x)
    {
        if (x.dim() != 3 && x.dim() != 4) fail(PyExc_ValueError, "%s must be [T][heads][d] or [B][T][heads][d]", name);
        heads = x.size(-2);
        d = x.size(-1);
        if (x.dim() == 3) {
            rows = x.size(0);
            ld = row_distance(x, 1, {rows, heads, d}, name);
        } else {
            rows = x.size(0) * x.size(1);
            ld = row_distance(x, 2, {x.size(0), x.size(1), heads, d}, name);
        }
    }
    // Rows of the same shape as `like`, `heads` heads.
    HeadRows(const at::Tensor &x, const char *name, const at::Tensor &like, int64_t heads_) : HeadRows(x, name)
    {
        if (x.dim() != like.dim() || x.size(0) != like.size(0) || (x.dim() == 4 && x.size(1) != like.size(1)) ||
            heads != heads_ || d != like.size(-1))
            fail(PyExc_ValueError, "%s must have the same rows and dimensions", name);
    }
};

// (q, k, positions, inv_freq, axes, interleaved, factor, q_out, k_out, stream); k may be None
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("rotary", n, 10);
        Where on;
        const HeadRows q(tensor(a[0], "q", BF16, on), "q");
        const HeadRows k = a[1] == Py_None ? HeadRows() : HeadRows(tensor(a[1], "k", BF16, on), "k");
        if (k.t && (k.t->dim() != q.t->dim() || k.rows != q.rows || k.t->size(0) != q.t->size(0) || k.d != q.d))
            fail(PyExc_ValueError, "k must have the rows and dimensions of q");
        const at::Tensor &freq = tensor(a[3], "inv_freq", F32, on);
        if (freq.dim() != 1 || !freq.is_contiguous()) fail(PyExc_ValueError, "inv_freq must be contiguous [rot / 2]");
        const at::Tensor &pos = tensor(a[2], "positions", at::kInt, on);
        if (!pos.is_contiguous()) fail(PyExc_TypeError, "positions must be contiguous");
        // [axes] and the rows' dimensions, or those alone
        const int64_t lead = q.t->dim() - 2;
        if (pos.dim() != lead && pos.dim() != lead + 1) fail(PyExc_ValueError, "positions must be one for each row, or [axes] of them");
        const bool many = pos.dim() == lead + 1;
        for (int64_t i = 0; i < lead; ++i)
            if (pos.size(i + many) != q.t->size(i)) fail(PyExc_ValueError, "positions must be one for each row, or [axes] of them");
        const int64_t axes = many ? pos.size(0) : 1;
        const int32_t *axis = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor &t = tensor(a[4], "axes", at::kInt, on);
            if (!t.is_contiguous() || t.numel() != freq.numel()) fail(PyExc_ValueError, "axes must have one entry per frequency");
            axis = ptr<const int32_t>(t);
        }
        const Stream stream(a[9], *q.t);
        const at::Tensor qo = output(a[7], "q_out", q.t->sizes(), *q.t, BF16, on);
        const HeadRows to(qo, "q_out", *q.t, q.heads);
        if (!k.t && a[8] != Py_None) fail(PyExc_ValueError, "k_out without k");
        at::Tensor ko;
        HeadRows kto;
        if (k.t) {
            ko = output(a[8], "k_out", k.t->sizes(), *k.t, BF16, on);
            kto = HeadRows(ko, "k_out", *k.t, k.heads);
        }
        check_status("rotary_embed",
                     rotary_embed(ptr<const sv_bf16>(*q.t), q.ld, count(q.heads, "heads"), k.t ? ptr<const sv_bf16>(*k.t) : nullptr,
                                  k.ld, count(k.heads, "heads"), count(q.rows, "rows"), count(q.d, "dimensions"),
                                  count(2 * freq.numel(), "frequencies"), ptr<const int32_t>(pos), q.rows, count(axes, "axes"),
                                  axis, ptr<const float>(freq), static_cast<float>(real(a[6])), truth(a[5]) ? SV_ROTARY_PAIRED : 0,
                                  ptr<sv_bf16>(qo), to.ld, k.t ? ptr<sv_bf16>(ko) : nullptr, kto.ld, stream.raw));
        if (!k.t) return Py_BuildValue("(NO)", wrap(a[7], qo), Py_None);
        return Py_BuildValue("(NN)", wrap(a[7], qo), wrap(a[8], ko));
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The cache of a call, its sequences' pages and lengths.
struct Cache {
    sv_kv4_cache c{};
    const int32_t *lens = nullptr, *cu = nullptr;
    bool ragged = false;                        // cu_seqlens is given
    int64_t B = 0;

    Cache(PyObject *cache, PyObject *table, PyObject *lens_, PyObject *cu_, PyObject *k_scale, PyObject *v_scale, Where &on)
    {
        const at::Tensor &t = tensor(cache, "cache", at::kByte, on);
        if (t.dim() != 3 || !t.is_contiguous()) fail(PyExc_TypeError, "cache must be contiguous [pages][Hk][36 d]");
        if (t.size(2) % 36) fail(PyExc_ValueError, "cache must be [pages][Hk][36 d]");
        const at::Tensor &pt = tensor(table, "page_table", at::kInt, on);
        if (pt.dim() != 2) fail(PyExc_TypeError, "page_table must be [B][pages]");
        B = pt.size(0);
        c.pages = ptr<uint8_t>(t);
        c.page_table = ptr<const int32_t>(pt);
        c.ldt = row_distance(pt, 1, {B, pt.size(1)}, "page_table");
        c.n_pages = count(t.size(0), "pages");
        c.max_pages = count(pt.size(1), "pages");
        c.Hk = count(t.size(1), "heads");
        c.d = count(t.size(2) / 36, "dimensions");
        c.k_scale = static_cast<float>(real(k_scale));
        c.v_scale = static_cast<float>(real(v_scale));
        lens = indices(lens_, "seq_lens", on, B);
        if ((ragged = cu_ != Py_None)) {
            cu = indices(cu_, "cu_seqlens", on);
            if (THPVariable_Unpack(cu_).numel() != B + 1) fail(PyExc_ValueError, "cu_seqlens must have B + 1 entries");
        }
    }
    // The rows of x, [R][heads][d] with cu_seqlens, [B][T][heads][d] without.
    HeadRows rows(const at::Tensor &x, const char *name, int64_t heads) const
    {
        const HeadRows r(x, name);
        if (x.dim() != (ragged ? 3 : 4)) fail(PyExc_ValueError, "%s must be %s", name, ragged ? "[R][heads][d]" : "[B][T][heads][d]");
        if (!ragged && x.size(0) != B) fail(PyExc_ValueError, "%s must have as many sequences as page_table", name);
        if (heads >= 0 && r.heads != heads) fail(PyExc_ValueError, "%s must have the cache's heads", name);
        if (r.d != c.d) fail(PyExc_ValueError, "%s must have the cache's dimensions", name);
        return r;
    }
};

// (k, v, cache, page_table, seq_lens, cu_seqlens, k_scale, v_scale, stream)
PyObject *kv4_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("kv4_append", n, 9);
        Where on;
        const at::Tensor &k = tensor(a[0], "k", BF16, on), &v = tensor(a[1], "v", BF16, on);
        const Cache c(a[2], a[3], a[4], a[5], a[6], a[7], on);
        const HeadRows kr = c.rows(k, "k", c.c.Hk), vr = c.rows(v, "v", c.c.Hk);
        if (kr.rows != vr.rows) fail(PyExc_ValueError, "k and v must have as many rows");
        const Stream stream(a[8], k);
        check_status("kv4_append", ::kv4_append(ptr<const sv_bf16>(k), kr.ld, ptr<const sv_bf16>(v), vr.ld, count(kr.rows, "rows"),
                                                c.cu, c.lens, count(c.B, "sequences"), &c.c, stream.raw));
        Py_RETURN_NONE;
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (cache, page_table, seq_lens, rows, cu_seqlens, k_scale, v_scale, k, v, stream); rows: T, or R with cu_seqlens
PyObject *kv4_gather(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("kv4_gather", n, 10);
        Where on;
        const Cache c(a[0], a[1], a[2], a[4], a[5], a[6], on);
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const long rows = PyLong_AsLong(a[3]);
        if (rows == -1 && PyErr_Occurred()) throw PyFail{};
        if (rows < 0 || rows > 0x7FFFFFFF) fail(PyExc_ValueError, "rows must not be negative");
        const Stream stream(a[9], t);
        const int64_t four[4] = {c.B, rows, c.c.Hk, c.c.d}, three[3] = {rows, c.c.Hk, c.c.d};
        const at::IntArrayRef shape = c.ragged ? at::IntArrayRef(three, 3) : at::IntArrayRef(four, 4);
        const at::Tensor k = output(a[7], "k", shape, t, BF16, on), v = output(a[8], "v", shape, t, BF16, on);
        const HeadRows kr = c.rows(k, "k", c.c.Hk), vr = c.rows(v, "v", c.c.Hk);
        const int64_t R = c.ragged ? rows : c.B * rows;
        if (kr.rows != R || vr.rows != R) fail(PyExc_ValueError, "k and v must have as many rows");
        check_status("kv4_gather", ::kv4_gather(ptr<sv_bf16>(k), kr.ld, ptr<sv_bf16>(v), vr.ld, count(R, "rows"), c.cu, c.lens,
                                                count(c.B, "sequences"), &c.c, stream.raw));
        return Py_BuildValue("(NN)", wrap(a[7], k), wrap(a[8], v));
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (q, cache, page_table, seq_lens, cu_seqlens, scale, window, sinks, k_scale, v_scale, o, workspace, stream)
PyObject *kv4_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        arguments("kv4_attention", n, 13);
        Where on;
        const at::Tensor &q = tensor(a[0], "q", BF16, on);
        const Cache c(a[1], a[2], a[3], a[4], a[8], a[9], on);
        const HeadRows r = c.rows(q, "q", -1);
        if (r.heads < 1 || c.c.Hk < 1 || r.heads % c.c.Hk) fail(PyExc_ValueError, "the heads of q must be a multiple of the cache's");
        const long window = PyLong_AsLong(a[6]);
        if (window == -1 && PyErr_Occurred()) throw PyFail{};
        const long sinks = PyLong_AsLong(a[7]);
        if (sinks == -1 && PyErr_Occurred()) throw PyFail{};
        if (window < 0 || window > 1 << 30 || sinks < 0 || sinks > 1 << 30) fail(PyExc_ValueError, "window and sinks must be 0 .. 2^30");
        const double scale = a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.c.d)) : real(a[5]);
        const Stream stream(a[12], q);
        const at::Tensor o = output(a[10], "o", q.sizes(), q, BF16, on);
        const HeadRows to(o, "o", q, r.heads);
        const int R = count(r.rows, "rows"), B = count(c.B, "sequences"), Hq = count(r.heads, "heads");
        if (R && B) {
            at::Tensor ws;
            if (a[11] == Py_None) {
                const size_t need = kv4_attention_bytes(R, B, c.ragged, Hq, &c.c);
                ws = make({static_cast<int64_t>(need < 16 ? 16 : need)}, q, at::kByte);
            } else {
                ws = tensor(a[11], "workspace", at::kByte, on);
                if (!ws.is_contiguous()) fail(PyExc_TypeError, "workspace must be contiguous");
            }
            check_status("kv4_attention",
                         ::kv4_attention(ptr<const sv_bf16>(q), r.ld, R, Hq, c.cu, c.lens, B, &c.c, static_cast<float>(scale),
                                         static_cast<int>(window), static_cast<int>(sinks), ptr<sv_bf16>(o), to.ld, ws.data_ptr(),
                                         static_cast<size_t>(ws.numel()), stream.raw));
        }
        return wrap(a[10], o);
    } catch (const PyFail &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (SpecVerifyError)
PyObject *set_error(PyObject *, PyObject *type)
{
    Py_INCREF(type);
    Py_XSETREF(g_status_error, type);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(rmsnorm), FAST(rmsnorm_fp8), FAST(gated_delta_step), FAST(gated_delta_chunk),
                           FAST(w4a16_gate_up), FAST(rotary), FAST(kv4_append), FAST(kv4_gather), FAST(kv4_attention),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_layer", "Calls between the weight reads, on torch tensors.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&g_module); }
