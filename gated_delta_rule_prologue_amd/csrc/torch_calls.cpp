// torch_calls.cpp -- the Python calls of the layer operators (binding.py), as a
// CPython module: argument checks, outputs and workspaces, and the C ABI call on
// the current stream of the tensors' device.
//
// These calls are small: a decode step's norm runs 4 us on the GPU.  Checked and
// marshalled in Python through ctypes one call cost 16 to 32 us of host time,
// which bounded every serving step; here the tensors are read directly.  The
// module computes nothing.
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>

#include "prism.h"

namespace {

PyObject* prism_error = nullptr;                 // binding.PrismError

struct Raised {};                                // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& what)
{
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}

std::string text(at::IntArrayRef shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i)
        s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

std::string text(at::ScalarType t)
{
    switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    default: return std::string("torch.") + c10::toString(t);
    }
}

const at::Tensor& tensor(const char* name, PyObject* o)
{
    if (o == Py_None)
        fail(PyExc_ValueError, std::string(name) + " is required");
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The tensor that gives a call its dtype and device.
const at::Tensor& leading(const char* name, PyObject* o)
{
    const at::Tensor& t = tensor(name, o);
    if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
        fail(PyExc_TypeError, "unsupported dtype " + text(t.scalar_type()) + " (bfloat16 or float32)");
    return t;
}

int dtype_code(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? PRISM_BF16 : PRISM_F32; }

// Address of a contiguous device tensor of exactly this shape and dtype, on
// like's device.
void* arg(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like)
{
    const at::Tensor& t = tensor(name, o);
    if (t.sizes() != shape)
        fail(PyExc_ValueError, std::string(name) + ": expected shape " + text(shape) + ", got " + text(t.sizes()));
    if (t.scalar_type() != dtype)
        fail(PyExc_TypeError, std::string(name) + ": expected " + text(dtype) + ", got " + text(t.scalar_type()));
    if (t.device() != like.device())
        fail(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", not on " + like.device().str());
    if (!t.is_cuda())
        fail(PyExc_ValueError, "libprism takes device tensors");
    if (!t.is_contiguous())
        fail(PyExc_ValueError, "libprism takes contiguous tensors");
    return t.data_ptr();
}

void* opt(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like)
{
    return o == Py_None ? nullptr : arg(name, o, shape, dtype, like);
}

void on_device(const at::Tensor& like)
{
    if (!like.is_cuda())
        fail(PyExc_ValueError, "libprism takes device tensors");
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like)
{
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}

// An output: the caller's tensor if one is given, else a new one.
struct Out {
    at::Tensor t;
    void* p = nullptr;
    Out() = default;
    Out(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like)
    {
        if (o == Py_None) {
            t = fresh(shape, dtype, like);
            p = t.data_ptr();
        } else {
            p = arg(name, o, shape, dtype, like);
            t = THPVariable_Unpack(o);
        }
    }
};

void apart(const char* a, const void* pa, const char* b, const void* pb)
{
    if (pa && pa == pb)
        fail(PyExc_ValueError, std::string(a) + " and " + b + " are the same buffer");
}

// The caller's workspace, or one allocated on the current stream (none if none is needed).
struct Scratch {
    at::Tensor t;
    void* p = nullptr;
    size_t bytes = 0;
    Scratch(PyObject* o, size_t need, const at::Tensor& like)
    {
        if (o == Py_None) {
            if (need == 0)
                return;
            t = fresh({(int64_t)need}, at::kByte, like);
        } else {
            t = tensor("workspace", o);
            if (t.device() != like.device())
                fail(PyExc_ValueError,
                     "workspace is on " + t.device().str() + ", not on " + like.device().str());
            if (!t.is_contiguous())
                fail(PyExc_ValueError, "libprism takes contiguous tensors");
        }
        p = t.data_ptr();
        bytes = t.nbytes();
        if (bytes < need)
            fail(PyExc_ValueError, "workspace needs " + std::to_string(need) + " bytes");
    }
};

void done(const char* fn, prism_status s)
{
    if (s == PRISM_OK)
        return;
    PyObject* e = PyObject_CallFunction(prism_error, "si", fn, (int)s);
    if (e) {
        PyErr_SetObject(prism_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

void* stream_of(const at::Tensor& t) { return (void*)c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

PyObject* wrap(const at::Tensor& t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

// Steals nothing: a new tuple of the wrapped tensors.
template <typename... Ts> PyObject* wrap_all(const Ts&... ts)
{
    PyObject* out = PyTuple_New(sizeof...(Ts));
    if (!out)
        throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor* t : {&ts...}) {
        PyObject* o = wrap(*t);
        if (!o) {
            Py_DECREF(out);
            throw Raised{};
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

double number(PyObject* o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1. && PyErr_Occurred())
        throw Raised{};
    return x;
}

long whole(PyObject* o)
{
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred())
        throw Raised{};
    return x;
}

bool truth(PyObject* o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0)
        throw Raised{};
    return x;
}

prism_norm_dims rows_of(const at::Tensor& x)
{
    if (x.dim() < 1 || x.size(-1) < 1)
        fail(PyExc_ValueError, "rows of at least one element expected");
    if (x.size(-1) > INT32_MAX)
        fail(PyExc_ValueError, "rows of at most 2^31 - 1 elements expected");
    prism_norm_dims d;
    d.width = (int32_t)x.size(-1);
    d.rows = x.numel() / d.width;
    d.heads = 1;
    d.dtype = dtype_code(x);
    return d;
}

// With a weight a head o is [..., H, width].
prism_norm_dims gate_dims(const at::Tensor& o, const at::Tensor& w)
{
    prism_norm_dims d = rows_of(o);
    if (w.dim() == 2) {
        if (o.dim() < 2 || w.size(0) != o.size(-2) || w.size(0) < 1 || w.size(0) > INT32_MAX)
            fail(PyExc_ValueError, "w " + text(w.sizes()) + " needs " + std::to_string(w.size(0)) +
                                       " heads, o is " + text(o.sizes()));
        d.heads = (int32_t)w.size(0);
    }
    return d;
}

prism_dims dims_of(const at::Tensor& k, PyObject* v_obj, PyObject* cu_obj)
{
    const at::Tensor &v = tensor("v", v_obj), &cu = tensor("cu_seqlens", cu_obj);
    if (k.dim() != 3)
        fail(PyExc_ValueError, "q / k must be [T, H, dk]");
    if (v.dim() != 3)
        fail(PyExc_ValueError, "v must be [T, H, dv]");
    if (cu.scalar_type() != at::kInt || cu.dim() != 1 || cu.numel() < 2)
        fail(PyExc_ValueError, "cu_seqlens must be int32 [n_seqs + 1] with n_seqs >= 1");
    if (k.size(0) > INT32_MAX || k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || v.size(2) > INT32_MAX ||
        cu.numel() > INT32_MAX)
        fail(PyExc_ValueError, "a size exceeds 2^31 - 1");
    return {(int32_t)(cu.numel() - 1), (int32_t)k.size(0), (int32_t)k.size(1), (int32_t)k.size(2),
            (int32_t)v.size(2), dtype_code(k)};
}

// ---- the calls: positional arguments in the order of binding.py

PyObject* norm_residual(PyObject* const* a)
{
    const at::Tensor& x = leading("x", a[0]);
    const prism_norm_dims d = rows_of(x);
    const int64_t vec[1] = {d.width};
    const auto dt = x.scalar_type();
    const bool add = a[2] != Py_None;
    if (a[3] != Py_None && !add)
        fail(PyExc_ValueError, "scale without y");
    if (a[5] != Py_None && a[5] == a[6])
        fail(PyExc_ValueError, "r and n are the same buffer");
    on_device(x);
    const c10::DeviceGuard guard(x.device());
    void *xp = arg("x", a[0], x.sizes(), dt, x), *yp = opt("y", a[2], x.sizes(), dt, x);
    void *sp = opt("scale", a[3], vec, dt, x), *wp = arg("w", a[1], vec, dt, x);
    Out r, n("n", a[6], x.sizes(), dt, x);
    if (add || a[5] != Py_None)
        r = Out("r", a[5], x.sizes(), dt, x);
    apart("r", r.p, "n", n.p);
    done("prism_norm_residual", prism_norm_residual(&d, xp, yp, sp, wp, (float)number(a[4]), r.p, n.p, stream_of(x)));
    return wrap_all(n.t, r.t.defined() ? r.t : x);
}

PyObject* norm_residual_bwd(PyObject* const* a)
{
    const at::Tensor& r = leading("r", a[0]);
    const prism_norm_dims d = rows_of(r);
    const int64_t vec[1] = {d.width};
    const auto dt = r.scalar_type();
    const bool scaled = a[5] != Py_None;
    if (scaled && a[4] == Py_None)
        fail(PyExc_ValueError, "scale without y");
    on_device(r);
    const c10::DeviceGuard guard(r.device());
    void *rp = arg("r", a[0], r.sizes(), dt, r), *wp = arg("w", a[1], vec, dt, r);
    void *dnp = arg("dn", a[2], r.sizes(), dt, r), *drp = opt("dr", a[3], r.sizes(), dt, r);
    void *yp = opt("y", a[4], r.sizes(), dt, r), *sp = opt("scale", a[5], vec, dt, r);
    at::Tensor dx = fresh(r.sizes(), dt, r), dw = fresh(vec, at::kFloat, r), dy, ds;
    if (scaled) {
        dy = fresh(r.sizes(), dt, r);
        if (truth(a[8]))
            ds = fresh(vec, at::kFloat, r);
    }
    const Scratch ws(a[7], prism_norm_workspace_bytes(&d), r);
    done("prism_norm_residual_bwd",
         prism_norm_residual_bwd(&d, rp, yp, sp, wp, (float)number(a[6]), dnp, drp, dx.data_ptr(),
                                 dy.defined() ? dy.data_ptr() : nullptr, dw.data_ptr<float>(),
                                 ds.defined() ? ds.data_ptr<float>() : nullptr, ws.p, ws.bytes, stream_of(r)));
    if (!scaled && a[4] != Py_None)
        dy = dx;
    return wrap_all(dx, dy, dw, ds);
}

PyObject* norm_gate(PyObject* const* a)
{
    const at::Tensor &o = leading("o", a[0]), &w = tensor("w", a[2]);
    const prism_norm_dims d = gate_dims(o, w);
    const int64_t wshape[2] = {d.heads, d.width};
    const auto dt = o.scalar_type();
    on_device(o);
    const c10::DeviceGuard guard(o.device());
    void *op = arg("o", a[0], o.sizes(), dt, o), *zp = arg("z", a[1], o.sizes(), dt, o);
    void* wp = arg("w", a[2], w.dim() == 2 ? at::IntArrayRef(wshape, 2) : at::IntArrayRef(wshape + 1, 1), dt, o);
    Out y("y", a[5], o.sizes(), dt, o);
    done("prism_norm_gate",
         prism_norm_gate(&d, op, zp, wp, (float)number(a[3]), (int)whole(a[4]), y.p, stream_of(o)));
    return wrap(y.t);
}

PyObject* norm_gate_bwd(PyObject* const* a)
{
    const at::Tensor &o = leading("o", a[0]), &w = tensor("w", a[2]);
    const prism_norm_dims d = gate_dims(o, w);
    const int64_t wshape[2] = {d.heads, d.width};
    const auto ws_shape = w.dim() == 2 ? at::IntArrayRef(wshape, 2) : at::IntArrayRef(wshape + 1, 1);
    const auto dt = o.scalar_type();
    on_device(o);
    const c10::DeviceGuard guard(o.device());
    void *op = arg("o", a[0], o.sizes(), dt, o), *zp = arg("z", a[1], o.sizes(), dt, o);
    void *wp = arg("w", a[2], ws_shape, dt, o), *dyp = arg("dy", a[3], o.sizes(), dt, o);
    at::Tensor d_o = fresh(o.sizes(), dt, o), dz = fresh(o.sizes(), dt, o), dw = fresh(ws_shape, at::kFloat, o);
    const Scratch ws(a[6], prism_norm_workspace_bytes(&d), o);
    done("prism_norm_gate_bwd",
         prism_norm_gate_bwd(&d, op, zp, wp, (float)number(a[4]), (int)whole(a[5]), dyp, d_o.data_ptr(),
                             dz.data_ptr(), dw.data_ptr<float>(), ws.p, ws.bytes, stream_of(o)));
    return wrap_all(d_o, dz, dw);
}

PyObject* decode_draft(PyObject* const* a)
{
    const at::Tensor& q = leading("q", a[0]);
    const prism_dims d = dims_of(q, a[2], a[9]);
    const int64_t n = d.n_seqs, T = d.total_tokens, H = d.heads, dk = d.dk, dv = d.dv, L = whole(a[10]);
    const int64_t tk[3] = {T, H, dk}, tv[3] = {T, H, dv}, th[2] = {T, H}, lev[4] = {T, H, L - 1, dk};
    const int64_t cw[3] = {H, dk, 4}, cu[1] = {n + 1}, state[4] = {n, H, dk, dv}, hist[4] = {n, H, 3, dk};
    const auto dt = q.scalar_type();
    on_device(q);
    const c10::DeviceGuard guard(q.device());
    void *qp = arg("q", a[0], tk, dt, q), *kp = arg("k", a[1], tk, dt, q), *vp = arg("v", a[2], tv, dt, q);
    void *up = nullptr, *ap = nullptr, *hp = nullptr;
    if (L > 1) {
        up = arg("u", a[3], lev, dt, q);
        ap = arg("a", a[6], lev, dt, q);
        hp = arg("h", a[7], lev, dt, q);
    }
    void *gp = arg("g", a[4], th, dt, q), *bp = arg("b", a[5], th, dt, q);
    void *cwp = arg("conv_w", a[8], cw, dt, q), *cup = arg("cu_seqlens", a[9], cu, at::kInt, q);
    void *Sp = arg("S", a[11], state, at::kFloat, q), *hip = arg("k_hist", a[12], hist, dt, q);
    Out o("o", a[13], tv, dt, q), kw("kw", a[14], tk, at::kFloat, q), p("p", a[15], tv, at::kFloat, q);
    apart("o", o.p, "kw", kw.p);
    apart("o", o.p, "p", p.p);
    apart("kw", kw.p, "p", p.p);
    done("prism_decode_draft",
         prism_decode_draft(&d, qp, kp, vp, up, gp, bp, ap, hp, cwp, (const int32_t*)cup, (int)L, (int)whole(a[16]),
                            (const float*)Sp, hip, o.p, (float*)kw.p, (float*)p.p, stream_of(q)));
    return wrap_all(o.t, kw.t, p.t);
}

PyObject* decode_commit(PyObject* const* a)
{
    const at::Tensor& k = leading("k", a[0]);
    const prism_dims d = dims_of(k, a[1], a[4]);
    const int64_t n = d.n_seqs, T = d.total_tokens, H = d.heads, dk = d.dk, dv = d.dv;
    const int64_t tk[3] = {T, H, dk}, tv[3] = {T, H, dv}, th[2] = {T, H}, cu[1] = {n + 1}, nn[1] = {n};
    const int64_t state[4] = {n, H, dk, dv}, hist[4] = {n, H, 3, dk};
    const auto dt = k.scalar_type();
    on_device(k);
    const c10::DeviceGuard guard(k.device());
    void *kp = arg("k", a[0], tk, dt, k), *vp = arg("v", a[1], tv, dt, k), *gp = arg("g", a[2], th, dt, k);
    void *bp = arg("b", a[3], th, dt, k), *cup = arg("cu_seqlens", a[4], cu, at::kInt, k);
    void *np = arg("n_accept", a[5], nn, at::kInt, k), *kwp = arg("kw", a[6], tk, at::kFloat, k);
    void *pp = arg("p", a[7], tv, at::kFloat, k), *Sp = arg("S", a[8], state, at::kFloat, k);
    void* hp = arg("k_hist", a[9], hist, dt, k);
    // in place unless another buffer is given
    void* So = a[10] == Py_None ? Sp : arg("S_out", a[10], state, at::kFloat, k);
    void* ho = a[11] == Py_None ? hp : arg("k_hist_out", a[11], hist, dt, k);
    done("prism_decode_commit",
         prism_decode_commit(&d, kp, vp, gp, bp, (const int32_t*)cup, (const int32_t*)np, (const float*)kwp,
                             (const float*)pp, (const float*)Sp, hp, (float*)So, ho, stream_of(k)));
    return Py_BuildValue("OO", a[10] == Py_None ? a[8] : a[10], a[11] == Py_None ? a[9] : a[11]);
}

PyObject* verify_draft(PyObject* const* a)
{
    const at::Tensor &p = leading("p", a[0]), &cu = tensor("cu_seqlens", a[2]);
    if (p.dim() != 2 || p.size(0) > INT32_MAX || p.size(1) > INT32_MAX)
        fail(PyExc_ValueError, "p must be [T, vocab]");
    if (cu.dim() != 1 || cu.numel() < 2 || cu.numel() > INT32_MAX)
        fail(PyExc_ValueError, "cu_seqlens must be int32 [n_seqs + 1] with n_seqs >= 1");
    const int64_t n = cu.numel() - 1, T = p.size(0), nn[1] = {n}, n1[1] = {n + 1}, tt[1] = {T};
    const prism_verify_dims d = {(int32_t)n, (int32_t)T, (int32_t)p.size(1), dtype_code(p)};
    const auto dt = p.scalar_type();
    if (a[6] != Py_None && a[6] == a[7])
        fail(PyExc_ValueError, "n_accept and next_token are the same buffer");
    on_device(p);
    const c10::DeviceGuard guard(p.device());
    void *pp = arg("p", a[0], p.sizes(), dt, p), *qp = opt("q", a[5], p.sizes(), dt, p);
    void *tp = arg("tokens", a[1], tt, at::kInt, p), *cup = arg("cu_seqlens", a[2], n1, at::kInt, p);
    void *ua = arg("u_accept", a[3], tt, at::kFloat, p), *us = arg("u_sample", a[4], nn, at::kFloat, p);
    Out na("n_accept", a[6], nn, at::kInt, p), nt("next_token", a[7], nn, at::kInt, p);
    apart("n_accept", na.p, "next_token", nt.p);
    const Scratch ws(a[8], prism_verify_workspace_bytes(&d), p);
    done("prism_verify_draft",
         prism_verify_draft(&d, pp, qp, (const int32_t*)tp, (const int32_t*)cup, (const float*)ua, (const float*)us,
                            (int32_t*)na.p, (int32_t*)nt.p, ws.p, ws.bytes, stream_of(p)));
    return wrap_all(na.t, nt.t);
}

// Address of a device tensor of this dtype on like's device whose last axis is dense; its
// other strides are the caller's to read.
void* strided(const char* name, const at::Tensor& t, at::ScalarType dtype, const at::Tensor& like)
{
    if (t.scalar_type() != dtype)
        fail(PyExc_TypeError, std::string(name) + ": expected " + text(dtype) + ", got " + text(t.scalar_type()));
    if (t.device() != like.device())
        fail(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", not on " + like.device().str());
    if (t.size(-1) > 1 && t.stride(-1) != 1)
        fail(PyExc_ValueError, std::string(name) + ": the last axis must be contiguous");
    return t.data_ptr();
}

int32_t size32(const char* what, int64_t n)
{
    if (n > INT32_MAX)
        fail(PyExc_ValueError, std::string(what) + " exceeds 2^31 - 1");
    return (int32_t)n;
}

// x [T, C] with any row stride, w [C, K]; n_seqs sequences.
prism_conv_dims conv_dims(const at::Tensor& x, PyObject* w_obj, int64_t n_seqs)
{
    const at::Tensor& w = tensor("w", w_obj);
    if (x.dim() != 2 || x.size(1) < 1)
        fail(PyExc_ValueError, "x must be [T, channels]");
    if (w.dim() != 2 || w.size(0) != x.size(1) || w.size(1) < 1)
        fail(PyExc_ValueError, "w must be [channels, taps], got " + text(w.sizes()));
    prism_conv_dims d;
    d.n_seqs = size32("the number of sequences", n_seqs);
    d.total_tokens = size32("the number of tokens", x.size(0));
    d.channels = size32("channels", x.size(1));
    d.taps = size32("taps", w.size(1));
    d.dtype = dtype_code(x);
    d.x_stride = x.stride(0);
    return d;
}

int64_t sequences(PyObject* o)
{
    const at::Tensor& cu = tensor("cu_seqlens", o);
    if (cu.scalar_type() != at::kInt || cu.dim() != 1 || cu.numel() < 2)
        fail(PyExc_ValueError, "cu_seqlens must be int32 [n_seqs + 1] with n_seqs >= 1");
    return cu.numel() - 1;
}

// x, w, cu_seqlens, bias, activation, hist, hist_out, y
PyObject* short_conv(PyObject* const* a)
{
    const at::Tensor& x = leading("x", a[0]);
    const prism_conv_dims d = conv_dims(x, a[1], sequences(a[2]));
    const int64_t C = d.channels, n1[1] = {(int64_t)d.n_seqs + 1}, vec[1] = {C}, w[2] = {C, d.taps};
    const int64_t hist[3] = {d.n_seqs, d.taps - 1, C};
    const auto dt = x.scalar_type();
    on_device(x);
    const c10::DeviceGuard guard(x.device());
    void *xp = strided("x", x, dt, x), *wp = arg("w", a[1], w, dt, x), *cup = arg("cu_seqlens", a[2], n1, at::kInt, x);
    void *bp = opt("bias", a[3], vec, dt, x), *hp = opt("hist", a[5], hist, dt, x);
    void* ho = opt("hist_out", a[6], hist, dt, x);
    Out y("y", a[7], x.sizes(), dt, x);
    done("prism_short_conv_ex",                      // a new y holds anything: its rows behind the last sequence too are written
         prism_short_conv_ex(&d, xp, wp, bp, hp, (const int32_t*)cup, (int)whole(a[4]), a[7] == Py_None, y.p, ho,
                             stream_of(x)));
    return wrap(y.t);
}

// x, w, hist, bias, activation, hist_out, y
PyObject* short_conv_step(PyObject* const* a)
{
    const at::Tensor& x = leading("x", a[0]);
    if (x.dim() != 2 || x.size(0) < 1)
        fail(PyExc_ValueError, "x must be [n_seqs, channels] with n_seqs >= 1");
    const prism_conv_dims d = conv_dims(x, a[1], x.size(0));
    const int64_t C = d.channels, vec[1] = {C}, w[2] = {C, d.taps}, hist[3] = {d.n_seqs, d.taps - 1, C};
    const auto dt = x.scalar_type();
    on_device(x);
    const c10::DeviceGuard guard(x.device());
    void *xp = strided("x", x, dt, x), *wp = arg("w", a[1], w, dt, x), *hp = arg("hist", a[2], hist, dt, x);
    void* bp = opt("bias", a[3], vec, dt, x);
    void* ho = a[5] == Py_None ? hp : arg("hist_out", a[5], hist, dt, x);        // in place unless another is given
    Out y("y", a[6], x.sizes(), dt, x);
    done("prism_short_conv_step", prism_short_conv_step(&d, xp, wp, bp, hp, (int)whole(a[4]), y.p, ho, stream_of(x)));
    return wrap(y.t);
}

// x, w, cu_seqlens, dy, bias, activation, hist, workspace, want_dhist
PyObject* short_conv_bwd(PyObject* const* a)
{
    const at::Tensor& x = leading("x", a[0]);
    const prism_conv_dims d = conv_dims(x, a[1], sequences(a[2]));
    const int64_t C = d.channels, n1[1] = {(int64_t)d.n_seqs + 1}, vec[1] = {C}, w[2] = {C, d.taps};
    const int64_t hist[3] = {d.n_seqs, d.taps - 1, C};
    const auto dt = x.scalar_type();
    on_device(x);
    const c10::DeviceGuard guard(x.device());
    void *xp = strided("x", x, dt, x), *wp = arg("w", a[1], w, dt, x), *cup = arg("cu_seqlens", a[2], n1, at::kInt, x);
    void *dyp = arg("dy", a[3], x.sizes(), dt, x), *bp = opt("bias", a[4], vec, dt, x);
    void* hp = opt("hist", a[6], hist, dt, x);
    at::Tensor dx = fresh(x.sizes(), dt, x), dw = fresh(w, at::kFloat, x), db, dh;
    if (bp)
        db = fresh(vec, at::kFloat, x);
    if (a[6] != Py_None && truth(a[8]))
        dh = fresh(hist, dt, x);
    const Scratch ws(a[7], prism_conv_workspace_bytes(&d), x);
    done("prism_short_conv_bwd",
         prism_short_conv_bwd(&d, xp, wp, bp, hp, (const int32_t*)cup, (int)whole(a[5]), dyp, dx.data_ptr(),
                              dw.data_ptr<float>(), db.defined() ? db.data_ptr<float>() : nullptr,
                              dh.defined() ? dh.data_ptr() : nullptr, ws.p, ws.bytes, stream_of(x)));
    return wrap_all(dx, dw, db, dh);
}

// What both passes of qk_norm read: q, k, wq, wk, positions, freqs.
struct QkInputs {
    prism_qk_dims d;
    const at::Tensor& q;
    const at::Tensor* k = nullptr;
    void *qp, *kp = nullptr, *wq, *wk = nullptr, *pos = nullptr, *freqs = nullptr;

    QkInputs(PyObject* qo, PyObject* ko, PyObject* wqo, PyObject* wko, PyObject* po, PyObject* fo) : q(leading("q", qo))
    {
        if (q.dim() != 3 || q.size(1) < 1 || q.size(2) < 1)
            fail(PyExc_ValueError, "q must be [T, heads, width]");
        const auto dt = q.scalar_type();
        on_device(q);
        d = {};
        d.tokens = q.size(0);
        d.heads_q = size32("heads", q.size(1));
        d.width = size32("width", q.size(2));
        d.dtype = dtype_code(q);
        d.q_stride = q.stride(0);
        d.q_head_stride = q.stride(1);
        qp = strided("q", q, dt, q);
        const int64_t vec[1] = {d.width}, t[1] = {d.tokens};
        wq = opt("wq", wqo, vec, dt, q);
        if (ko != Py_None) {
            k = &tensor("k", ko);
            if (k->dim() != 3 || k->size(0) != q.size(0) || k->size(1) < 1 || k->size(2) != q.size(2))
                fail(PyExc_ValueError, "k must be [T, heads, width] with q's T and width, got " + text(k->sizes()));
            d.heads_k = size32("heads", k->size(1));
            d.k_stride = k->stride(0);
            d.k_head_stride = k->stride(1);
            kp = strided("k", *k, dt, q);
            wk = opt("wk", wko, vec, dt, q);
            if (!wq != !wk)
                fail(PyExc_ValueError, "wq and wk come together");
        } else if (wko != Py_None) {
            fail(PyExc_ValueError, "wk without k");
        }
        if ((po == Py_None) != (fo == Py_None))
            fail(PyExc_ValueError, "positions and freqs come together");
        if (po != Py_None) {
            const at::Tensor& f = tensor("freqs", fo);
            if (f.dim() != 1 || 2 * f.numel() > d.width)
                fail(PyExc_ValueError, "freqs must be [rot / 2] with rot <= width, got " + text(f.sizes()));
            d.rot = (int32_t)(2 * f.numel());
            pos = arg("positions", po, t, at::kInt, q);
            freqs = arg("freqs", fo, f.sizes(), at::kFloat, q);
        }
    }
};

// q, k, wq, wk, norm, eps, positions, freqs, layout, rot_scale, q_out, k_out
PyObject* qk_norm(PyObject* const* a)
{
    const at::Tensor& q = leading("q", a[0]);
    on_device(q);
    const c10::DeviceGuard guard(q.device());
    const QkInputs in(a[0], a[1], a[2], a[3], a[6], a[7]);
    Out qo("q_out", a[10], q.sizes(), q.scalar_type(), q), ko;
    if (in.k)
        ko = Out("k_out", a[11], in.k->sizes(), q.scalar_type(), q);
    else if (a[11] != Py_None)
        fail(PyExc_ValueError, "k_out without k");
    done("prism_qk_norm",
         prism_qk_norm(&in.d, in.qp, in.kp, in.wq, in.wk, (int)whole(a[4]), (float)number(a[5]), (const int32_t*)in.pos,
                       (const float*)in.freqs, (int)whole(a[8]), (float)number(a[9]), qo.p, ko.p, stream_of(q)));
    return wrap_all(qo.t, ko.t);
}

// q, dq_out, k, dk_out, wq, wk, norm, eps, positions, freqs, layout, rot_scale, workspace
PyObject* qk_norm_bwd(PyObject* const* a)
{
    const at::Tensor& q = leading("q", a[0]);
    on_device(q);
    const c10::DeviceGuard guard(q.device());
    const QkInputs in(a[0], a[2], a[4], a[5], a[8], a[9]);
    const auto dt = q.scalar_type();
    const int64_t vec[1] = {in.d.width};
    void *dqo = arg("dq_out", a[1], q.sizes(), dt, q), *dko = nullptr;
    at::Tensor dq = fresh(q.sizes(), dt, q), dk, dwq, dwk;
    if (in.k) {
        dko = arg("dk_out", a[3], in.k->sizes(), dt, q);
        dk = fresh(in.k->sizes(), dt, q);
    } else if (a[3] != Py_None) {
        fail(PyExc_ValueError, "dk_out without k");
    }
    if (in.wq)
        dwq = fresh(vec, at::kFloat, q);
    if (in.wk)
        dwk = fresh(vec, at::kFloat, q);
    const Scratch ws(a[12], in.wq ? prism_qk_workspace_bytes(&in.d) : 0, q);
    done("prism_qk_norm_bwd",
         prism_qk_norm_bwd(&in.d, in.qp, in.kp, in.wq, in.wk, (int)whole(a[6]), (float)number(a[7]),
                           (const int32_t*)in.pos, (const float*)in.freqs, (int)whole(a[10]), (float)number(a[11]), dqo,
                           dko, dq.data_ptr(), dk.defined() ? dk.data_ptr() : nullptr,
                           dwq.defined() ? dwq.data_ptr<float>() : nullptr,
                           dwk.defined() ? dwk.data_ptr<float>() : nullptr, ws.p, ws.bytes, stream_of(q)));
    return wrap_all(dq, dk, dwq, dwk);
}

// logits, u, temperature, top_k, top_p, min_p, want_probs, tokens, probs, workspace
PyObject* sample(PyObject* const* a)
{
    const at::Tensor& l = leading("logits", a[0]);
    if (l.dim() != 2 || l.size(1) < 1)
        fail(PyExc_ValueError, "logits must be [rows, vocab]");
    on_device(l);
    const c10::DeviceGuard guard(l.device());
    const int64_t rows[1] = {l.size(0)};
    prism_sample_dims d;
    d.rows = l.size(0);
    d.vocab = size32("vocab", l.size(1));
    d.dtype = dtype_code(l);
    d.stride = l.stride(0);
    void *lp = strided("logits", l, l.scalar_type(), l), *up = opt("u", a[1], rows, at::kFloat, l);
    void *tp = opt("temperature", a[2], rows, at::kFloat, l), *kp = opt("top_k", a[3], rows, at::kInt, l);
    void *pp = opt("top_p", a[4], rows, at::kFloat, l), *mp = opt("min_p", a[5], rows, at::kFloat, l);
    const bool want_probs = a[8] != Py_None || truth(a[6]);
    if (a[1] == Py_None && a[7] != Py_None)
        fail(PyExc_ValueError, "tokens without u");
    if (a[1] == Py_None && !want_probs)
        fail(PyExc_ValueError, "u (for tokens) or want_probs is required");
    Out tokens, probs;
    if (a[1] != Py_None)
        tokens = Out("tokens", a[7], rows, at::kInt, l);
    if (want_probs)
        probs = Out("probs", a[8], l.sizes(), at::kFloat, l);
    const Scratch ws(a[9], prism_sample_workspace_bytes(&d), l);
    done("prism_sample",
         prism_sample(&d, lp, (const float*)tp, (const int32_t*)kp, (const float*)pp, (const float*)mp,
                      (const float*)up, (int32_t*)tokens.p, (float*)probs.p, ws.p, ws.bytes, stream_of(l)));
    return wrap_all(tokens.t, probs.t);
}

// No C++ exception leaves the module: torch's become their Python exceptions.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, count);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls)
{
    Py_INCREF(cls);
    Py_XSETREF(prism_error, cls);
    Py_RETURN_NONE;
}

#define PRISM_CALL(f, n) {#f, (PyCFunction)(void (*)())(call<f, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PRISM_CALL(norm_residual, 7),  PRISM_CALL(norm_residual_bwd, 9), PRISM_CALL(norm_gate, 6),
    PRISM_CALL(norm_gate_bwd, 7),  PRISM_CALL(decode_draft, 17),     PRISM_CALL(decode_commit, 12),
    PRISM_CALL(verify_draft, 9),   PRISM_CALL(short_conv, 8),        PRISM_CALL(short_conv_step, 7),
    PRISM_CALL(short_conv_bwd, 9), PRISM_CALL(qk_norm, 12),          PRISM_CALL(qk_norm_bwd, 13),
    PRISM_CALL(sample, 10),        {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
