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
    PRISM_CALL(verify_draft, 9),   {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
