"""torch.autograd wrapper of the operator: the forward runs prism_fwd_ckpt where
the chunkwise backward serves the shape (keeping every chunk's start state for
the backward, prism_bwd_ckpt, which stores the token-sized gradients of bf16
inputs in bf16 directly), else prism_fwd_resume and prism_bwd_ex (all in
libprism; nothing is computed here except casting the remaining fp32 gradients
to each input's dtype).

    o, S_final = prism(q, k, v, u, g, b, a, h, conv_w, cu_seqlens, L,
                       S_init=None, residual="linear")

Gradients flow to q, k, v, u, g, b, a, h, conv_w and S_init (fp32), for the
upstream gradients of o and S_final (either may be unused).  The carried
convolution history of prism_fwd_resume is not taken: the backward entry point
differentiates sequences that start with a zero history.

The norms around the operator, differentiable in every tensor they take:

    n, r = norm_residual(x, w, y=None, scale=None, eps=1e-6)
    y = norm_gate(o, z, w, eps=1e-6, gate="silu")

The steps in front of it, differentiable in x, w, bias and hist, and in q, k, wq and wk:

    y = short_conv(x, w, cu_seqlens, bias=None, activation="silu", hist=None)
    q, k = qk_norm(q, k, wq=None, wk=None, norm="l2", ...)
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding

_INPUTS = ("q", "k", "v", "u", "g", "b", "a", "h", "conv_w")


def _aligned(t):
    """t as the kernels take it: contiguous, from an address that is a multiple of 16 (autograd
    hands out slices, as for a concatenation, that begin at any element)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _upstream(grad, like):
    """An upstream gradient as the kernels take it, or None."""
    return None if grad is None else _aligned(grad.to(like.dtype))


class PrismFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, u, g, b, a, h, conv_w, cu_seqlens, L, S_init, residual):
        ckpt = None
        if binding.checkpoint_bytes(binding._dims_of(q, v, cu_seqlens)) > 0:
            try:
                o, S_final, ckpt = binding.fwd_ckpt(q, k, v, u, g, b, a, h, conv_w, cu_seqlens, L,
                                                    S_init=S_init, residual=residual)
            except binding.PrismError as err:        # the environment selects another scan
                if err.status != binding.PRISM_EUNSUPPORTED:
                    raise
        if ckpt is None:
            o, S_final, _ = binding.fwd_resume(q, k, v, u, g, b, a, h, conv_w, cu_seqlens, L,
                                               S_init=S_init, residual=residual)
        ctx.save_for_backward(q, k, v, u, g, b, a, h, conv_w, cu_seqlens, S_init, ckpt)
        ctx.L, ctx.residual = L, residual
        ctx.has_s_init = S_init is not None
        return o, S_final

    @staticmethod
    def backward(ctx, d_o, d_s):
        q, k, v, u, g, b, a, h, conv_w, cu_seqlens, S_init, ckpt = ctx.saved_tensors
        if not ctx.has_s_init:
            S_init = None
        d_o = torch.zeros_like(v) if d_o is None else _upstream(d_o, v)
        d_s = None if d_s is None else _aligned(d_s.to(torch.float32))
        want_s = ctx.has_s_init and ctx.needs_input_grad[11]
        args = (q, k, v, u, g, b, a, h, conv_w, cu_seqlens, ctx.L, d_o)
        kw = dict(dS_final=d_s, S_init=S_init, want_dS_init=want_s, residual=ctx.residual)
        grads = None
        if ckpt is not None:
            try:
                gdt = torch.bfloat16 if q.dtype == torch.bfloat16 else None
                grads = binding.bwd(*args, checkpoints=ckpt, grad_dtype=gdt, **kw)
            except binding.PrismError as err:        # PRISM_BWD_CHUNKED=0 since the forward
                if err.status != binding.PRISM_EUNSUPPORTED:
                    raise
        if grads is None:
            grads = binding.bwd(*args, **kw)
        src = dict(zip(_INPUTS, (q, k, v, u, g, b, a, h, conv_w)))
        out = []
        for i, name in enumerate(_INPUTS):
            gr = grads[name]
            out.append(None if gr is None or not ctx.needs_input_grad[i] else gr.to(src[name].dtype))
        return (*out, None, None, grads["S_init"] if want_s else None, None)


def prism(q, k, v, u, g, b, a, h, conv_w, cu_seqlens, L: int, S_init=None, residual="linear"):
    """Differentiable forward pass: returns (o, S_final)."""
    return PrismFunction.apply(q, k, v, u, g, b, a, h, conv_w, cu_seqlens, L, S_init, residual)


class NormResidualFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, y, scale, eps):
        ctx.set_materialize_grads(False)
        n, r = binding.norm_residual(x, w, y=y, scale=scale, eps=eps)
        ctx.save_for_backward(r, w, y if scale is not None else None, scale)
        ctx.eps, ctx.has_y = eps, y is not None
        if y is None:                        # r is x itself: only n is an output of this step
            return n
        return n, r

    @staticmethod
    @once_differentiable
    def backward(ctx, dn, dr=None):
        r, w, y, scale = ctx.saved_tensors
        if dn is None and dr is None:
            return None, None, None, None, None
        dn = torch.zeros_like(r) if dn is None else _upstream(dn, r)
        grads = binding.norm_residual_bwd(r, w, dn, dr=_upstream(dr, r), y=y, scale=scale, eps=ctx.eps,
                                          want_dscale=ctx.needs_input_grad[3])
        want = ctx.needs_input_grad
        dy = (grads["x"] if scale is None else grads["y"]) if ctx.has_y and want[2] else None
        return (grads["x"] if want[0] else None, grads["w"].to(w.dtype) if want[1] else None, dy,
                grads["scale"].to(scale.dtype) if want[3] else None, None)


def norm_residual(x, w, y=None, scale=None, eps: float = 1e-6):
    """Differentiable binding.norm_residual: returns (n, r)."""
    if y is None:
        if scale is not None:
            raise ValueError("scale without y")
        return NormResidualFunction.apply(x, w, None, None, eps), x
    return NormResidualFunction.apply(x, w, y, scale, eps)


class NormGateFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, z, w, eps, gate):
        y = binding.norm_gate(o, z, w, eps=eps, gate=gate)
        ctx.save_for_backward(o, z, w)
        ctx.eps, ctx.gate = eps, gate
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        o, z, w = ctx.saved_tensors
        grads = binding.norm_gate_bwd(o, z, w, _upstream(dy, o), eps=ctx.eps, gate=ctx.gate)
        want = ctx.needs_input_grad
        return (grads["o"] if want[0] else None, grads["z"] if want[1] else None,
                grads["w"].to(w.dtype) if want[2] else None, None, None)


def norm_gate(o, z, w, eps: float = 1e-6, gate: str = "silu"):
    """Differentiable binding.norm_gate: returns y."""
    return NormGateFunction.apply(o, z, w, eps, gate)


class ShortConvFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, hist, cu_seqlens, activation):
        y, _ = binding.short_conv(x, w, cu_seqlens, bias=bias, activation=activation, hist=hist)
        # a copy: histories are moved on in place, as a rule before the backward
        ctx.save_for_backward(x, w, bias, None if hist is None else hist.clone(), cu_seqlens)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, bias, hist, cu_seqlens = ctx.saved_tensors
        want = ctx.needs_input_grad
        grads = binding.short_conv_bwd(x, w, cu_seqlens, _upstream(dy, x), bias=bias, activation=ctx.activation,
                                       hist=hist, want_dhist=want[3])
        return (grads["x"] if want[0] else None, grads["w"].to(w.dtype) if want[1] else None,
                grads["bias"].to(bias.dtype) if want[2] else None, grads["hist"] if want[3] else None, None, None)


def short_conv(x, w, cu_seqlens, bias=None, activation="silu", hist=None):
    """Differentiable binding.short_conv: returns y, zero behind the last sequence.  No gradient reaches ``hist`` from a history
    carried out: sequences cut into pieces are trained piece by piece, and ``hist`` may be moved on to the
    next piece (binding.short_conv with hist_out=hist) before this one's backward."""
    return ShortConvFunction.apply(x, w, bias, hist, cu_seqlens, activation)


class QkNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, positions, freqs, how):
        q_out, k_out = binding.qk_norm(q, k, wq, wk, positions=positions, freqs=freqs, **how)
        ctx.save_for_backward(q, k, wq, wk, positions, freqs)
        ctx.how = how
        return q_out if k is None else (q_out, k_out)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        q, k, wq, wk, positions, freqs = ctx.saved_tensors
        grads = binding.qk_norm_bwd(q, _upstream(dq, q), k, None if k is None else _upstream(dk, k), wq, wk,
                                    positions=positions, freqs=freqs, **ctx.how)
        want = ctx.needs_input_grad
        return (grads["q"] if want[0] else None, grads["k"] if want[1] else None,
                grads["wq"].to(wq.dtype) if want[2] else None, grads["wk"].to(wk.dtype) if want[3] else None,
                None, None, None)


def qk_norm(q, k=None, wq=None, wk=None, norm="l2", eps: float = 1e-6, positions=None, freqs=None, layout="half",
            rot_scale: float = 1.0):
    """Differentiable binding.qk_norm: returns (q, k).  Frequencies take no gradient."""
    if freqs is not None and freqs.requires_grad:
        raise ValueError("no gradient is formed for freqs")
    how = dict(norm=norm, eps=eps, layout=layout, rot_scale=rot_scale)
    if k is None:
        return QkNormFunction.apply(q, None, wq, wk, positions, freqs, how), None
    return QkNormFunction.apply(q, k, wq, wk, positions, freqs, how)
