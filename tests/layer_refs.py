"""Plain 64-bit references of the layer operators (norms, drafted tokens,
verification), written from their formulas with numpy and torch on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch

EPS32 = 2.0 ** -24                       # half a step of fp32, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: EPS32}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def norm_residual(x, w, y, scale, eps):
    """(n, r) and the magnitudes that their rounding errors scale with."""
    add = 0 if y is None else (y if scale is None else y * scale)
    r = x + add
    rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    mag = x.abs() + (add.abs() if y is not None else 0)
    return r * rstd * w, r, mag * rstd * w.abs(), mag


def norm_residual_loss(x, w, y, scale, eps, dn, dr):
    n, r, _, _ = norm_residual(x, w, y, scale, eps)
    loss = (n * dn).sum()
    return loss if dr is None else loss + (r * dr).sum()


def norm_gate(o, z, w, eps, gate):
    sig = 1 / (1 + torch.exp(-z))
    act = z * sig if gate == "silu" else sig
    return o / torch.sqrt((o * o).mean(-1, keepdim=True) + eps) * w * act


def gelu(x):
    return x * 0.5 * (1 + torch.erf(x / math.sqrt(2)))


def draft(d, cu, L, S, hist, residual):
    """Token by token over every sequence: (o, kw, p) and the state after every
    token, [T, H, dk, dv]; d holds q, k, v, u, g, b, a, h, conv_w in 64 bits."""
    T, H, dk = d["k"].shape
    dv = d["v"].shape[2]
    o, kw_all, p_all = torch.zeros(T, H, dv).double(), torch.zeros(T, H, dk).double(), torch.zeros(T, H, dv).double()
    states = torch.zeros(T, H, dk, dv).double()
    for n in range(len(cu) - 1):
        s = S[n].clone()
        past = [hist[n, :, 0], hist[n, :, 1], hist[n, :, 2]]
        for t in range(cu[n], cu[n + 1]):
            k, b, g = d["k"][t], d["b"][t][:, None], d["g"][t][:, None, None]
            w = d["conv_w"]
            r = w[..., 3] * k + w[..., 2] * past[2] + w[..., 1] * past[1] + w[..., 0] * past[0]
            kw = b * k
            for l in range(L - 1):
                a, h, u = d["a"][t, :, l], d["h"][t, :, l], d["u"][t, :, l]
                kw = kw + a * r * u
                r = r - a * gelu(h * r) if residual == "gelu" else r * (1 - a * h)
            p = torch.einsum("hij,hi->hj", s, k)
            s = g * (s - (b * k)[:, :, None] * p[:, None, :]) + kw[:, :, None] * d["v"][t][:, None, :]
            o[t] = torch.einsum("hij,hi->hj", s, d["q"][t])
            kw_all[t], p_all[t], states[t] = kw, p, s
            past = [past[1], past[2], k]
    return o, kw_all, p_all, states


def commit(k, v, g, b, cu, kept, kw, p, S, hist):
    S, hist = S.clone(), hist.clone()
    for n, m in enumerate(kept):
        m = max(0, min(int(m), cu[n + 1] - cu[n]))
        for t in range(cu[n], cu[n] + m):
            S[n] = g[t][:, None, None] * (S[n] - (b[t][:, None] * k[t])[:, :, None] * p[t][:, None, :])
            S[n] = S[n] + kw[t][:, :, None] * v[t][:, None, :]
            hist[n] = torch.cat([hist[n, :, 1:], k[t][:, None]], 1)
    return S, hist


def _weights(w):
    return np.where((w > 0) & np.isfinite(w), w, 0.0)


def pick(w, s):
    w = _weights(w)
    if not (w > 0).any():
        return None
    c = np.cumsum(w)
    hit = np.nonzero((w > 0) & (c > s * c[-1]))[0]
    return int(hit[0]) if len(hit) else int(np.nonzero(w > 0)[0][-1])


def verify(p, q, tokens, cu, u_accept, u_sample):
    """p, q: float64 numpy [T, V] (q may be None).  (n_accept, next) lists."""
    V = p.shape[1]
    kept, nxt = [], []
    for n in range(len(cu) - 1):
        c0, c1 = cu[n], cu[n + 1]
        if c1 <= c0:
            kept.append(0)
            nxt.append(-1)
            continue
        t = c0 + 1
        while t < c1:
            x = int(tokens[t])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else q[t - 1, x]
            if not float(u_accept[t]) * qx < p[t - 1, x]:
                break
            t += 1
        m = t - c0
        full = p[t - 1]
        token = None
        if t < c1:
            if q is None:
                w = _weights(full).copy()
                if 0 <= int(tokens[t]) < V:
                    w[int(tokens[t])] = 0
            else:
                with np.errstate(invalid="ignore"):
                    w = full - q[t - 1]
            token = pick(w, float(u_sample[n]))
        if token is None:
            token = pick(full, float(u_sample[n]))
        kept.append(m)
        nxt.append(-1 if token is None else token)
    return kept, nxt


def check(name, got, ref, mag, terms, dtype=None):
    """|got - ref| <= half a step of the storage type + terms roundings of fp32 on the
    magnitude `mag` (same shape, or a number)."""
    g, r = f64(got), ref.double()
    assert g.shape == r.shape, (name, g.shape, r.shape)
    dtype = dtype or got.dtype
    tol = (HALF_STEP[dtype] if dtype == torch.bfloat16 else EPS32) * r.abs() + terms * EPS32 * mag
    tol = tol + 2.0 ** -126                                # the smallest normal fp32: subnormals may flush
    err = (g - r).abs()
    assert torch.isfinite(g).all(), name
    worst = float((err - tol).max()) if err.numel() else -1.0
    ratio = float((err / tol).max()) if err.numel() else 0.0
    assert worst <= 0, (name, worst, ratio)
    return ratio
