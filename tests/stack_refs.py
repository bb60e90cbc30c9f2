"""Plain 64-bit references of the short convolution, the norm and rotation of queries and
keys, and the choice of a token, written from their formulas on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch


def rows_of(x, hist, cu, n, t, K):
    """The K rows that end with row t of sequence n, oldest first (zero in front without a history)."""
    out = []
    for m in range(K):
        r = t - K + 1 + m
        if r >= cu[n]:
            out.append(x[r])
        elif hist is not None:
            out.append(hist[n, K - 1 + r - cu[n]])
        else:
            out.append(torch.zeros_like(x[t]))
    return torch.stack(out)                                   # [K, C]


def short_conv(x, w, cu, bias=None, silu=True, hist=None):
    """(y, the sums s in front of the activation, the magnitude of their terms), rows behind the last
    sequence zero; differentiable."""
    K = w.shape[1]
    zero = torch.zeros_like(x[0]) if x.shape[0] else None
    s, mag = [zero] * x.shape[0], [zero] * x.shape[0]
    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            win = rows_of(x, hist, cu, n, t, K)
            s[t] = (win * w.t()).sum(0) + (0 if bias is None else bias)
            mag[t] = (win * w.t()).abs().sum(0) + (0 if bias is None else bias.abs())
    s = torch.stack(s) if s else x * w[:, 0]                  # no rows: nothing but the leaves
    mag = torch.stack(mag) if mag else torch.zeros_like(x)
    return s * torch.sigmoid(s) if silu else s, s, mag.detach()


def conv_tolerances(x, w, cu, dy, bias, silu, hist):
    """Errors in units of 2^-24 that fp32 arithmetic may leave in y, dx, dw, dbias and dhist
    before their storage rounding (see test_gpu_short_conv)."""
    K = w.shape[1]
    _, s, mag = short_conv(x, w, cu, bias, silu, hist)
    es = (K + 2) * mag                                        # K products and additions
    c = torch.sigmoid(-s)
    if silu:
        y = (s * torch.sigmoid(s)).abs()
        ey = 1.1 * es + (16 + 2 * s.abs()) * y
        top = torch.sigmoid(s) * (1 + s.abs() * c)            # |silu'| without its cancellation
        eds = dy.abs() * (0.5 * es + (16 + 2 * s.abs()) * top)
        ds = dy.abs() * top
    else:
        ey, eds, ds = es, torch.zeros_like(s), dy.abs()
    C = x.shape[1]
    ex, ew, eb = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(C).double()
    eh = None if hist is None else torch.zeros_like(hist)
    adds = 128                                                # of a lane's run, its workgroup and the workgroups
    for n in range(len(cu) - 1):
        for t in range(cu[n], cu[n + 1]):
            win = rows_of(x, hist, cu, n, t, K).abs()
            ew += ((eds[t] + adds * ds[t]) * win).t()
            eb += eds[t] + adds * ds[t]
            for m in range(K):
                r = t - K + 1 + m
                e = w[:, m].abs() * (eds[t] + (K + 1) * ds[t])
                if r >= cu[n]:
                    ex[r] += e
                elif eh is not None:
                    eh[n, K - 1 + r - cu[n]] += e
    return ey, ex, ew, eb, eh


def carried(x, hist, cu, K):
    """[N, K - 1, C]: the last K - 1 rows of every [history; sequence]."""
    out = []
    for n in range(len(cu) - 1):
        h = torch.zeros(K - 1, x.shape[1], dtype=x.dtype) if hist is None else hist[n]
        rows = torch.cat([h, x[cu[n]:cu[n + 1]]])
        out.append(rows[rows.shape[0] - (K - 1):])
    return torch.stack(out)


def pairs(rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, positions, freqs, layout, scale=1.0):
    """x [T, H, d] with the first 2 len(freqs) elements turned."""
    rot = 2 * freqs.numel()
    angle = positions.double()[:, None] * freqs.double()
    c, s = torch.cos(angle)[:, None] * scale, torch.sin(angle)[:, None] * scale
    a, b = pairs(rot, layout)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def partner_sum(x, rot, layout, scale=1.0):
    """|a| + |b| in the place of each of a pair, |x| elsewhere."""
    y = x.abs().clone()
    a, b = pairs(rot, layout)
    y[..., a] = y[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(scale)
    return y


def rstd_of(x, norm, eps):
    if norm == "none":
        return torch.ones_like(x[..., :1])
    ss = (x * x).sum(-1, keepdim=True)
    return 1 / torch.sqrt((ss / x.shape[-1] if norm == "rms" else ss) + eps)


def qk_norm(x, w, norm, eps, positions=None, freqs=None, layout="half", scale=1.0):
    y = x * rstd_of(x, norm, eps)
    if w is not None:
        y = y * w
    return y if freqs is None else rotate(y, positions, freqs, layout, scale)


def kept(l, t=1.0, k=0, p=1.0, m=0.0):
    """The entries that stay, in the order of falling logits, and their weights; l float64 [V]."""
    l = np.where(np.isnan(l), -np.inf, l)
    if not (l > -np.inf).any():
        return np.zeros(0, dtype=int), np.zeros(0)
    if (l == np.inf).any():
        l = np.where(l == np.inf, 0.0, -np.inf)
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if not t > 0:
        return order[:1], np.ones(1)
    with np.errstate(over="ignore", under="ignore"):
        w = np.exp((l[order] - l[order[0]]) / t)
    if k > 0:
        order, w = order[:k], w[:k]
    if p < 1:
        c = np.cumsum(w)
        before = np.concatenate([[0.0], c[:-1]])
        n = max(1, int((before < p * c[-1]).sum()))
        order, w = order[:n], w[:n]
    if m > 0:
        n = max(1, int((w >= min(m, 1.0)).sum()))
        order, w = order[:n], w[:n]
    return order, w


def sample(l, u, **filters):
    order, w = kept(l, **filters)
    if not len(order):
        return -1
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -24)
    c = np.cumsum(w)
    return int(order[int(np.nonzero(c > u * c[-1])[0][0])])


def probs(l, **filters):
    order, w = kept(l, **filters)
    out = np.zeros(len(l))
    if len(order):
        out[order] = w / math.fsum(w)
    return out
