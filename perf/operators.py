"""The layer operators around the PRISM memory-writing operator and its decoding
of drafted tokens: cases to time, and their plain forms.

  norm_residual   residual add of the block before, scaled per channel, and the
                  RMS norm in front of the next block; forward and backward
  norm_gate       RMS norm of every head's output row, times its gate; forward
                  and backward
  decode_draft    the operator over the few drafted tokens of every sequence,
                  from a carried state that is left as it is
  decode_commit   the carried state moved on by the tokens that were kept
  verify_draft    which drafted tokens are kept, and the next token, from the
                  target's and the draft's probabilities and given random numbers

With ``own`` false ``run`` computes the plain form with elementary torch
operations in 32 bits (64 for the cumulative sums that choose a token); with
``own`` true it calls the library.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # serving: the residual stream of 8 sequences, one token each, 6 heads of 128 channels
        {"name": "residual norm, decode", "op": "norm_residual", "pass": "fwd", "rows": 8, "width": 768,
         "dtype": "bf16", "add": True, "scale": True},
        # training: the LM layer's 8 x 2048 tokens, backward with every gradient
        {"name": "residual norm, LM bwd", "op": "norm_residual", "pass": "bwd", "rows": 16384,
         "width": 768, "dtype": "bf16", "add": True, "scale": True},
        # an odd width in fp32, no scale: rows that start at any 4-byte address
        {"name": "residual norm, odd fp32", "op": "norm_residual", "pass": "fwd", "rows": 4099,
         "width": 1001, "dtype": "f32", "add": True, "scale": False},
        # one long context: 65,536 tokens of 16 heads, one weight for all heads
        {"name": "gated norm, 64k", "op": "norm_gate", "pass": "fwd", "tokens": 65536, "heads": 16,
         "width": 128, "dtype": "bf16", "per_head": False, "gate": "silu"},
        # training on user histories: 64 x 1024 tokens of 4 heads, a weight for each head
        {"name": "gated norm, histories bwd", "op": "norm_gate", "pass": "bwd", "tokens": 65536,
         "heads": 4, "width": 64, "dtype": "bf16", "per_head": True, "gate": "silu"},
        # serving: 8 sequences, the last token and 4 drafted ones
        {"name": "draft, 8 x 6 heads", "op": "decode_draft", "seqs": 8, "lo": 5, "hi": 5, "lens": 1,
         "heads": 6, "dk": 128, "dv": 128, "L": 4, "dtype": "bf16", "residual": "linear"},
        # 512 user histories with ragged drafts, some sequences idle
        {"name": "draft, 512 x 8 heads", "op": "decode_draft", "seqs": 512, "lo": 0, "hi": 9, "lens": 2,
         "heads": 8, "dk": 64, "dv": 64, "L": 8, "dtype": "bf16", "residual": "linear"},
        # a full serving batch of the LM layer
        {"name": "draft, 256 x 6 heads", "op": "decode_draft", "seqs": 256, "lo": 1, "hi": 8, "lens": 3,
         "heads": 6, "dk": 128, "dv": 128, "L": 4, "dtype": "bf16", "residual": "linear"},
        # the same batches when the kept tokens enter the states
        {"name": "commit, 8 x 6 heads", "op": "decode_commit", "seqs": 8, "lo": 5, "hi": 5, "lens": 4,
         "heads": 6, "dk": 128, "dv": 128, "dtype": "bf16"},
        {"name": "commit, 256 x 6 heads", "op": "decode_commit", "seqs": 256, "lo": 1, "hi": 8,
         "lens": 5, "heads": 6, "dk": 128, "dv": 128, "dtype": "bf16"},
        # one sequence with 4 drafted tokens: latency
        {"name": "verify, one sequence", "op": "verify_draft", "seqs": 1, "lo": 5, "hi": 5, "lens": 6,
         "vocab": 32000, "dtype": "f32", "draft": True},
        # a serving batch with ragged drafts and a large vocabulary
        {"name": "verify, 64 sequences", "op": "verify_draft", "seqs": 64, "lo": 1, "hi": 6, "lens": 7,
         "vocab": 128000, "dtype": "f32", "draft": True},
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_residual", "norm_gate", "decode_draft", "decode_commit", "verify_draft"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm_residual":
        width = _log(rng, 1, 8192)
        if rng.random() < 0.6:                       # most models' widths fill whole vectors
            width = max(8, width // 8 * 8)
        rows = _log(rng, 1, max(2, min(200000, (1 << 25) // width)))
        add = rng.random() < 0.8
        return {"op": op, "pass": rng.choice(["fwd", "bwd"]), "rows": rows, "width": width,
                "dtype": dtype, "add": add, "scale": add and rng.random() < 0.5}
    if op == "norm_gate":
        width = rng.choice([64, 128, 64, 128, 256, rng.randint(1, 512)])
        heads = rng.randint(1, 16)
        tokens = _log(rng, 1, max(2, (1 << 25) // (width * heads)))
        return {"op": op, "pass": rng.choice(["fwd", "bwd"]), "tokens": tokens, "heads": heads,
                "width": width, "dtype": dtype, "per_head": rng.random() < 0.5,
                "gate": rng.choice(["silu", "silu", "sigmoid"])}
    if op == "verify_draft":
        vocab = _log(rng, 100, 140000)
        hi = rng.randint(1, 8)
        return {"op": op, "seqs": _log(rng, 1, max(2, min(256, (1 << 25) // (vocab * hi)))),
                "lo": rng.randint(0, 1), "hi": hi, "lens": rng.randint(0, 1 << 30), "vocab": vocab,
                "dtype": dtype, "draft": rng.random() < 0.8}
    heads, dk, dv = rng.randint(1, 8), rng.choice([64, 128]), rng.choice([64, 128])
    case = {"op": op, "seqs": _log(rng, 1, max(2, 24_000_000 // (heads * dk * dv))),
            "lo": rng.randint(0, 2), "hi": rng.choice([2, 4, 5, 8, 9, 16, 20]),
            "lens": rng.randint(0, 1 << 30), "heads": heads, "dk": dk, "dv": dv, "dtype": dtype}
    if op == "decode_draft":
        case["L"] = rng.randint(1, 8)
        case["residual"] = rng.choice(["linear", "linear", "gelu"])
    return case


def _lens(case):
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _kept(case):
    """The number of tokens kept of each sequence."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(min(1, n), n) for n in _lens(case)]


def work(case):
    op, e = case["op"], ELEM[case["dtype"]]
    if op == "norm_residual":
        n, w = case["rows"] * case["width"], case["width"]
        vec = w * (2 if case["scale"] else 1)
        if case["pass"] == "fwd":                    # x, y in; r, n out
            return {"bytes": n * e * (4 if case["add"] else 2) + vec * e, "flops": 6 * n}
        many = 4 + (1 if case["scale"] else 0) + (1 if case["scale"] else 0)   # r, dn, dr, dx; y, dy
        return {"bytes": n * e * many + vec * (e + 4), "flops": 14 * n}
    if op == "norm_gate":
        n = case["tokens"] * case["heads"] * case["width"]
        w = case["width"] * (case["heads"] if case["per_head"] else 1)
        if case["pass"] == "fwd":
            return {"bytes": 3 * n * e + w * e, "flops": 12 * n}
        return {"bytes": 5 * n * e + w * (e + 4), "flops": 26 * n}
    lens = _lens(case)
    if op == "verify_draft":
        T, live = sum(lens), sum(1 for n in lens if n)
        rows = 0                                     # a row of p, and one of q, for each sequence
        rows += live * (2 if case["draft"] else 1)
        return {"bytes": rows * case["vocab"] * e + T * 16 + case["seqs"] * 16,
                "flops": live * case["vocab"] * 3}
    H, dk, dv = case["heads"], case["dk"], case["dv"]
    live = sum(1 for n in lens if n)
    if op == "decode_draft":
        T, lv = sum(lens), case["L"] - 1
        tok = (2 * dk + dv + 3 * lv * dk + 2) * e + dv * e + 4 * (dk + dv)
        return {"bytes": live * H * (4 * dk * dv + 3 * dk * e) + T * H * tok + H * dk * 4 * e,
                "flops": H * (T * 4 * dk * dv + sum(n * n for n in lens) * 3 * (dk + dv))}
    kept = _kept(case)
    tok = (dk + dv + 2) * e + 4 * (dk + dv)
    return {"bytes": case["seqs"] * H * (8 * dk * dv + 6 * dk * e) + sum(kept) * H * tok,
            "flops": H * dk * dv * sum(4 * m + 1 for m in kept)}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)).to(dt)

    op = case["op"]
    st = {"case": case}
    if op == "norm_residual":
        shape = (case["rows"], case["width"])
        st["w"] = (1 + 0.1 * normal(case["width"])).to(dt)
        st["scale"] = (0.5 + 0.1 * normal(case["width"])).to(dt) if case["scale"] else None
        st["y"] = normal(*shape).to(dt) if case["add"] else None
        if case["pass"] == "fwd":
            st["x"] = (2 * normal(*shape)).to(dt)
        else:
            st["r"] = (2 * normal(*shape)).to(dt)
            st["dn"] = normal(*shape).to(dt)
            st["dr"] = normal(*shape).to(dt)
        return st
    if op == "norm_gate":
        shape = (case["tokens"], case["heads"], case["width"])
        st["o"] = (0.2 * normal(*shape)).to(dt)
        st["z"] = normal(*shape).to(dt)
        st["w"] = (1 + 0.1 * normal(*((case["heads"],) if case["per_head"] else ()), case["width"])).to(dt)
        if case["pass"] == "bwd":
            st["dy"] = normal(*shape).to(dt)
        return st

    lens = _lens(case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N = cu[-1], len(lens)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["max_len"] = max(lens)
    if op == "verify_draft":
        V = case["vocab"]
        logits = 3 * normal(T, V)
        st["p"] = torch.softmax(logits, -1).to(dt)
        q = torch.softmax(logits + 0.7 * normal(T, V), -1).to(dt)
        tokens = torch.zeros(T, dtype=torch.int32, device=dev)
        if T > 1:                                    # the token after row t is drawn from q[t]
            c = torch.cumsum(q[:-1].double(), -1)
            s = uniform(T - 1, 1).double() * c[:, -1:]
            tokens[1:] = torch.searchsorted(c, s, right=True)[:, 0].clamp_max(V - 1).to(torch.int32)
        st["q"] = q if case["draft"] else None
        st["tokens"] = tokens
        st["u_accept"] = uniform(T)
        st["u_sample"] = uniform(N)
        return st

    H, dk, dv = case["heads"], case["dk"], case["dv"]
    L = case.get("L", 1)
    st["q"], st["k"] = unit(T, H, dk), unit(T, H, dk)
    st["v"] = normal(T, H, dv).to(dt)
    st["g"] = torch.sigmoid(3 + normal(T, H)).to(dt)
    st["b"] = torch.sigmoid(normal(T, H)).to(dt)
    st["S"] = 0.3 * normal(N, H, dk, dv)
    st["k_hist"] = unit(N, H, 3, dk)
    if op == "decode_draft":
        if L > 1:
            st["u"] = unit(T, H, L - 1, dk)
            st["a"] = (0.5 * torch.sigmoid(normal(T, H, L - 1, dk))).to(dt)
            st["h"] = torch.sigmoid(normal(T, H, L - 1, dk)).to(dt)
        else:
            st["u"] = st["a"] = st["h"] = None
        st["conv_w"] = (0.5 * normal(H, dk, 4)).to(dt)
        return st
    # commit: the records that the draft left, and the number of tokens kept
    st["kw"] = st["b"].float()[..., None] * st["k"].float() + 0.02 * normal(T, H, dk)
    st["p"] = 0.3 * normal(T, H, dv)
    st["n_accept"] = torch.tensor(_kept(case), dtype=torch.int32, device=dev)
    st["S_out"], st["k_hist_out"] = torch.empty_like(st["S"]), torch.empty_like(st["k_hist"])
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return _library(state) if own else PLAIN[state["case"]["op"]](state)


def _library(st):
    from gated_delta_rule_prologue_amd import binding as B
    case = st["case"]
    op = case["op"]
    if op == "norm_residual":
        if case["pass"] == "fwd":
            n, r = B.norm_residual(st["x"], st["w"], y=st["y"], scale=st["scale"], eps=EPS)
            return {"n": n, "r": r} if case["add"] else {"n": n}
        g = B.norm_residual_bwd(st["r"], st["w"], st["dn"], dr=st["dr"], eps=EPS,
                                y=st["y"] if case["scale"] else None, scale=st["scale"])
        return {k: v for k, v in g.items() if v is not None}
    if op == "norm_gate":
        if case["pass"] == "fwd":
            return {"y": B.norm_gate(st["o"], st["z"], st["w"], eps=EPS, gate=case["gate"])}
        return B.norm_gate_bwd(st["o"], st["z"], st["w"], st["dy"], eps=EPS, gate=case["gate"])
    if op == "verify_draft":
        n, t = B.verify_draft(st["p"], st["tokens"], st["cu"], st["u_accept"], st["u_sample"], q=st["q"])
        return {"n_accept": n, "next": t}
    if op == "decode_draft":
        o, kw, p = B.decode_draft(st["q"], st["k"], st["v"], st["u"], st["g"], st["b"], st["a"], st["h"],
                                  st["conv_w"], st["cu"], case["L"], st["S"], st["k_hist"],
                                  residual=case["residual"])
        return {"o": o, "kw": kw, "p": p}
    S, hist = B.decode_commit(st["k"], st["v"], st["g"], st["b"], st["cu"], st["n_accept"], st["kw"],
                              st["p"], st["S"], st["k_hist"], S_out=st["S_out"],
                              k_hist_out=st["k_hist_out"])
    return {"S": S, "k_hist": hist}


def _norm_residual(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    w = st["w"].float()
    s = st["scale"].float() if st["scale"] is not None else None
    if case["pass"] == "fwd":
        r = st["x"].float()
        if case["add"]:
            y = st["y"].float()
            r = r + (y if s is None else s * y)
        n = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * w
        return {"n": n.to(dt), "r": r.to(dt)} if case["add"] else {"n": n.to(dt)}
    r, dn = st["r"].float(), st["dn"].float()
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    rh = r * rstd
    e = dn * w
    t = rstd * (e - rh * (e * rh).mean(-1, keepdim=True)) + st["dr"].float()
    out = {"x": t.to(dt), "w": (dn * rh).sum(0)}
    if s is not None:
        out["y"] = (s * t).to(dt)
        out["scale"] = (t * st["y"].float()).sum(0)
    return out


def _norm_gate(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    o, z, w = st["o"].float(), st["z"].float(), st["w"].float()
    sig = torch.sigmoid(z)
    act = z * sig if case["gate"] == "silu" else sig
    rstd = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    oh = o * rstd
    if case["pass"] == "fwd":
        return {"y": (oh * w * act).to(dt)}
    dy = st["dy"].float()
    slope = sig * (1 + z * (1 - sig)) if case["gate"] == "silu" else sig * (1 - sig)
    e = dy * act * w
    do = rstd * (e - oh * (e * oh).mean(-1, keepdim=True))
    dw = dy * act * oh
    return {"o": do.to(dt), "z": (dy * oh * w * slope).to(dt),
            "w": dw.sum(0) if case["per_head"] else dw.sum((0, 1))}


def _padded(cu, max_len):
    """[N, max_len] packed row of every (sequence, position), and which of them exist."""
    pos = torch.arange(max_len, device=cu.device)
    start = cu[:-1].long()[:, None]
    row = start + pos
    there = row < cu[1:].long()[:, None]
    return torch.where(there, row, torch.zeros_like(row)), there


def _gelu(x):
    return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))


def _decode_draft(st):
    case = st["case"]
    dt, L, M = DTYPES[case["dtype"]], case["L"], st["max_len"]
    T, H, dk = st["k"].shape
    dv = st["v"].shape[2]
    o = torch.zeros(T, H, dv, device=st["k"].device)
    kw_out = torch.zeros(T, H, dk, device=st["k"].device)
    p_out = torch.zeros(T, H, dv, device=st["k"].device)
    if T == 0:
        return {"o": o.to(dt), "kw": kw_out, "p": p_out}
    row, there = _padded(st["cu"], M)
    S, hist, cw = st["S"].clone(), st["k_hist"].float(), st["conv_w"].float()
    k3, k2, k1 = hist[:, :, 0], hist[:, :, 1], hist[:, :, 2]
    for t in range(M):
        i, m = row[:, t], there[:, t]
        k, q, v = st["k"][i].float(), st["q"][i].float(), st["v"][i].float()
        g, b = st["g"][i].float()[..., None], st["b"][i].float()[..., None]
        r = cw[..., 0] * k3 + cw[..., 1] * k2 + cw[..., 2] * k1 + cw[..., 3] * k
        kw = b * k
        for l in range(L - 1):
            a, h = st["a"][i][:, :, l].float(), st["h"][i][:, :, l].float()
            kw = kw + a * r * st["u"][i][:, :, l].float()
            r = r - a * _gelu(h * r) if case["residual"] == "gelu" else r * (1 - a * h)
        p = (S * k[..., None]).sum(2)
        S = g[..., None] * (S - (b * k)[..., None] * p[:, :, None, :]) + kw[..., None] * v[:, :, None, :]
        at = i[m]
        o[at] = (S * q[..., None]).sum(2)[m]
        kw_out[at], p_out[at] = kw[m], p[m]
        k3, k2, k1 = k2, k1, k
    return {"o": o.to(dt), "kw": kw_out, "p": p_out}


def _decode_commit(st):
    M = st["max_len"]
    S, hist = st["S"], st["k_hist"]
    if st["k"].shape[0] == 0:
        return {"S": S.clone(), "k_hist": hist.clone()}
    row, _ = _padded(st["cu"], M)
    keep = st["n_accept"].long()
    for t in range(M):
        i = row[:, t]
        k, v, g, b = (st[x][i].float() for x in ("k", "v", "g", "b"))
        new = g[..., None, None] * (S - (b[..., None] * k)[..., None] * st["p"][i][:, :, None, :])
        new = new + st["kw"][i][..., None] * v[:, :, None, :]
        on = (t < keep)
        S = torch.where(on[:, None, None, None], new, S)
        moved = torch.cat([hist[:, :, 1:], st["k"][i][:, :, None]], 2)
        hist = torch.where(on[:, None, None, None], moved, hist)
    return {"S": S, "k_hist": hist}


def _pick(w, s):
    """The smallest index whose cumulative weight passes s times the total, of those with
    weight; the last one with weight if none does; -1 in a row without weight."""
    w = torch.where((w > 0) & (w < math.inf), w, torch.zeros_like(w))
    c = torch.cumsum(w, -1)
    idx = torch.arange(w.shape[1], device=w.device)
    live = w > 0
    hit = live & (c > s[:, None] * c[:, -1:])
    first = torch.where(hit, idx, w.shape[1]).amin(-1)
    last = torch.where(live, idx, -1).amax(-1)
    return torch.where(hit.any(-1), first, last), live.any(-1)


def _verify_draft(st):
    p, q, tok, cu, M = st["p"], st["q"], st["tokens"].long(), st["cu"].long(), st["max_len"]
    N, V = cu.numel() - 1, p.shape[1]
    none = torch.zeros(N, dtype=torch.int32, device=p.device)
    if p.shape[0] == 0:
        return {"n_accept": none, "next": none - 1}
    row, there = _padded(cu, M)
    going = there[:, 0]
    n = going.long()
    for t in range(1, M):
        x, before = tok[row[:, t]], row[:, t - 1]
        ok = (x >= 0) & (x < V)
        xs = x.clamp(0, V - 1)
        px = p[before, xs].double()
        qx = torch.ones_like(px) if q is None else q[before, xs].double()
        going = going & there[:, t] & ok & (st["u_accept"][row[:, t]].double() * qx < px)
        n = n + going
    length = cu[1:] - cu[:-1]
    at = (cu[:-1] + n - 1).clamp(0, p.shape[0] - 1)
    full = p[at].double()
    rejected = n < length
    x = tok[(at + 1).clamp_max(p.shape[0] - 1)]
    if q is None:
        ids = torch.arange(V, device=p.device)
        less = torch.where(ids == x[:, None], torch.zeros_like(full), full)
    else:
        less = full - q[at].double()
    s = st["u_sample"].double()
    first, some = _pick(torch.where(rejected[:, None], less, full), s)
    second, _ = _pick(full, s)
    token = torch.where(some, first, second)
    return {"n_accept": n.to(torch.int32), "next": torch.where(length > 0, token, -1).to(torch.int32)}


PLAIN = {"norm_residual": _norm_residual, "norm_gate": _norm_gate, "decode_draft": _decode_draft,
         "decode_commit": _decode_commit, "verify_draft": _verify_draft}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in st.items()}
    return EXACT[case["op"]](case, d)


def _exact_norm_residual(case, d):
    """Forward from the definition; backward by differentiating it."""
    def norm(r, w):
        return w * r / torch.sqrt(torch.mean(r ** 2, -1, keepdim=True) + EPS)

    if case["pass"] == "fwd":
        r = d["x"]
        if case["add"]:
            r = torch.addcmul(r, d["y"], d["scale"].expand_as(r) if case["scale"] else torch.ones_like(r))
            return {"n": norm(r, d["w"]), "r": r}
        return {"n": norm(r, d["w"])}
    r, w = d["r"].requires_grad_(True), d["w"].requires_grad_(True)
    t, dw = torch.autograd.grad((norm(r, w) * d["dn"]).sum() + (r * d["dr"]).sum(), (r, w))
    out = {"x": t, "w": dw}
    if case["scale"]:
        out["y"] = d["scale"] * t
        out["scale"] = torch.einsum("rc,rc->c", t, d["y"])
    return out


def _exact_norm_gate(case, d):
    def gated(o, z, w):
        act = 1 / (1 + torch.exp(-z))
        if case["gate"] == "silu":
            act = act * z
        return act * w * (o / torch.sqrt(torch.mean(o ** 2, -1, keepdim=True) + EPS))

    if case["pass"] == "fwd":
        y = torch.empty_like(d["o"])
        for i in range(0, y.shape[0], 4096):         # in parts: 64-bit temporaries are large
            y[i:i + 4096] = gated(d["o"][i:i + 4096], d["z"][i:i + 4096], d["w"])
        return {"y": y}
    leaves = [d[n].requires_grad_(True) for n in ("o", "z", "w")]
    do, dz, dw = torch.autograd.grad((gated(*leaves) * d["dy"]).sum(), leaves)
    return {"o": do, "z": dz, "w": dw}


def _exact_decode_draft(case, d):
    """Sequence positions in turn, the state moved by its transition matrix."""
    T, H, dk = d["k"].shape
    dv = d["v"].shape[2]
    new = dict(device=d["k"].device, dtype=torch.float64)
    out = {"o": torch.zeros(T, H, dv, **new), "kw": torch.zeros(T, H, dk, **new),
           "p": torch.zeros(T, H, dv, **new)}
    cu = d["cu"].tolist()
    eye = torch.eye(dk, **new)
    state = d["S"].clone()
    for t in range(max(d["max_len"], 0)):
        live = [n for n in range(len(cu) - 1) if cu[n] + t < cu[n + 1]]
        if not live:
            break
        n = torch.tensor(live, device=state.device)
        at = torch.tensor([cu[i] + t for i in live], device=state.device)
        k = d["k"][at]
        r = d["conv_w"][:, :, 3] * k
        for back in (1, 2, 3):                       # the k rows before: this draft's, or carried
            if t >= back:
                past = d["k"][at - back]
            else:
                past = d["k_hist"][n, :, 3 + t - back]
            r = r + d["conv_w"][:, :, 3 - back] * past
        kw = d["b"][at].unsqueeze(-1) * k
        keep = torch.ones_like(r)
        for l in range(case["L"] - 1):
            a, h, u = (d[x][at, :, l] for x in ("a", "h", "u"))
            if case["residual"] == "gelu":
                kw = kw + a * r * u
                x = h * r
                r = r - a * x * 0.5 * torch.erfc(-x / math.sqrt(2))
            else:                                    # the closed form: the anchor times a product
                kw = kw + a * (r * keep) * u
                keep = keep * (1 - a * h)
        S = state[n]
        move = eye - (d["b"][at].unsqueeze(-1) * k).unsqueeze(-1) * k.unsqueeze(-2)
        out["p"][at] = torch.matmul(k.unsqueeze(-2), S).squeeze(-2)
        S = torch.matmul(d["g"][at][..., None, None] * move, S) + kw.unsqueeze(-1) * d["v"][at].unsqueeze(-2)
        state[n] = S
        out["kw"][at] = kw
        out["o"][at] = torch.matmul(d["q"][at].unsqueeze(-2), S).squeeze(-2)
    return out


def _exact_decode_commit(case, d):
    """The kept tokens' writes, each weighted by the gates that follow it."""
    cu, kept = d["cu"].tolist(), _kept(case)
    S, hist = torch.empty_like(d["S"]), torch.empty_like(d["k_hist"])
    for n, m in enumerate(kept):
        rows = slice(cu[n], cu[n] + m)
        g, b, k, p = d["g"][rows], d["b"][rows], d["k"][rows], d["p"][rows]
        after = torch.ones(m + 1, g.shape[1], device=g.device, dtype=g.dtype)
        for j in range(m - 1, -1, -1):               # the product of the gates j..m-1
            after[j] = after[j + 1] * g[j]
        S[n] = after[0][:, None, None] * d["S"][n]
        erase = (after[:m] * b)[..., None] * k
        S[n] -= torch.matmul(erase.permute(1, 2, 0), p.permute(1, 0, 2))
        write = after[1:][..., None] * d["kw"][rows]
        S[n] += torch.matmul(write.permute(1, 2, 0), d["v"][rows].permute(1, 0, 2))
        hist[n] = torch.cat([d["k_hist"][n], k.permute(1, 0, 2)], 1)[:, -3:]
    return {"S": S, "k_hist": hist}


def _exact_verify_draft(case, d):
    cu = d["cu"].tolist()
    tok, u = d["tokens"].tolist(), d["u_accept"].tolist()
    V = case["vocab"]
    n_accept, nxt = [], []
    for n in range(len(cu) - 1):
        c0, c1 = cu[n], cu[n + 1]
        if c0 == c1:
            n_accept.append(0)
            nxt.append(-1)
            continue
        t = c0
        while t + 1 < c1:
            x = tok[t + 1]
            px = d["p"][t, x].item()
            qx = 1.0 if d["q"] is None else d["q"][t, x].item()
            if not u[t + 1] * qx < px:
                break
            t += 1
        w = d["p"][t].clone()
        if t + 1 < c1:
            if d["q"] is None:
                w[tok[t + 1]] = 0
            else:
                w = (w - d["q"][t]).clamp_min(0)
            if not bool((w > 0).any()):
                w = d["p"][t].clone()
        c = torch.cumsum(w, 0)
        j = int(torch.searchsorted(c, d["u_sample"][n] * c[-1], right=True))
        n_accept.append(t - c0 + 1)
        nxt.append(min(j, int(torch.nonzero(w)[-1])))
    dev = d["p"].device
    return {"n_accept": torch.tensor(n_accept, dtype=torch.int32, device=dev),
            "next": torch.tensor(nxt, dtype=torch.int32, device=dev)}


EXACT = {"norm_residual": _exact_norm_residual, "norm_gate": _exact_norm_gate,
         "decode_draft": _exact_decode_draft, "decode_commit": _exact_decode_commit,
         "verify_draft": _exact_verify_draft}
