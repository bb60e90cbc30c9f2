"""Operators in front of the PRISM memory-writing operator and behind the model's last
product: cases to time, and their plain forms.

  short_conv   causal depthwise convolution over packed sequences, with its bias and
               SiLU, as the projections of q, k and v pass through it; forward from a
               carried history, backward, and the form for one token a sequence
  qk_norm      every head's query and key normalised, weighted and rotated by its position
               in one pass; forward and backward
  sample       temperature, top-k, top-p and min-p over rows of logits: the token that a
               given random number draws, and the distribution that is left

With ``own`` false ``run`` computes the plain form with elementary torch operations, in 32
bits (64 for the angles of positions and for the sums that choose a token); with ``own``
true it calls the library.
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
        # training: q, k and v (6 heads of 128) of the LM layer's 8 x 2048 tokens, columns of the
        # fused projection's rows
        {"name": "conv, LM layer", "op": "short_conv", "pass": "fwd", "seqs": 8, "lo": 2048, "hi": 2048,
         "lens": 1, "channels": 2304, "taps": 4, "dtype": "bf16", "bias": False, "act": "silu",
         "hist": False, "wide": True},
        # training on packed user histories (8 heads of 64, q, k and v), every gradient
        {"name": "conv, histories bwd", "op": "short_conv", "pass": "bwd", "seqs": 64, "lo": 16,
         "hi": 8192, "lens": 2, "channels": 1536, "taps": 4, "dtype": "bf16", "bias": True,
         "act": "silu", "hist": False, "wide": False},
        # serving: one token each of 256 sequences, 6 heads of 128
        {"name": "conv, decode 256", "op": "short_conv", "pass": "step", "seqs": 256, "lo": 1, "hi": 1,
         "lens": 3, "channels": 2304, "taps": 4, "dtype": "bf16", "bias": False, "act": "silu",
         "hist": True, "wide": False},
        # prompts taken up again, some of them empty, an odd number of channels in fp32
        {"name": "conv, resumed odd fp32", "op": "short_conv", "pass": "fwd", "seqs": 33, "lo": 0,
         "hi": 700, "lens": 4, "channels": 1001, "taps": 3, "dtype": "f32", "bias": True,
         "act": "none", "hist": True, "wide": False},
        # the LM layer's queries and keys, L2 norm and rotation, columns of the fused projection
        {"name": "qk norm, LM layer", "op": "qk_norm", "pass": "fwd", "tokens": 16384, "period": 2048,
         "hq": 6, "hk": 6, "d": 128, "rot": 128, "layout": "half", "norm": "l2", "weight": False,
         "dtype": "bf16", "wide": True},
        # the same layer's gradients, with RMS norms and their weights
        {"name": "qk norm, LM bwd", "op": "qk_norm", "pass": "bwd", "tokens": 16384, "period": 2048,
         "hq": 6, "hk": 6, "d": 128, "rot": 128, "layout": "half", "norm": "rms", "weight": True,
         "dtype": "bf16", "wide": False},
        # serving: 256 sequences, one token each, anywhere in a long context
        {"name": "qk norm, decode 256", "op": "qk_norm", "pass": "fwd", "tokens": 256, "period": 1,
         "hq": 6, "hk": 6, "d": 128, "rot": 128, "layout": "half", "norm": "l2", "weight": False,
         "dtype": "bf16", "wide": True},
        # shared keys, part of an odd head rotated, interleaved pairs, fp32
        {"name": "qk norm, odd fp32 bwd", "op": "qk_norm", "pass": "bwd", "tokens": 2999, "period": 1500,
         "hq": 5, "hk": 1, "d": 75, "rot": 30, "layout": "interleaved", "norm": "rms", "weight": True,
         "dtype": "f32", "wide": False},
        # one sequence: latency
        {"name": "sample, one sequence", "op": "sample", "rows": 1, "vocab": 32000, "dtype": "f32",
         "filters": "k+p", "masked": False, "out": "tokens"},
        # a serving batch whose requests bring their own settings, a large vocabulary
        {"name": "sample, 64 mixed", "op": "sample", "rows": 64, "vocab": 128000, "dtype": "f32",
         "filters": "mixed", "masked": False, "out": "tokens"},
        # a large batch, bf16 logits with many ties, entries that a grammar masks
        {"name": "sample, 256 bf16 masked", "op": "sample", "rows": 256, "vocab": 32000, "dtype": "bf16",
         "filters": "p", "masked": True, "out": "tokens"},
        # the distributions that the verification of drafted tokens takes, an odd vocabulary
        {"name": "sample, distributions", "op": "sample", "rows": 320, "vocab": 50001, "dtype": "f32",
         "filters": "mixed", "masked": False, "out": "probs"},
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, spread evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["short_conv", "short_conv", "qk_norm", "qk_norm", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "short_conv":
        c = _log(rng, 8, 4096)
        if rng.random() < 0.6:                       # most models' channels fill whole vectors
            c = max(8, c // 8 * 8)
        pas = rng.choice(["fwd", "bwd", "step"])
        case = {"op": op, "pass": pas, "channels": c, "taps": rng.choice([2, 3, 4, 4, 4, 5, 8]),
                "dtype": dtype, "bias": rng.random() < 0.5, "act": rng.choice(["silu", "silu", "none"]),
                "hist": pas == "step" or rng.random() < 0.4, "wide": rng.random() < 0.3,
                "lens": rng.randint(0, 1 << 30)}
        if pas == "step":
            return {**case, "seqs": _log(rng, 1, 1024), "lo": 1, "hi": 1}
        most = max(2, (1 << 26) // c)                # tokens
        hi = _log(rng, 1, min(8192, most))
        return {**case, "seqs": _log(rng, 1, max(1, min(512, most // hi))), "lo": rng.choice([0, 1, hi]),
                "hi": hi}
    if op == "qk_norm":
        d = rng.choice([64, 128, 64, 128, 80, 256, rng.randint(2, 300)])
        hk = rng.randint(1, 8)
        hq = hk * rng.choice([1, 1, 2, 4])
        rot = rng.choice([d // 2 * 2, d // 2 * 2, d // 4 * 2, 0])
        norm = rng.choice(["l2", "rms", "rms", "none"])
        return {"op": op, "pass": rng.choice(["fwd", "bwd"]),
                "tokens": _log(rng, 1, max(2, min(32768, (1 << 25) // (d * (hq + hk))))),
                "period": _log(rng, 1, 2048), "hq": hq, "hk": hk, "d": d, "rot": rot,
                "layout": rng.choice(["half", "interleaved"]), "norm": norm,
                "weight": norm != "none" and rng.random() < 0.6, "dtype": dtype,
                "wide": rng.random() < 0.4}
    vocab = _log(rng, 100, 140000)
    return {"op": op, "rows": _log(rng, 1, max(2, min(512, (1 << 24) // vocab))), "vocab": vocab,
            "dtype": dtype, "filters": rng.choice(["none", "k", "p", "k+p", "min_p", "mixed", "mixed"]),
            "masked": rng.random() < 0.3, "out": rng.choice(["tokens", "tokens", "probs"])}


def _lens(case):
    r = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    return [0 if lo == 0 and r.random() < 0.15 else _log(r, max(1, lo), max(1, hi))
            for _ in range(case["seqs"])]


def work(case):
    op, e = case["op"], ELEM[case["dtype"]]
    if op == "short_conv":
        c, k, n = case["channels"], case["taps"], case["seqs"]
        vec = c * (k + (1 if case["bias"] else 0))
        hist = n * (k - 1) * c * e
        if case["pass"] == "step":                   # x, history in; y, history out
            return {"bytes": 2 * n * c * e + 2 * hist + vec * e, "flops": n * c * (2 * k + 6)}
        t = sum(_lens(case))
        if case["pass"] == "fwd":
            return {"bytes": 2 * t * c * e + (2 * hist if case["hist"] else 0) + vec * e,
                    "flops": t * c * (2 * k + 6)}
        return {"bytes": 3 * t * c * e + (2 * hist if case["hist"] else 0) + vec * (e + 4),
                "flops": t * c * (6 * k + 14)}
    if op == "qk_norm":
        rows = case["tokens"] * (case["hq"] + case["hk"])
        vec = 2 * case["d"] * (1 if case["weight"] else 0)
        n = rows * case["d"]
        side = case["tokens"] * 4 + case["rot"] * 2 if case["rot"] else 0
        if case["pass"] == "fwd":
            return {"bytes": 2 * n * e + vec * e + side, "flops": 8 * n}
        return {"bytes": 3 * n * e + vec * (e + 4) + side, "flops": 18 * n}
    n = case["rows"] * case["vocab"]
    out = n * 4 if case["out"] == "probs" else case["rows"] * 4
    return {"bytes": n * e + out + case["rows"] * 20, "flops": 20 * n}


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

    op = case["op"]
    st = {"case": case}
    if op == "short_conv":
        c, k = case["channels"], case["taps"]
        lens = _lens(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        t = cu[-1]
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        # `wide`: the columns of a projection whose rows hold the gates too
        st["x"] = normal(t, c + (16 if case["wide"] else 0)).to(dt)[:, :c]
        st["w"] = (normal(c, k) / math.sqrt(k)).to(dt)
        st["bias"] = (0.1 * normal(c)).to(dt) if case["bias"] else None
        st["hist"] = normal(len(lens), k - 1, c).to(dt) if case["hist"] else None
        st["hist_out"] = torch.empty_like(st["hist"]) if case["hist"] and case["pass"] != "bwd" else None
        if case["pass"] == "bwd":
            st["dy"] = normal(t, c).to(dt)
        return st
    if op == "qk_norm":
        t, hq, hk, d = case["tokens"], case["hq"], case["hk"], case["d"]
        if case["wide"]:                             # q, k and v are columns of one projection
            rows = normal(t, (hq + 2 * hk) * d).to(dt)
            st["q"] = rows[:, :hq * d].view(t, hq, d)
            st["k"] = rows[:, hq * d:(hq + hk) * d].view(t, hk, d)
        else:
            st["q"], st["k"] = normal(t, hq, d).to(dt), normal(t, hk, d).to(dt)
        for name in ("wq", "wk"):
            st[name] = (1 + 0.1 * normal(d)).to(dt) if case["weight"] else None
        st["positions"] = st["freqs"] = None
        if case["rot"]:
            first = (uniform(-(-t // case["period"])) * 100000).to(torch.int32)
            at = torch.arange(t, device=dev)
            st["positions"] = first[at // case["period"]] + (at % case["period"]).to(torch.int32)
            i = torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64)
            st["freqs"] = (10000.0 ** (-2 * i / case["rot"])).float()
        if case["pass"] == "bwd":
            st["dq"], st["dk"] = normal(t, hq, d).to(dt), normal(t, hk, d).to(dt)
        return st

    n, v = case["rows"], case["vocab"]
    logits = 3 * normal(n, v)
    if case["masked"]:                               # a third of the entries may not be drawn
        logits = logits.masked_fill(uniform(v) < 0.33, -math.inf)
        logits[:, v // 2] = 0.5
    st["logits"] = logits.to(dt)
    st["u"] = uniform(n) if case["out"] == "tokens" else None
    st["temperature"] = 0.3 + 1.2 * uniform(n)
    f, mixed = case["filters"], case["filters"] == "mixed"
    st["top_k"] = st["top_p"] = st["min_p"] = None
    if f in ("k", "k+p") or mixed:
        st["top_k"] = (torch.exp(uniform(n) * math.log(200)) + 0.5).to(torch.int32)
    if f in ("p", "k+p") or mixed:
        st["top_p"] = 0.5 + 0.5 * uniform(n)
    if f == "min_p" or mixed:
        st["min_p"] = 0.2 * uniform(n)
    if mixed:                                        # requests that leave some of them off, or are greedy
        st["temperature"] = torch.where(uniform(n) < 0.15, 0.0, st["temperature"])
        st["top_k"] = torch.where(uniform(n) < 0.5, 0, st["top_k"])
        st["top_p"] = torch.where(uniform(n) < 0.3, 1.0, st["top_p"])
        st["min_p"] = torch.where(uniform(n) < 0.6, 0.0, st["min_p"])
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return _library(state) if own else PLAIN[state["case"]["op"]](state)


def _library(st):
    from gated_delta_rule_prologue_amd import binding as B
    case = st["case"]
    op = case["op"]
    if op == "short_conv":
        act = case["act"] if case["act"] != "none" else None
        if case["pass"] == "step":
            y, hist = B.short_conv_step(st["x"], st["w"], st["hist"], bias=st["bias"], activation=act,
                                        hist_out=st["hist_out"])
            return {"y": y, "hist": hist}
        if case["pass"] == "fwd":
            y, hist = B.short_conv(st["x"], st["w"], st["cu"], bias=st["bias"], activation=act,
                                   hist=st["hist"], hist_out=st["hist_out"])
            return {"y": y, "hist": hist} if case["hist"] else {"y": y}
        g = B.short_conv_bwd(st["x"], st["w"], st["cu"], st["dy"], bias=st["bias"], activation=act,
                             hist=st["hist"])
        return {k: v for k, v in g.items() if v is not None}
    if op == "qk_norm":
        how = dict(wq=st["wq"], wk=st["wk"], norm=case["norm"], eps=EPS, positions=st["positions"],
                   freqs=st["freqs"], layout=case["layout"])
        if case["pass"] == "fwd":
            q, k = B.qk_norm(st["q"], st["k"], **how)
            return {"q": q, "k": k}
        g = B.qk_norm_bwd(st["q"], st["dq"], st["k"], st["dk"], **how)
        return {k: v for k, v in g.items() if v is not None}
    tokens, probs = B.sample(st["logits"], u=st["u"], temperature=st["temperature"], top_k=st["top_k"],
                             top_p=st["top_p"], min_p=st["min_p"], want_probs=case["out"] == "probs")
    return {"tokens": tokens} if case["out"] == "tokens" else {"probs": probs}


def _back(x, by, start, hist):
    """Row t - by of x for every row t; rows in front of a sequence are its history's last."""
    t = x.shape[0]
    at = torch.arange(t, device=x.device)
    inside = at - by >= start
    rows = x[(at - by).clamp_min(0)]
    if hist is None:
        return torch.where(inside[:, None], rows, torch.zeros_like(rows))
    seq, h = hist
    slot = (h.shape[1] + at - by - start).clamp(0, max(h.shape[1] - 1, 0))
    return torch.where(inside[:, None], rows, h[seq, slot].float())


def _short_conv(st):
    case = st["case"]
    dt, k = DTYPES[case["dtype"]], case["taps"]
    x, w = st["x"].float(), st["w"].float()
    bias = st["bias"].float() if case["bias"] else torch.zeros_like(w[:, 0])
    if case["pass"] == "step":
        rows = torch.cat([st["hist"].float(), x[:, None]], 1)            # [N, K, C]
        s = (rows * w.t()).sum(1) + bias
        y = s * torch.sigmoid(s) if case["act"] == "silu" else s
        hist = torch.cat([st["hist"], st["x"][:, None]], 1)[:, 1:]
        return {"y": y.to(dt), "hist": hist.contiguous()}
    cu = st["cu"].long()
    lens = cu[1:] - cu[:-1]
    n, t = lens.numel(), x.shape[0]
    seq = torch.repeat_interleave(torch.arange(n, device=x.device), lens, output_size=t)
    start = cu[:-1][seq]
    carried = None if st["hist"] is None else (seq, st["hist"])
    s = bias + w[:, k - 1] * x
    for by in range(1, k):
        s = s + w[:, k - 1 - by] * _back(x, by, start, carried)
    if case["pass"] == "fwd":
        y = s * torch.sigmoid(s) if case["act"] == "silu" else s
        if st["hist"] is None:
            return {"y": y.to(dt)}
        at = cu[1:, None] - (k - 1) + torch.arange(k - 1, device=x.device)   # rows that the histories end with
        old = (lens[:, None] + torch.arange(k - 1, device=x.device)).clamp_max(max(k - 2, 0))
        own_row = at >= cu[:-1, None]
        new = st["x"][at.clamp(0, max(t - 1, 0))] if t else torch.zeros_like(st["hist"])
        kept = st["hist"][torch.arange(n, device=x.device)[:, None], old]
        return {"y": y.to(dt), "hist": torch.where(own_row[..., None], new, kept)}
    sig = torch.sigmoid(s)
    ds = st["dy"].float()
    if case["act"] == "silu":
        ds = ds * sig * (1 + s * (1 - sig))
    del s, sig
    end = cu[1:][seq]
    at = torch.arange(t, device=x.device)
    dx = w[:, k - 1] * ds
    dw = [(ds * x).sum(0)]
    for by in range(1, k):                           # x's row is tap k - 1 - by of the row `by` behind it
        later = (at + by < end)[:, None]
        dx = dx + w[:, k - 1 - by] * torch.where(later, ds[(at + by).clamp_max(t - 1)], torch.zeros_like(ds))
        dw.append((ds * _back(x, by, start, carried)).sum(0))
    out = {"x": dx.to(dt), "w": torch.stack(dw[::-1], 1)}
    if case["bias"]:
        out["bias"] = ds.sum(0)
    if st["hist"] is not None:                       # slot m is tap m - p of the sequence's row p <= m
        dh = torch.zeros(st["hist"].shape, device=x.device)
        for p in range(k - 1):
            there = (lens > p)[:, None]
            row = ds[(cu[:-1] + p).clamp_max(t - 1)] if t else torch.zeros(n, x.shape[1], device=x.device)
            row = torch.where(there, row, torch.zeros_like(row))
            for m in range(p, k - 1):
                dh[:, m] += w[:, m - p] * row
        out["hist"] = dh.to(dt)
    return out


def _angles(st):
    """cos and sin of position times frequency, [T, 1, rot / 2]: the product and the angle in 64 bits."""
    a = st["positions"].double()[:, None] * st["freqs"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, rot, layout, cos, sin):
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _qk_norm(st):
    case = st["case"]
    dt, rot, layout = DTYPES[case["dtype"]], case["rot"], case["layout"]
    if rot:
        cos, sin = _angles(st)
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        w = st["w" + name].float() if case["weight"] else None
        rstd = torch.ones_like(x[..., :1])
        if case["norm"] != "none":
            ss = (x * x).sum(-1, keepdim=True)
            rstd = torch.rsqrt((ss / case["d"] if case["norm"] == "rms" else ss) + EPS)
        xh = x * rstd
        if case["pass"] == "fwd":
            y = xh if w is None else xh * w
            out[name] = (_rotate(y, rot, layout, cos, sin) if rot else y).to(dt)
            continue
        e = st["d" + name].float()
        if rot:                                      # the rotation back
            e = _rotate(e, rot, layout, cos, -sin)
        if w is not None:
            out["w" + name] = (e * xh).sum((0, 1))
            e = e * w
        if case["norm"] != "none":
            dot = (e * xh).sum(-1, keepdim=True)
            e = rstd * (e - xh * (dot / case["d"] if case["norm"] == "rms" else dot))
        out[name] = e.to(dt)
    return out


def _sample(st):
    """Prefixes of the order of falling logits (ties: the lowest index first), in 64 bits: sums of
    10^5 weights and the borders between them."""
    logits = st["logits"]
    n, v = logits.shape
    order_l, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    z = order_l.double()
    live = z > -math.inf
    t = st["temperature"].double()[:, None]
    greedy = ~(t > 0)
    rank = torch.arange(v, device=logits.device)
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, torch.ones_like(t), t))
    keep = live & ((rank == 0) | ~greedy)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep = keep & ((rank < k) | (k <= 0))
    w = torch.where(keep, w, torch.zeros_like(w))
    if st["top_p"] is not None:
        c = torch.cumsum(w, -1)
        p = st["top_p"].double()[:, None]
        before = torch.cat([torch.zeros_like(c[:, :1]), c[:, :-1]], -1)
        in_p = (before < p * c[:, -1:]) | ~(p < 1) | (rank == 0)
        if st["min_p"] is not None:
            in_p = in_p & ((w >= st["min_p"].double()[:, None]) | (rank == 0))
        keep = keep & in_p
    elif st["min_p"] is not None:
        keep = keep & ((w >= st["min_p"].double()[:, None]) | (rank == 0))
    w = torch.where(keep, w, torch.zeros_like(w))
    c = torch.cumsum(w, -1)
    if st["u"] is None:
        probs = torch.empty_like(w).scatter_(1, order, w / c[:, -1:])
        return {"probs": probs.float()}
    hit = keep & (c > st["u"].double()[:, None] * c[:, -1:])
    last = torch.where(keep & (w > 0), rank, 0).amax(-1)
    first = torch.where(hit, rank, v).amin(-1)
    at = torch.where(hit.any(-1), first, last)
    return {"tokens": order.gather(1, at[:, None])[:, 0].to(torch.int32)}


PLAIN = {"short_conv": _short_conv, "qk_norm": _qk_norm, "sample": _sample}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in st.items()}
    return EXACT[case["op"]](case, d)


def _exact_short_conv(case, d):
    """Every sequence behind its own history in one long column, convolved as a whole; the
    backward by differentiating that."""
    k, w = case["taps"], d["w"]
    lens = _lens(case) if case["pass"] != "step" else [1] * case["seqs"]
    n, c = len(lens), case["channels"]
    dev = w.device
    where, heads, at = [], [], 0
    for m in lens:
        heads.append(torch.arange(at, at + k - 1))
        where.append(torch.arange(at + k - 1, at + k - 1 + m))
        at += k - 1 + m
    where = torch.cat(where).to(dev)
    heads = torch.stack(heads).to(dev)

    def conv(x, w, bias, hist):
        col = torch.zeros(at, c, dtype=torch.float64, device=dev)
        col = col.index_copy(0, where, x)
        if hist is not None and k > 1:
            col = col.index_copy(0, heads.flatten(), hist.reshape(-1, c))
        s = sum(col[m:at - (k - 1) + m] * w[:, m] for m in range(k))     # row r: the window that begins there
        s = s[where - (k - 1)]
        if bias is not None:
            s = s + bias
        return s / (1 + torch.exp(-s)) if case["act"] == "silu" else s, col

    if case["pass"] == "bwd":
        leaves = {"x": d["x"].contiguous(), "w": w, "bias": d["bias"], "hist": d["hist"]}
        leaves = {name: v.requires_grad_(True) for name, v in leaves.items() if v is not None}
        y, _ = conv(leaves["x"], leaves["w"], leaves.get("bias"), leaves.get("hist"))
        grads = torch.autograd.grad(y, list(leaves.values()), d["dy"], allow_unused=True)
        return {name: torch.zeros_like(v) if g is None else g for (name, v), g in zip(leaves.items(), grads)}
    y, col = conv(d["x"], w, d["bias"], d["hist"])
    if d["hist"] is None:
        return {"y": y}
    ends = heads + torch.tensor(lens, device=dev)[:, None]
    return {"y": y, "hist": col[ends.flatten()].view(n, k - 1, c)}


def _exact_qk_norm(case, d):
    """The rotation as a product of complex numbers; the backward by differentiating."""
    rot, D = case["rot"], case["d"]
    turn = None
    if rot:
        a = torch.outer(d["positions"].double(), d["freqs"])
        turn = torch.polar(torch.ones_like(a), a)[:, None]

    def f(x, w):
        if case["norm"] == "rms":
            x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS)
        elif case["norm"] == "l2":
            x = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) + EPS)
        if w is not None:
            x = x * w
        if not rot:
            return x
        if case["layout"] == "half":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            return torch.cat([z.real, z.imag, x[..., rot:]], -1)
        z = torch.complex(x[..., :rot:2], x[..., 1:rot:2]) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)

    out = {}
    for name in ("q", "k"):
        if case["pass"] == "fwd":
            out[name] = f(d[name], d["w" + name])
            continue
        x = d[name].clone().requires_grad_(True)
        w = d["w" + name].requires_grad_(True) if case["weight"] else None
        g = torch.autograd.grad(f(x, w), [x] + ([w] if w is not None else []), d["d" + name])
        out[name] = g[0]
        if w is not None:
            out["w" + name] = g[1]
    return out


def _exact_sample(case, d):
    """Row by row: the values that are left, cut at thresholds."""
    tokens, probs = [], []
    for r in range(case["rows"]):
        l = d["logits"][r]
        index = torch.nonzero(l > -math.inf)[:, 0]
        order = index[torch.argsort(-l[index], stable=True)]
        t = d["temperature"][r].item()
        if t <= 0:
            order = order[:1]
            t = 1.0
        if d["top_k"] is not None and d["top_k"][r].item() > 0:
            order = order[:d["top_k"][r].item()]
        w = torch.exp((l[order] - l[order[0]]) / t)
        keep = len(order)
        if d["top_p"] is not None and d["top_p"][r].item() < 1:
            c = torch.cumsum(w, 0)                   # the first at which the sum reaches the mass is the last
            keep = min(keep, int((c < d["top_p"][r] * c[-1]).sum()) + 1)
        if d["min_p"] is not None:
            keep = min(keep, max(1, int((w >= d["min_p"][r]).sum())))
        order, w = order[:keep], w[:keep]
        if case["out"] == "probs":
            row = torch.zeros_like(l)
            row[order] = w / w.sum()
            probs.append(row)
            continue
        c = torch.cumsum(w, 0)
        j = int(torch.searchsorted(c, d["u"][r] * c[-1], right=True))
        tokens.append(int(order[min(j, int(torch.nonzero(w)[-1]))]))
    if case["out"] == "probs":
        return {"probs": torch.stack(probs)}
    return {"tokens": torch.tensor(tokens, dtype=torch.int32, device=d["logits"].device)}


EXACT = {"short_conv": _exact_short_conv, "qk_norm": _exact_qk_norm, "sample": _exact_sample}
