"""The short convolution (prism_short_conv, its step and its gradients) against its formula in 64
bits, and the gradients against differences.

Tolerances.  An output is rounded once to its type (half a step: 2^-8 of the value for
bf16, 2^-24 for fp32).  Before it, in roundings of 2^-24: the sum s has K products and
additions and the bias, on the magnitude of its terms (K + 2); silu passes that on with a slope of at
most 1.1 and adds its own, some 8 roundings and one of the exponent, whose error grows with |s|
in bf16: 16 + 2 |s| on |y|.  The slope's own slope is at most 1/2, and its terms may cancel, so its
error counts on s (1 + |s| c).  dx adds K products.  A weight's gradient adds a run of 64
tokens a lane, up to 32 groups, a 64th of the workgroups and 6 more: 128 on the absolute terms,
where a lane has one run (up to a million elements here)."""
import numpy as np
import pytest

from tests import stack_refs as R
from tests.gpu_common import say
from tests.layer_refs import check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def offsets(lens):
    return [0] + list(np.cumsum(lens))


def make(lens, C, K, dtype="bf16", bias=True, hist=True, wide=0, seed=0, behind=0):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(seed)
    cu = [int(c) for c in offsets(lens)]
    T = cu[-1] + behind
    rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
    x = rand(T, C + wide)[:, wide:]
    return {"x": x, "w": rand(C, K), "bias": rand(C) if bias else None,
            "hist": rand(len(lens), K - 1, C) if hist else None, "dy": rand(T, C), "cu": cu,
            "cu_t": torch.tensor(cu, dtype=torch.int32).cuda()}


def check_all(d, act):
    """Forward and backward of one set of inputs; the worst share of a tolerance."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    K, live = d["w"].shape[1], d["cu"][-1]
    ho = None if d["hist"] is None else torch.empty_like(d["hist"])
    y, h = B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"], activation=act, hist=d["hist"], hist_out=ho)
    g = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], bias=d["bias"], activation=act, hist=d["hist"])
    silu = act == "silu"
    x6, w6, b6, h6, dy6 = f64(d["x"])[:live], f64(d["w"]), f64(d["bias"]), f64(d["hist"]), f64(d["dy"])[:live]
    leaves = [t.requires_grad_(True) for t in (x6, w6, b6, h6) if t is not None]
    ref, _, _ = R.short_conv(x6, w6, d["cu"], b6, silu, h6)
    grads = torch.autograd.grad((ref * dy6).sum(), leaves, allow_unused=True)
    grads = [torch.zeros_like(l) if r is None else r for l, r in zip(leaves, grads)]
    for t in leaves:
        t.requires_grad_(False)
    ey, ex, ew, eb, eh = R.conv_tolerances(x6, w6, d["cu"], dy6, b6, silu, h6)
    worst = max(check("y", y[:live], ref.detach(), ey, 1), check("dx", g["x"][:live], grads[0], ex, 1),
                check("dw", g["w"], grads[1], ew, 1))
    rest = grads[2:]
    if b6 is not None:
        worst = max(worst, check("dbias", g["bias"], rest.pop(0), eb, 1))
    else:
        assert g["bias"] is None
    if h6 is not None:
        if K > 1:
            worst = max(worst, check("dhist", g["hist"], rest.pop(0), eh, 1))
        assert h is ho and torch.equal(f64(ho), R.carried(x6, h6, d["cu"], K))
    else:
        assert g["hist"] is None and h is None
    assert (g["x"][live:] == 0).all()
    return worst


# empty sequences at both ends, single tokens, sequences that end with a run of 32 and 64 or one
# token off it, sequences shorter than the taps
LENS = [0, 1, 31, 1, 2, 0, 0, 3, 26, 33, 64, 7, 65, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("K", range(1, 9))
def test_taps(dtype, act, K):
    worst = max(check_all(make(LENS, 24, K, dtype, bias=K % 2 == 0, hist=h, seed=K), act) for h in (False, True))
    say(f"short_conv {K} taps {dtype} {act}: worst share of the tolerance {worst:.2f}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_channels(dtype):
    """Channels that fill vectors and workgroups, and do not; columns of a wider tensor, at any element."""
    worst = 0.0
    for C in (1, 2, 3, 7, 8, 9, 31, 64, 100, 130, 255, 257, 512, 520, 777):
        for wide in (0, 1, 8):
            worst = max(worst, check_all(make([5, 0, 37, 1], C, 4, dtype, wide=wide, seed=C), "silu"))
    say(f"short_conv channels {dtype}: worst share of the tolerance {worst:.2f}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_runs(dtype):
    """Long runs in the backward, several rounds of workgroups in the forward, and weight gradients of many
    tokens.  The reference by shifted sums of one sequence."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    T, C, K = 40_000, 2304 if dtype == "bf16" else 1152, 4
    d = make([T], C, K, dtype, hist=False, seed=5)
    y, _ = B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"])
    g = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], bias=d["bias"])
    cols = torch.arange(0, C, 97)
    x, w, b, dy = f64(d["x"][:, cols]), f64(d["w"][cols]), f64(d["bias"][cols]), f64(d["dy"][:, cols])
    xp = torch.cat([torch.zeros(K - 1, x.shape[1]).double(), x])
    s = sum(xp[m:m + T] * w[:, m] for m in range(K)) + b
    mag = sum((xp[m:m + T] * w[:, m]).abs() for m in range(K)) + b.abs()
    sig = torch.sigmoid(s)
    es = (K + 2) * mag
    check("y", y[:, cols], s * sig, 1.1 * es + (16 + 2 * s.abs()) * (s * sig).abs(), 1)
    slope, top = sig * (1 + s * (1 - sig)), sig * (1 + s.abs() * (1 - sig))
    ds, dsa = dy * slope, dy.abs() * top
    eds = dy.abs() * (0.5 * es + (16 + 2 * s.abs()) * top)
    dsp = torch.cat([ds, torch.zeros(K - 1, x.shape[1]).double()])
    pad = lambda v: torch.cat([v, torch.zeros(K - 1, x.shape[1]).double()])
    check("dx", g["x"][:, cols], sum(w[:, m] * dsp[K - 1 - m:K - 1 - m + T] for m in range(K)),
          sum(w[:, m].abs() * pad(eds + (K + 1) * dsa)[K - 1 - m:K - 1 - m + T] for m in range(K)), 1)
    # a lane adds its run of tokens, then come the lanes of a workgroup and the workgroups: at most 300 here
    adds = 300 + 64
    dw = torch.stack([(ds * xp[m:m + T]).sum(0) for m in range(K)], 1)
    ew = torch.stack([((eds + adds * dsa) * xp[m:m + T].abs()).sum(0) for m in range(K)], 1)
    check("dw", g["w"][cols], dw, ew, 1)
    check("dbias", g["bias"][cols], ds.sum(0), (eds + adds * dsa).sum(0), 1)
    again = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], bias=d["bias"])
    assert all(torch.equal(g[n], again[n]) for n in ("x", "w", "bias"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 4, 7])
def test_steps_continue_a_prompt(dtype, K):
    """Prompts in one call, then token by token in place: the same as the whole sequences at once."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    N, C, whole, cut = 5, 70, 9, 4
    d = make([whole] * N, C, K, dtype, hist=False, seed=K)
    ref, _ = B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"])
    x = d["x"].view(N, whole, C)
    hist = torch.full((N, K - 1, C), 7.0, dtype=x.dtype, device="cuda")
    cu = torch.arange(0, N * cut + 1, cut, dtype=torch.int32).cuda()
    y, h = B.short_conv(x[:, :cut].reshape(N * cut, C), d["w"], cu, bias=d["bias"], hist_out=hist)
    assert h is hist
    outs = [y.view(N, cut, C)]
    for t in range(cut, whole):
        before = hist.clone()
        y2, h2 = B.short_conv_step(x[:, t], d["w"], hist, bias=d["bias"], hist_out=torch.empty_like(hist))
        y1, h1 = B.short_conv_step(x[:, t], d["w"], hist, bias=d["bias"])      # rows N apart: a strided x
        assert h1 is hist and torch.equal(y1, y2) and torch.equal(hist, h2)
        if K > 1:
            assert torch.equal(hist, torch.cat([before[:, 1:], x[:, t:t + 1]], 1))
        outs.append(y1[:, None])
    assert torch.equal(torch.cat(outs, 1).reshape(N * whole, C), ref)


def test_history_in_place():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    for C in (16, 17):
        d = make(LENS, C, 4, seed=3)
        other = torch.empty_like(d["hist"])
        y, _ = B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"], hist=d["hist"], hist_out=other)
        h = d["hist"].clone()
        y2, h2 = B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"], hist=h, hist_out=h)
        assert h2 is h and torch.equal(y, y2) and torch.equal(h, other)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence(dtype):
    """They are neither read nor written, whatever they hold; dx is zero there."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    for lens, behind in (([5, 60, 0], 70), ([64, 32], 3), ([0, 0], 40)):
        d = make(lens, 40, 4, dtype, behind=behind, seed=behind)
        live = d["cu"][-1]
        d["x"][live:] = float("nan")
        d["dy"][live:] = float("inf")
        y = torch.full_like(d["dy"], 3.0)
        check_all(d, "silu")
        B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"], hist=d["hist"], y=y)
        assert (y[live:] == 3.0).all() and torch.isfinite(y).all()


def test_values_that_are_not_finite_stay_in_their_window():
    """An infinity or NaN reaches the K rows that its row is a tap of, in its channel, and
    neither the neighbours' sequences nor their gradients."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    for bad in (float("inf"), float("nan")):
        d = make([10, 12, 11], 16, 4, "f32", hist=False, seed=1)
        clean, _ = B.short_conv(d["x"], d["w"], d["cu_t"], activation=None)
        gc = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], activation=None)
        for row, rows in ((14, range(14, 18)), (9, range(9, 10)), (21, range(21, 22)), (22, range(22, 26))):
            x = d["x"].clone()
            x[row, 3] = bad
            y, _ = B.short_conv(x, d["w"], d["cu_t"], activation=None)
            hit = torch.zeros_like(y, dtype=torch.bool)
            hit[list(rows), 3] = True
            assert torch.equal(torch.isfinite(y), ~hit) and torch.equal(y[~hit], clean[~hit])
        dy = d["dy"].clone()
        dy[15, 3] = bad                                       # reaches dx of rows 12..15
        g = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], dy, activation=None)
        hit = torch.zeros_like(dy, dtype=torch.bool)
        hit[12:16, 3] = True
        assert torch.equal(torch.isfinite(g["x"]), ~hit) and torch.equal(g["x"][~hit], gc["x"][~hit])
        dy = d["dy"].clone()
        dy[10, 3] = bad                                       # the first row of a sequence: its own dx alone
        g = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], dy, activation=None)
        hit[:] = False
        hit[10, 3] = True
        assert torch.equal(torch.isfinite(g["x"]), ~hit)


def test_open_and_closed_gates():
    """Sums of either sign up to where the exponential overflows."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    s = torch.tensor([-3e38, -200., -100., -88., -20., -1., -1e-30, 0., 1e-30, 1., 20., 88., 200., 3e38])
    x = s.repeat(8, 1).t().contiguous().cuda()
    one = torch.ones(8, 1).cuda()
    cu = torch.tensor([0, len(s)], dtype=torch.int32).cuda()
    y, _ = B.short_conv(x, one, cu)
    ref = s.double() / (1 + torch.exp(-s.double()))
    assert ((f64(y) - ref[:, None]).abs() <= 16 * 2.0 ** -24 * ref.abs()[:, None] + 2.0 ** -126).all()
    g = B.short_conv_bwd(x, one, cu, torch.ones_like(x))
    sig = 1 / (1 + torch.exp(-s.double()))
    c = 1 / (1 + torch.exp(s.double()))
    slope = sig * (1 + s.double() * c)
    mag = sig * (1 + s.double().abs() * c)
    assert ((f64(g["x"]) - slope[:, None]).abs() <= 16 * 2.0 ** -24 * mag[:, None] + 2.0 ** -126).all()


def test_gradients_against_differences():
    import torch
    from gated_delta_rule_prologue_amd.autograd import short_conv
    d = make([6, 0, 9, 2], 5, 3, "f32", seed=9)
    names = ("x", "w", "bias", "hist")
    leaves = {n: d[n].clone().requires_grad_(True) for n in names}
    up = d["dy"]

    def loss(v):
        return (short_conv(v["x"], v["w"], d["cu_t"], v["bias"], "silu", v["hist"]).double() * up.double()).sum()

    grads = torch.autograd.grad(loss(leaves), list(leaves.values()))
    h = 2.0 ** -8                                             # error h^2 of the third derivative, 2^-24 / h of the values
    for name, g in zip(names, grads):
        flat = leaves[name].detach().reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 7)):
            v = {n: t.detach().clone() for n, t in leaves.items()}
            vals = []
            for sign in (1, -1):
                v[name] = flat.clone().index_add_(0, torch.tensor([i]).cuda(), torch.tensor([sign * h]).cuda()).view_as(leaves[name])
                vals.append(loss(v).item())
            diff = (vals[0] - vals[1]) / (2 * h)
            assert abs(diff - g.reshape(-1)[i].item()) <= 2e-2 * (1 + abs(diff)), (name, i)


def test_autograd_returns_what_is_asked_for():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    from gated_delta_rule_prologue_amd.autograd import short_conv
    d = make([20, 3], 24, 4, seed=2)
    full = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], bias=d["bias"], hist=d["hist"])
    for want in ("x", "w", "bias", "hist"):
        v = {n: d[n].detach().clone().requires_grad_(n == want) for n in ("x", "w", "bias", "hist")}
        y = short_conv(v["x"], v["w"], d["cu_t"], v["bias"], "silu", v["hist"])
        y.backward(d["dy"])
        assert torch.equal(v[want].grad, full[want].to(v[want].dtype))
        assert all(v[n].grad is None for n in v if n != want)
    # an expanded upstream gradient, one that starts at any element, and columns of a projection
    p = torch.randn(23, 30, dtype=torch.bfloat16, device="cuda").requires_grad_(True)
    y = short_conv(p[:, 3:27], d["w"], d["cu_t"])
    y.sum().backward()
    g = B.short_conv_bwd(p.detach()[:, 3:27], d["w"], d["cu_t"], torch.ones_like(d["dy"]))
    assert torch.equal(p.grad[:, 3:27], g["x"]) and (p.grad[:, :3] == 0).all()
    with pytest.raises(RuntimeError):
        v = d["x"].detach().clone().requires_grad_(True)
        gx, = torch.autograd.grad(short_conv(v, d["w"], d["cu_t"]).float().sum(), v, create_graph=True)
        gx.float().sum().backward()


def test_no_tokens():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    d = make([0, 0, 0], 16, 4)
    ho = torch.empty_like(d["hist"])
    y, _ = B.short_conv(d["x"], d["w"], d["cu_t"], bias=d["bias"], hist=d["hist"], hist_out=ho)
    assert y.shape == (0, 16) and torch.equal(ho, d["hist"])
    g = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], bias=d["bias"], hist=d["hist"])
    assert all((g[n] == 0).all() for n in ("w", "bias", "hist"))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last sequence's values are those that it has alone."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    C, T, last = 4096, 530_000, 301
    assert C * T > 2 ** 31
    gen = torch.Generator().manual_seed(12)
    x = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    x[-last - 2:] = torch.randn(last + 2, C, generator=gen).to(x)
    dy[-last:] = torch.randn(last, C, generator=gen).to(x)
    w, bias = torch.randn(C, 4, generator=gen).to(x), torch.randn(C, generator=gen).to(x)
    hist = torch.randn(2, 3, C, generator=gen).to(x)
    cu = torch.tensor([0, T - last, T], dtype=torch.int32).cuda()
    alone = torch.tensor([0, last], dtype=torch.int32).cuda()
    ho, ho1 = torch.empty_like(hist), torch.empty_like(hist[1:])
    y, _ = B.short_conv(x, w, cu, bias=bias, hist=hist, hist_out=ho)
    y1, _ = B.short_conv(x[-last:], w, alone, bias=bias, hist=hist[1:], hist_out=ho1)
    assert torch.equal(y[-last:], y1) and torch.equal(ho[1:], ho1) and torch.equal(ho[0, 1:], x[-last - 2:-last])
    del y
    g = B.short_conv_bwd(x, w, cu, dy, bias=bias, hist=hist)
    g1 = B.short_conv_bwd(x[-last:], w, alone, dy[-last:], bias=bias, hist=hist[1:])
    assert torch.equal(g["x"][-last:], g1["x"]) and torch.equal(g["hist"][1:], g1["hist"])
    # sums of the same 301 terms beside zeros, in two orders: 301 roundings of their magnitudes each
    size = (dy[-last:].float().abs() * 1.1).sum(0)
    assert ((g["bias"] - g1["bias"]).abs() <= 2 * 301 * 2.0 ** -24 * size).all()


def test_gradient_of_a_bias_that_is_zero():
    """The C entry forms dbias without a bias too: that of a bias of zeros."""
    import ctypes
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    d = make([37, 0, 260, 3], 48, 4, "f32", bias=False, hist=False, seed=21)
    T, C = d["x"].shape
    zero = torch.zeros(C, device="cuda")
    want = B.short_conv_bwd(d["x"], d["w"], d["cu_t"], d["dy"], bias=zero)
    dims = B.ConvDims(4, T, C, 4, 0, C)
    dx, dw, db = torch.empty_like(d["x"]), torch.empty(C, 4, device="cuda"), torch.full((C,), 7.0, device="cuda")
    ws = torch.empty(B.conv_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    got = B.lib().prism_short_conv_bwd(ctypes.byref(dims), p(d["x"]), p(d["w"]), None, None, p(d["cu_t"]), 1, p(d["dy"]), p(dx),
                                       p(dw), p(db), None, p(ws), ws.numel(),
                                       ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert got == B.PRISM_OK
    assert torch.equal(dx, want["x"]) and torch.equal(dw, want["w"]) and torch.equal(db, want["bias"])
