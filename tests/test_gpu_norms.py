"""The norms around the operator (prism_norm_residual, prism_norm_gate and their
gradients) against their formulas in 64 bits, and the gradients against
differences.

Tolerances.  An output is rounded once to its type (half a step: 2^-8 of the value
for bf16, 2^-24 for fp32), after fp32 arithmetic whose error is counted in
roundings of 2^-24 on the magnitude of the terms that are added up, never on a
sum that cancels.  A row's sum of squares has at most 16 terms a lane, then 9 + 8
additions across lanes and wavefronts: 33 roundings of positive terms, halved by
the square root; with the root, the products and the activation (exp2 and
reciprocal to one step each, a few products) 64 covers a forward output.  A
gradient holds a second such sum whose terms cancel: its magnitude is the sum
of their absolute values, and 128 covers it.  A weight's gradient adds at most
rows / (workgroups x groups) terms a lane, 32 groups, 1024 / 64 partials and 6
more: 80 beyond the 128 at up to 20 rows a lane."""
import numpy as np
import pytest

from tests.gpu_common import say
from tests.layer_refs import check, f64
from tests import layer_refs as R

pytestmark = pytest.mark.gpu
FWD, BWD, SUM = 64, 128, 208
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def rand(gen, shape, dt, mul=1.0, add=0.0):
    import torch
    return (mul * torch.randn(shape, generator=gen) + add).to(dt).cuda()


def dtypes():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


# widths: one element, below a vector, odd, every register shape's edges (vectors of 8 bf16 or
# 4 fp32 in rows of 8, 16, 32, 64 lanes, then 2 to 4 vectors a lane and whole
# workgroups; single elements in rows of 8 lanes to a workgroup of 512)
WIDTHS = [1, 2, 7, 8, 12, 32, 63, 64, 65, 72, 128, 136, 250, 256, 264, 512, 516, 520, 768, 1001, 1024, 1028,
          1032, 2048, 2052, 2056, 3001, 4096, 4100, 4104, 8191, 8192]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["plain", "add", "scaled"])
def test_norm_residual_widths(dtype, form):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dt = dtypes()[dtype]
    worst = 0.0
    for width in WIDTHS:
        gen = torch.Generator().manual_seed(width)
        rows = 9 if width > 64 else 130
        x, w = rand(gen, (rows, width), dt, 2.0), rand(gen, width, dt, 0.2, 1.0)
        y = rand(gen, (rows, width), dt) if form != "plain" else None
        s = rand(gen, width, dt, 0.3, 0.5) if form == "scaled" else None
        n, r = B.norm_residual(x, w, y=y, scale=s, eps=EPS)
        nr, rr, nmag, rmag = R.norm_residual(f64(x), f64(w), f64(y), f64(s), EPS)
        worst = max(worst, check(f"n {width}", n, nr, nmag, FWD))
        if y is None:
            assert r is x
        else:
            worst = max(worst, check(f"r {width}", r, rr, rmag, 3))
    say(f"norm_residual {dtype} {form}: worst share of the tolerance {worst:.2f}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["plain", "add", "scaled"])
def test_norm_residual_bwd_widths(dtype, form):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dt = dtypes()[dtype]
    worst = 0.0
    for width in WIDTHS:
        gen = torch.Generator().manual_seed(width + 1)
        rows = 11 if width > 64 else 150
        r, w, dn = rand(gen, (rows, width), dt, 2.0), rand(gen, width, dt, 0.2, 1.0), rand(gen, (rows, width), dt)
        dr = rand(gen, (rows, width), dt) if form != "plain" else None
        y = rand(gen, (rows, width), dt) if form == "scaled" else None
        s = rand(gen, width, dt, 0.3, 0.5) if form == "scaled" else None
        g = B.norm_residual_bwd(r, w, dn, dr=dr, y=y, scale=s, eps=EPS)
        r6, w6, dn6 = f64(r).requires_grad_(True), f64(w).requires_grad_(True), f64(dn)
        t, dw = torch.autograd.grad(R.norm_residual_loss(r6, w6, None, None, EPS, dn6,
                                                         None if dr is None else f64(dr)), (r6, w6))
        r6, w6 = r6.detach(), w6.detach()
        rstd = 1 / torch.sqrt((r6 * r6).mean(-1, keepdim=True) + EPS)
        e, rh = (dn6 * w6).abs(), (r6 * rstd).abs()
        mag = rstd * (e + rh * (e * rh).mean(-1, keepdim=True)) + (0 if dr is None else f64(dr).abs())
        worst = max(worst, check(f"dx {width}", g["x"], t, mag, BWD),
                    check(f"dw {width}", g["w"], dw, (dn6.abs() * rh).sum(0), SUM))
        if s is not None:
            s6, y6 = f64(s), f64(y)
            worst = max(worst, check(f"dy {width}", g["y"], s6 * t, s6.abs() * mag, BWD),
                        check(f"ds {width}", g["scale"], (t * y6).sum(0), (mag * y6.abs()).sum(0), SUM))
        else:
            assert g["scale"] is None and g["y"] is None
    say(f"norm_residual_bwd {dtype} {form}: worst share of the tolerance {worst:.2f}")


GATE_WIDTHS = [1, 5, 8, 16, 63, 64, 72, 96, 128, 130, 256, 260, 512, 520, 768, 1000, 1001, 1024]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_gate_widths(dtype, gate, per_head):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dt = dtypes()[dtype]
    worst = 0.0
    for i, width in enumerate(GATE_WIDTHS):
        gen = torch.Generator().manual_seed(width + 2)
        T, H = (37, 3) if i % 2 else (5, 7)
        o, z = rand(gen, (T, H, width), dt, 0.3), rand(gen, (T, H, width), dt, 2.0)
        w = rand(gen, (H, width) if per_head else (width,), dt, 0.2, 1.0)
        dy = rand(gen, (T, H, width), dt)
        y = B.norm_gate(o, z, w, eps=EPS, gate=gate)
        leaves = [f64(t).requires_grad_(True) for t in (o, z, w)]
        ref = R.norm_gate(*leaves, EPS, gate)
        # the sigmoid's argument is rounded before exp2: its error grows with |z|
        zmag = 1 + leaves[1].detach().abs()
        worst = max(worst, check(f"y {width}", y, ref.detach(), ref.detach().abs() * zmag, FWD))
        g = B.norm_gate_bwd(o, z, w, dy, eps=EPS, gate=gate)
        do, dz, dw = torch.autograd.grad((ref * f64(dy)).sum(), leaves)
        o6, z6, w6 = (t.detach() for t in leaves)
        rstd = 1 / torch.sqrt((o6 * o6).mean(-1, keepdim=True) + EPS)
        oh = (o6 * rstd).abs()
        act = torch.sigmoid(z6) * (z6.abs() if gate == "silu" else 1)
        e = f64(dy).abs() * act * w6.abs() * zmag
        # the slope s (1 + z (1 - s)) cancels near its zero
        slope = torch.sigmoid(z6) * ((1 + z6.abs() * torch.sigmoid(-z6)) if gate == "silu" else 1) * zmag
        worst = max(worst,
                    check(f"do {width}", g["o"], do, rstd * (e + oh * (e * oh).mean(-1, keepdim=True)), BWD),
                    check(f"dz {width}", g["z"], dz, f64(dy).abs() * oh * w6.abs() * slope, BWD),
                    check(f"dw {width}", g["w"], dw,
                          (f64(dy).abs() * act * zmag * oh).sum(0) if per_head
                          else (f64(dy).abs() * act * zmag * oh).sum((0, 1)), SUM))
    say(f"norm_gate {dtype} {gate} per_head={per_head}: worst share of the tolerance {worst:.2f}")


@pytest.mark.parametrize("rows", [0, 1, 2, 1023, 1025, 20000])
def test_row_counts(rows):
    """From no row to more rows than workgroups, both norms and directions."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(rows)
    dt, width = torch.bfloat16, 64
    x, y, dn = (rand(gen, (rows, width), dt) for _ in range(3))
    w, s = rand(gen, width, dt, 0.2, 1.0), rand(gen, width, dt, 0.3, 0.5)
    n, r = B.norm_residual(x, w, y=y, scale=s)
    nr, rr, nmag, rmag = R.norm_residual(f64(x), f64(w), f64(y), f64(s), EPS)
    check("n", n, nr, nmag, FWD)
    check("r", r, rr, rmag, 3)
    g = B.norm_residual_bwd(r, w, dn, dr=None, y=y, scale=s)
    r6, w6 = f64(r).requires_grad_(True), f64(w).requires_grad_(True)
    t, dw = torch.autograd.grad(R.norm_residual_loss(r6, w6, None, None, EPS, f64(dn), None), (r6, w6))
    check("dw", g["w"], dw, (f64(dn).abs() * f64(r).abs() * 2).sum(0) + 1, SUM)
    check("ds", g["scale"], (t * f64(y)).sum(0), (f64(y).abs() * 16).sum(0) + 1, SUM)
    if rows % 2 == 0:
        o = x.view(rows // 2, 2, width)
        w2 = rand(gen, (2, width), dt, 0.2, 1.0)
        g = B.norm_gate_bwd(o, y.view_as(o), w2, dn.view_as(o))
        leaves = [f64(v).requires_grad_(True) for v in (o, y.view_as(o), w2)]
        ref = torch.autograd.grad((R.norm_gate(*leaves, EPS, "silu") * f64(dn).view(o.shape)).sum(), leaves)
        check("gate dw", g["w"], ref[2], (f64(dn).abs() * 16 * f64(y).abs()).sum() + 1, SUM)
        assert B.norm_gate(o, y.view_as(o), w2).shape == o.shape


def test_special_values():
    """Zero rows, the type's lowest values as a gate, infinities and NaN: as the formula
    has them, and in their own row alone."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    for dt in (torch.bfloat16, torch.float32):
        gen = torch.Generator().manual_seed(5)
        x, w = rand(gen, (6, 96), dt), rand(gen, 96, dt, 0.2, 1.0)
        x[1] = 0
        x[3, 5] = float("inf")
        x[4, 7] = float("nan")
        n, _ = B.norm_residual(x, w)
        n6 = R.norm_residual(f64(x), f64(w), None, None, EPS)[0]
        assert torch.equal(n[1].cpu().float(), torch.zeros(96))
        assert torch.isnan(n[4]).all() and torch.isnan(n[3, 5])
        for i in (0, 1, 2, 5):
            check("n", n[i], n6[i], n6[i].abs(), FWD)
        z = rand(gen, (6, 96), dt)
        z[0] = torch.finfo(dt).min
        z[2] = torch.finfo(dt).max
        z[5] = -100.0
        o = rand(gen, (6, 96), dt, 0.3)
        for gate in ("silu", "sigmoid"):
            y = B.norm_gate(o, z, w, gate=gate)
            assert torch.isfinite(y[[0, 1, 3, 4, 5]]).all(), gate
            assert (y[0].float().abs() == 0).all() and (y[5].float().abs() < 1e-30).all()
            if gate == "sigmoid":
                ref = R.norm_gate(f64(o), f64(z), f64(w), EPS, gate)
                check("y", y[2], ref[2], ref[2].abs(), FWD)
            g = B.norm_gate_bwd(o, z, w, torch.ones_like(o), gate=gate)
            assert torch.isfinite(g["o"][[0, 1, 3, 4, 5]]).all() and torch.isfinite(g["z"][[0, 1, 3, 4, 5]]).all()


def test_in_place_and_rows_behind():
    """Outputs may be the inputs' buffers, and nothing behind the rows is written."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(9)
    for width in (64, 768, 1001, 4096):
        dt = torch.bfloat16
        base = [rand(gen, (40, width), dt) for _ in range(4)]
        w, s = rand(gen, width, dt, 0.2, 1.0), rand(gen, width, dt, 0.3, 0.5)
        x, y = base[0][:33], base[1][:33]
        n_ref, r_ref = B.norm_residual(x, w, y=y, scale=s)
        tail = [b[33:].clone() for b in base]
        n, r = B.norm_residual(x, w, y=y, scale=s, r=x, n=y)
        assert r is x and n is y and torch.equal(r, r_ref) and torch.equal(n, n_ref)
        if width <= 1024:
            o, z = base[2][:33], base[3][:33]
            ref = B.norm_gate(o, z, w)
            assert torch.equal(B.norm_gate(o, z, w, y=z), ref)
        assert all(torch.equal(b[33:], t) for b, t in zip(base, tail))


def test_same_bits_twice():
    """The column sums do not depend on timing."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(3)
    r, dn, y = (rand(gen, (9000, 200), torch.bfloat16) for _ in range(3))
    w, s = rand(gen, 200, torch.bfloat16, 0.2, 1.0), rand(gen, 200, torch.bfloat16)
    a = B.norm_residual_bwd(r, w, dn, y=y, scale=s)
    b = B.norm_residual_bwd(r, w, dn, y=y, scale=s)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_gradients_against_differences():
    """(L(x + h d) - L(x - h d)) / 2h = <dL/dx, d> up to O(h^2): in fp32, with L summed in 64
    bits.  h = 2^-6: the third derivative along a random unit-variance d of these
    functions is a few times L's own scale n (one per element), h^2 / 6 of it below
    1e-3 n^(1/2) for random signs; an fp32 output's rounding adds 2^-24 / h = 4e-6 an
    element.  Bound: 5e-3 of the gradient's scale |g| |d|."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(4)
    f32, h = torch.float32, 2.0 ** -6
    x, y, dn, dr = (rand(gen, (12, 100), f32) for _ in range(4))
    w, s = rand(gen, 100, f32, 0.2, 1.0), rand(gen, 100, f32, 0.3, 0.5)

    def res(x, w, y, s):
        n, r = B.norm_residual(x, w, y=y, scale=s)
        return float((f64(n) * f64(dn)).sum() + (f64(r) * f64(dr)).sum())

    _, r = B.norm_residual(x, w, y=y, scale=s)
    g = B.norm_residual_bwd(r, w, dn, dr=dr, y=y, scale=s)
    args = {"x": x, "w": w, "y": y, "scale": s}
    for name in args:
        d = rand(gen, args[name].shape, f32)
        hi = res(*[v + h * d if k == name else v for k, v in args.items()])
        lo = res(*[v - h * d if k == name else v for k, v in args.items()])
        want, got = float((f64(g[name]) * f64(d)).sum()), (hi - lo) / (2 * h)
        say(f"norm_residual d{name}: {got:.6f} by differences, {want:.6f}")
        assert abs(got - want) <= 5e-3 * float(f64(g[name]).norm() * f64(d).norm()), name
    o, z, dy = (rand(gen, (6, 2, 64), f32) for _ in range(3))
    w = rand(gen, (2, 64), f32, 0.2, 1.0)
    for gate in ("silu", "sigmoid"):
        g = B.norm_gate_bwd(o, z, w, dy, gate=gate)
        args = {"o": o, "z": z, "w": w}
        for name in args:
            d = rand(gen, args[name].shape, f32)
            run = lambda sign: float((f64(B.norm_gate(*[v + sign * h * d if k == name else v
                                                        for k, v in args.items()], gate=gate)) * f64(dy)).sum())
            want, got = float((f64(g[name]) * f64(d)).sum()), (run(1) - run(-1)) / (2 * h)
            assert abs(got - want) <= 5e-3 * float(f64(g[name]).norm() * f64(d).norm()), (gate, name, got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd(dtype):
    """autograd.norm_residual and norm_gate give the bound gradients in each leaf's dtype,
    with unused outputs, strided upstream gradients and no add."""
    import torch
    from gated_delta_rule_prologue_amd import autograd as A, binding as B
    dt = dtypes()[dtype]
    gen = torch.Generator().manual_seed(8)
    x, y, dn, dr = (rand(gen, (30, 64), dt) for _ in range(4))
    w, s = rand(gen, 64, dt, 0.2, 1.0), rand(gen, 64, dt, 0.3, 0.5)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, y, s)]
    n, r = A.norm_residual(leaves[0], leaves[1], y=leaves[2], scale=leaves[3])
    got = torch.autograd.grad([n, r], leaves, [dn, dr.t().contiguous().t()])
    ref = B.norm_residual_bwd(r.detach(), w, dn, dr=dr, y=y, scale=s)
    for a, name in zip(got, ("x", "w", "y", "scale")):
        assert a.dtype == dt and torch.equal(a, ref[name].to(dt)), name
    # only r used; only n used, without a scale; no add at all
    n, r = A.norm_residual(leaves[0], leaves[1], y=leaves[2])
    gx, gy = torch.autograd.grad(r, [leaves[0], leaves[2]], dr)
    assert torch.equal(gx, dr) and torch.equal(gy, dr)
    n, r = A.norm_residual(leaves[0], leaves[1], y=leaves[2])
    gx, gw, gy = torch.autograd.grad(n, [leaves[0], leaves[1], leaves[2]], dn)
    ref = B.norm_residual_bwd(r.detach(), w, dn)
    assert torch.equal(gx, ref["x"]) and torch.equal(gy, ref["x"]) and torch.equal(gw, ref["w"].to(dt))
    n, r = A.norm_residual(leaves[0], leaves[1])
    assert r is leaves[0]
    gx, = torch.autograd.grad([n, r * 2], [leaves[0]], [dn, dr])
    ref = f64(B.norm_residual_bwd(x, w, dn)["x"]) + 2 * f64(dr)
    assert (f64(gx) - ref).abs().max() <= 2.0 ** -7 * ref.abs().max()
    o, z, wg = x.view(15, 2, 64), y.view(15, 2, 64), rand(gen, (2, 64), dt, 0.2, 1.0)
    leaves = [t.clone().requires_grad_(True) for t in (o, z, wg)]
    got = torch.autograd.grad(A.norm_gate(*leaves, gate="sigmoid"), leaves, dn.view(15, 2, 64))
    ref = B.norm_gate_bwd(o, z, wg, dn.view(15, 2, 64), gate="sigmoid")
    for a, name in zip(got, ("o", "z", "w")):
        assert a.dtype == dt and torch.equal(a, ref[name].to(dt)), name


def test_gradients_of_gradients_are_refused():
    """The backward passes have no gradients of their own: asking for them is an error, never a
    gradient without its second part."""
    import torch
    from gated_delta_rule_prologue_amd import autograd as A
    gen = torch.Generator().manual_seed(9)
    x, y, o = (rand(gen, (6, 2, 64), torch.float32).requires_grad_(True) for _ in range(3))
    w = rand(gen, 64, torch.float32, 0.2, 1.0).requires_grad_(True)
    for out in (A.norm_residual(x, w, y=y)[0], A.norm_gate(o, x, w)):
        g, = torch.autograd.grad(out.square().sum(), [x], create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.square().sum().backward()


def test_binding_refusals_on_device():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf, device="cuda"), torch.zeros(64, dtype=bf, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.norm_residual(torch.zeros(64, 4, dtype=bf, device="cuda").t(), w)
    with pytest.raises(ValueError, match="w: expected"):
        B.norm_gate(x, x, w[:32])
    with pytest.raises(ValueError, match="y: expected"):
        B.norm_residual(x, w, y=x[:3])
    with pytest.raises(TypeError, match="scale: expected"):
        B.norm_residual(x, w, y=x, scale=w.float())
    with pytest.raises(ValueError, match="w is on cpu"):
        B.norm_residual(x, w.cpu())
    with pytest.raises(ValueError, match="workspace needs"):
        B.norm_residual_bwd(x, w, x, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.PrismError):
        wide = torch.zeros(1, 8200, dtype=bf, device="cuda")
        B.norm_residual(wide, wide[0])
    with pytest.raises(B.PrismError):                  # an address that is not a multiple of 16
        flat = torch.zeros(4 * 64 + 1, dtype=bf, device="cuda")
        B.norm_residual(flat[1:].view(4, 64), w)
