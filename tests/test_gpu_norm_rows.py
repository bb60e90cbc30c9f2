"""Norms at more rows than workgroups, where every group of lanes takes several rows in turn and
adds up their column sums: all gradients, each against the magnitude of its own column's terms.

Tolerances as in test_gpu_norms.py: FWD, BWD and SUM roundings of 2^-24 on the magnitude of
the terms that are added up.  The most rows a lane adds here is 20,000 / 512 = 40 (one
group a workgroup: 3000 / 256 = 12): with 32 groups, 512 / 64 partials and 6 more, 86 beyond
a term's own 128, and SUM + 8 covers them."""
import pytest

from tests.layer_refs import EPS32, check, f64
from tests import layer_refs as R
from tests.test_gpu_norms import BWD, EPS, FWD, SUM, dtypes, rand

MANY = SUM + 8
# (rows, width) of 8, 16, 64 lanes a row, then of whole workgroups of 128, 256 and 512, with rows beyond
# the forward's workgroups too (4096, 2048, 1024 of them)
SHAPES = [(20000, 64), (20000, 61), (5000, 250), (4300, 1032), (4300, 1028), (3000, 2056), (3000, 4100), (1500, 8191)]


@pytest.fixture
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    return binding


def residual_grads(r, w, dn, dr, y, s):
    """Gradients from the formula in 64 bits, and the magnitudes of what each adds up."""
    import torch
    rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    rh, e = r * rstd, dn * w
    t = rstd * (e - rh * (e * rh).mean(-1, keepdim=True)) + dr
    mag = rstd * (e.abs() + rh.abs() * (e * rh).abs().mean(-1, keepdim=True)) + dr.abs()
    return {"x": (t, mag), "y": (s * t, s.abs() * mag), "w": ((dn * rh).sum(0), (dn * rh).abs().sum(0)),
            "scale": ((t * y).sum(0), (mag * y.abs()).sum(0))}


def gate_grads(o, z, w, dy, gate):
    import torch
    rstd = 1 / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS)
    s, c = torch.sigmoid(z), torch.sigmoid(-z)
    act, slope, smag = (z * s, s * (1 + z * c), s * (1 + z.abs() * c)) if gate == "silu" else (s, s * c, s * c)
    oh, e = o * rstd, dy * act * w
    do = rstd * (e - oh * (e * oh).mean(-1, keepdim=True))
    mag = rstd * (e.abs() + oh.abs() * (e * oh).abs().mean(-1, keepdim=True))
    over = 0 if w.dim() == 2 else (0, 1)
    return {"o": (do, mag), "z": (dy * oh * w * slope, (dy * oh * w).abs() * smag),
            "w": ((dy * act * oh).sum(over), (dy * act * oh).abs().sum(over))}


def against(what, got, ref):
    return max(check(f"{what} d{k}", got[k], *ref[k], MANY if k in ("w", "scale") else BWD) for k in ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_residual_norm(gpu, rows, width, dtype):
    import torch
    from tests.gpu_common import say
    dt, gen = dtypes()[dtype], torch.Generator().manual_seed(rows + width)
    x, y, dn, dr = (rand(gen, (rows, width), dt) for _ in range(4))
    w, s = rand(gen, width, dt, 0.2, 1.0), rand(gen, width, dt, 0.3, 0.5)
    n, r = gpu.norm_residual(x, w, y=y, scale=s, eps=EPS)
    nr, rr, nmag, rmag = R.norm_residual(f64(x), f64(w), f64(y), f64(s), EPS)
    check("n", n, nr, nmag, FWD)
    check("r", r, rr, rmag, 3)
    del nr, rr, nmag, rmag
    g = gpu.norm_residual_bwd(r, w, dn, dr=dr, y=y, scale=s, eps=EPS)
    worst = against(f"{rows} x {width}", g, residual_grads(*(f64(t) for t in (r, w, dn, dr, y, s))))
    say(f"{rows} x {width} {dtype}: worst share of the tolerance {worst:.2f}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("tokens,heads,width,gate", [(10000, 2, 64, "silu"), (9000, 3, 61, "sigmoid"), (700, 5, 250, "silu"),
                                                     (3000, 1, 1001, "sigmoid"), (700, 600, 8, "silu")])
def test_gated_norm(gpu, tokens, heads, width, gate, per_head, dtype):
    import torch
    from tests.gpu_common import say
    dt, gen = dtypes()[dtype], torch.Generator().manual_seed(tokens + width)
    o, z, dy = (rand(gen, (tokens, heads, width), dt) for _ in range(3))
    w = rand(gen, (heads, width) if per_head else (width,), dt, 0.2, 1.0)
    y = gpu.norm_gate(o, z, w, eps=EPS, gate=gate)
    want = R.norm_gate(f64(o), f64(z), f64(w), EPS, gate)
    check("y", y, want, want.abs(), FWD)
    g = gpu.norm_gate_bwd(o, z, w, dy, eps=EPS, gate=gate)
    worst = against(f"{tokens} x {heads} x {width}", g, gate_grads(*(f64(t) for t in (o, z, w, dy)), gate))
    say(f"{tokens} x {heads} x {width} {dtype} {gate}: worst share of the tolerance {worst:.2f}")


def test_the_tolerance_finds_lost_rows():
    """The bound on a weight's gradient is far below what one group of rows adds to it: a sum
    without the rows of a single workgroup (1 of 512) is outside it, in most columns."""
    import torch
    gen = torch.Generator().manual_seed(1)
    o, z, dy = (torch.randn(10000, 2, 64, generator=gen, dtype=torch.float64) for _ in range(3))
    w = torch.ones(2, 64, dtype=torch.float64)
    whole = gate_grads(o, z, w, dy, "silu")["w"]
    keep = torch.arange(10000) % 256 != 17
    lost = gate_grads(o[keep], z[keep], w, dy[keep], "silu")["w"][0]
    outside = (lost - whole[0]).abs() > EPS32 * (whole[0].abs() + MANY * whole[1])
    assert outside.double().mean() > 0.9
