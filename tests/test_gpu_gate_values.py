"""The gate's activation and its slope over the whole range of z, relative to their values.

With o of +-1, w = 1, eps = 0 and the weight's and upstream's factors 1, a row's mean of
squares is exactly 1, so y = +-act(z) and dz = +-act'(z) but for the reciprocal root's own
step, and every error is the activation's.  Half steps of fp32 (2^-24), counted: e^-|z| 2
(a step of exp2) + 1 (its reduced argument, at most 1/2, rounded once), 1 + e 1, its
reciprocal 2, the root 2, and 1 for each product (at most 5 in y, 6 in dz): 14, and 16 covers
them.  In bf16 the exponent |z| log2 e is one rounded product: off by |z| log2 e 2^-24, times ln 2
in e^-|z|, |z| half steps more.  Values below the smallest normal number may be off by that number
times |z|."""
import pytest

from tests.gpu_common import say
from tests.layer_refs import EPS32, HALF_STEP, f64

pytestmark = pytest.mark.gpu
STEPS = 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def gates(dt, lo=-100.0, hi=100.0):
    """[rows, 64] of z from lo to hi, with the same signs of o in every row."""
    import torch
    z = torch.linspace(lo, hi, 64 * 512, dtype=torch.float64)
    z = torch.cat([z, torch.linspace(-2, 2, 64 * 64, dtype=torch.float64)]).view(-1, 64).to(dt)
    o = torch.where(torch.arange(64) % 3 == 0, -1.0, 1.0).to(dt).expand_as(z).contiguous()
    return o.cuda(), z.cuda(), torch.ones(64, dtype=dt, device="cuda")


def within(name, got, want, mag, z):
    g = f64(got)
    assert g.isfinite().all(), name
    half = got.element_size() == 2
    tol = (HALF_STEP[got.dtype] if half else 0) * want.abs() + (STEPS + (z.abs() if half else 0)) * EPS32 * mag
    share = ((g - want).abs() / (tol + 2.0 ** -126 * (1 + z.abs())))
    worst = int(share.argmax())
    say(f"{name}: worst share {float(share.max()):.2f} at z = {float(z.flatten()[worst]):.4f}")
    assert share.max() <= 1, (name, float(share.max()), float(z.flatten()[worst]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_activation(gate, dtype):
    """The error of act(z) does not grow with |z|."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    o, z, w = gates({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    y = B.norm_gate(o, z, w, eps=0.0, gate=gate)
    z6 = f64(z)
    want = f64(o) * torch.sigmoid(z6) * (z6 if gate == "silu" else 1)
    within(f"{gate} {dtype}", y, want, want.abs(), z6)


def test_activation_of_infinite_gates():
    """z of +-infinity, NaN and the types' ends, as z / (1 + e^-z) and 1 / (1 + e^-z) have them."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    for dt in (torch.bfloat16, torch.float32):
        o, z, w = gates(dt)
        ends = [float("inf"), -float("inf"), float("nan"), torch.finfo(dt).max, torch.finfo(dt).min, 0.0, -0.0]
        z[0, :7] = torch.tensor(ends, dtype=dt)
        o[:] = 1.0
        y = B.norm_gate(o, z, w, eps=0.0, gate="sigmoid")[0, :7].float().cpu()
        assert y[[0, 1, 3, 4, 5, 6]].tolist() == [1.0, 0.0, 1.0, 0.0, 0.5, 0.5] and torch.isnan(y[2])
        y = B.norm_gate(o, z, w, eps=0.0)[0, :7].float().cpu()
        assert y[0] == float("inf") and torch.isnan(y[1:3]).all()
        assert y[3:].tolist() == [torch.finfo(dt).max, 0.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_slope(gate, dtype):
    """dz of gates that are nearly open or shut: s (1 - s), and s (1 + z (1 - s)), whose magnitude
    is s (1 + |z| (1 - s)) where its terms cancel (near z = -1.28)."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    o, z, w = gates({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    g = B.norm_gate_bwd(o, z, w, torch.ones_like(o), eps=0.0, gate=gate)
    z6, s, c = f64(z), torch.sigmoid(f64(z)), torch.sigmoid(-f64(z))
    want = s * (1 + z6 * c) if gate == "silu" else s * c
    mag = s * (1 + z6.abs() * c) if gate == "silu" else s * c
    within(f"slope of {gate} {dtype}", g["z"], f64(o) * want, mag, z6)
