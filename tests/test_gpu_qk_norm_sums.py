"""Weights' gradients of the norm of queries and keys over very many rows, past 2^31 elements among them, where every
term of a sum has one sign and one value: the roundings of such a sum have one sign too, and add up.

A lane adds up to 256 rows in turn, then these stretches (at most 40 here), then come the groups of a workgroup (at most
64), a 64th of the workgroups (at most 16) and 6 more, each rounding by 2^-24 of the sum at most: 382, whatever
the number of rows.  With a norm the terms hold its own roundings, 40."""
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu
ADDS = 256 + 40 + 64 + 16 + 6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


@pytest.mark.parametrize("dtype,T,hq,hk,d", [("bf16", 2_100_000, 8, 1, 128), ("f32", 800_000, 5, 1, 75),
                                             ("f32", 600_000, 4, 4, 256), ("bf16", 9000, 700, 257, 64),
                                             ("bf16", 8_000_000, 1, 0, 8), ("f32", 500_000, 6, 2, 500)])
@pytest.mark.parametrize("norm", ["none", "rms"])
def test_equal_terms(dtype, T, hq, hk, d, norm):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(T)
    rand = lambda: (1 + torch.rand(d, generator=gen)).to(dt).cuda()
    x, up, w = rand(), rand(), rand()
    same = lambda v, h: v.expand(T, h, d)                    # one row for all tokens and heads
    dq, dk = same(up, hq).contiguous(), same(up, hk).contiguous() if hk else None
    how = dict(wq=w, wk=w if hk else None, norm=norm)
    g = B.qk_norm_bwd(same(x, hq), dq, same(x, hk) if hk else None, dk, **how)
    x6, up6 = x.double().cpu(), up.double().cpu()
    if norm == "rms":
        x6 = x6 / torch.sqrt((x6 * x6).mean() + 1e-6)
    worst = 0.0
    for n, h in (("wq", hq), ("wk", hk)):
        if h:
            ref = T * h * x6 * up6
            allow = (ADDS + (40 if norm == "rms" else 0)) * 2.0 ** -24
            worst = max(worst, ((g[n].double().cpu() - ref).abs() / (allow * ref)).max().item())
    say(f"qk_norm sums of {T} x ({hq} + {hk}) x {d} {dtype} {norm}: worst share of the tolerance {worst:.2f}")
    assert worst <= 1
    again = B.qk_norm_bwd(same(x, hq), dq, same(x, hk) if hk else None, dk, **how)
    assert torch.equal(g["wq"], again["wq"]) and (not hk or torch.equal(g["wk"], again["wk"]))
