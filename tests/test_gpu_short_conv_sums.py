"""Weights' gradients of the short convolution over very many rows, where every term of a sum has one sign and one value:
the roundings of such a sum have one sign too, and add up.

A lane adds 256 rows in turn, then these stretches of its run (at most 40 here), then come the lanes of a
workgroup (at most 32), a 64th of the workgroups (at most 2) and 6 more, each rounding by 2^-24 of the sum at
most: 336, whatever the number of rows.  The terms themselves are the products of a fused addition, exact."""
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu
ADDS = 256 + 40 + 32 + 2 + 6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


@pytest.mark.parametrize("dtype,T,C,K", [("bf16", 1 << 20, 2304, 4), ("f32", 1 << 19, 2304, 4), ("bf16", 600_001, 768, 8),
                                         ("f32", 300_003, 770, 1), ("bf16", 200_000, 1536, 2), ("bf16", 90_000, 1536, 4),
                                         ("bf16", 5_000_000, 3, 4)])
def test_equal_terms(dtype, T, C, K):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(T)
    a, b = ((1 + torch.rand(C, generator=gen)).to(dt).cuda() for _ in range(2))
    x = a.expand(T, C)                                       # one row for all tokens
    dy = b.expand(T, C).contiguous()
    w, bias = torch.zeros(C, K, dtype=dt, device="cuda"), torch.zeros(C, dtype=dt, device="cuda")
    cut = T // 3
    cu = torch.tensor([0, cut, cut, T - 5, T], dtype=torch.int32).cuda()
    lens = [cut, 0, T - 5 - cut, 5]
    g = B.short_conv_bwd(x, w, cu, dy, bias=bias, activation=None)
    # tap m takes the rows that have one K - 1 - m before them in their sequence
    count = torch.tensor([sum(max(0, n - (K - 1 - m)) for n in lens) for m in range(K)]).double()
    dw, db = (a.double() * b.double()).cpu()[:, None] * count, T * b.double().cpu()
    worst = 0.0
    for got, ref in ((g["w"], dw), (g["bias"], db)):
        share = ((got.double().cpu() - ref).abs() / (ADDS * 2.0 ** -24 * ref)).max().item()
        worst = max(worst, share)
    say(f"short_conv sums of {T} rows of {C} {dtype}: worst share of the tolerance {worst:.2f}")
    assert worst <= 1
    again = B.short_conv_bwd(x, w, cu, dy, bias=bias, activation=None)
    assert torch.equal(g["w"], again["w"]) and torch.equal(g["bias"], again["bias"])
