"""Sequences trained piece by piece: the history is moved on in place between a piece's forward and its backward."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 4, 7])
def test_history_moved_before_the_backward(dtype, K):
    """Every gradient is that of the history as the forward saw it."""
    import torch
    from gated_delta_rule_prologue_amd import autograd as A
    from gated_delta_rule_prologue_amd import binding as B
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(K)
    rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
    C, lens = 48, [3, 40, 1]
    T = sum(lens)
    cu = torch.tensor([0, 3, 43, 44], dtype=torch.int32).cuda()
    w, bias, hist = rand(C, K), rand(C), rand(3, K - 1, C)
    for piece in range(3):
        x, dy = rand(T, C), rand(T, C)
        want = B.short_conv_bwd(x, w, cu, dy, bias=bias, hist=hist)
        v = {n: t.clone().requires_grad_(True) for n, t in (("x", x), ("w", w), ("bias", bias))}
        y = A.short_conv(v["x"], v["w"], cu, v["bias"], "silu", hist)
        again, _ = B.short_conv(x, w, cu, bias=bias, hist=hist, hist_out=hist)
        assert torch.equal(y, again)
        y.backward(dy)
        assert all(torch.equal(v[n].grad, want[n].to(dt)) for n in v), piece


def test_gradient_of_a_history_that_is_moved():
    import torch
    from gated_delta_rule_prologue_amd import autograd as A
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen).cuda()
    x, w, hist, dy = rand(30, 16), rand(16, 4), rand(2, 3, 16), rand(30, 16)
    cu = torch.tensor([0, 2, 30], dtype=torch.int32).cuda()
    want = B.short_conv_bwd(x, w, cu, dy, hist=hist)
    h = hist.clone().requires_grad_(True)
    y = A.short_conv(x, w, cu, hist=h)
    with torch.no_grad():
        h.zero_()                                            # torch's own in-place work too
    y.backward(dy)
    assert torch.equal(h.grad, want["hist"])
