"""The Python calls at the limits of the short convolution, the norm and rotation of queries and keys, and the
choice of a token: what exceeds them is named as unsupported, with nothing allocated for it."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def test_beyond_the_limits():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    x, w, cu = new(2, (1 << 22) + 1), new((1 << 22) + 1, 2), torch.tensor([0, 2], dtype=torch.int32).cuda()
    q, v = new(4, 1, 513), new(513)
    logits, u = new(3, (1 << 20) + 1), torch.zeros(3, device="cuda")
    calls = [lambda: B.short_conv(x, w, cu), lambda: B.short_conv_bwd(x, w, cu, x), lambda: B.qk_norm(q),
             lambda: B.qk_norm_bwd(q, q, wq=v), lambda: B.sample(logits, u), lambda: B.sample(logits[:, :-1], u)]
    y, dw = 2 * x.numel() + 4096, 4 * w.numel() + 4096       # the outputs' bytes
    for i, (call, most) in enumerate(zip(calls, (y, y + dw, 1 << 16, 1 << 16, 1 << 16))):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with pytest.raises(B.PrismError) as e:
            call()
        assert e.value.status == B.PRISM_EUNSUPPORTED, i
        assert torch.cuda.max_memory_allocated() - before <= most, i         # and no workspace
    tokens, _ = calls[-1]()
    assert (tokens == 0).all()
