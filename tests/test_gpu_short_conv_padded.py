"""Batches with rows behind the last sequence (prism_short_conv_ex): what the next layer reads there, and the gradients
of a stack on such a batch.

The weights' gradients of the padded and of the plain batch are the same terms, added in two orders: each
is off by at most 300 roundings of 2^-24 of their magnitudes (the count of the norm's and the convolution's own tests)."""
import ctypes

import pytest

from tests import stack_refs as R
from tests.layer_refs import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def poison(*shapes, dtype):
    """Leaves NaN in the memory that tensors of these shapes are given next."""
    import torch
    held = [torch.full(s, float("nan"), dtype=dtype, device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,K", [(1, 4), (5, 3), (64, 1), (77, 4), (2304, 4), (130, 8)])
def test_rows_behind_are_zero_or_left(dtype, C, K):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(C)
    for lens, behind in (([5, 60, 0], 70), ([64, 32], 3), ([0, 0], 40), ([1], 1000), ([17, 4], 0)):
        live = sum(lens)
        T = live + behind
        rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
        x, w = rand(T, C), rand(C, K)
        x[live:] = float("nan")
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
        want, _ = B.short_conv(x[:live].contiguous(), w, cu)
        poison((T, C), dtype=dt)
        y, _ = B.short_conv(x, w, cu)
        assert torch.equal(y[:live], want) and (y[live:] == 0).all()
        kept = torch.full((T, C), 3.0, dtype=dt, device="cuda")
        B.short_conv(x, w, cu, y=kept)
        assert torch.equal(kept[:live], want) and (kept[live:] == 3.0).all()
        dims = B.ConvDims(len(lens), T, C, K, B._dtype_code(x), C)
        p = lambda t: ctypes.c_void_p(t.data_ptr())
        for clear, left in ((0, 3.0), (1, 0.0)):
            out = torch.full((T, C), 3.0, dtype=dt, device="cuda")
            assert B.lib().prism_short_conv_ex(ctypes.byref(dims), p(x), p(w), None, None, p(cu), 1, clear, p(out), None,
                                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == B.PRISM_OK
            assert torch.equal(out[:live], want) and (out[live:] == left).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_a_padded_batch(dtype):
    """Convolution, then norms with weights over every row: nothing of the spare rows' memory reaches a gradient."""
    import torch
    from gated_delta_rule_prologue_amd import autograd as A
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(7)
    H, D, K, lens, behind = 2, 64, 4, [9, 30, 0, 21], 37
    live = sum(lens)
    cu = torch.tensor([0, 9, 39, 39, 60], dtype=torch.int32).cuda()
    rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
    x, w, wq, wk = rand(live + behind, 2 * H * D), rand(2 * H * D, K), rand(D), rand(D)
    up = rand(live, 2 * H, D)

    def run(T):
        v = {"x": x[:T].clone(), "w": w.clone(), "wq": wq.clone(), "wk": wk.clone()}
        v = {n: t.requires_grad_(True) for n, t in v.items()}
        poison((T, 2 * H * D), (T, H, D), dtype=dt)
        y = A.short_conv(v["x"], v["w"], cu)
        q, k = A.qk_norm(y[:, :H * D].view(T, H, D), y[:, H * D:].view(T, H, D), v["wq"], v["wk"], norm="rms")
        (torch.cat([q, k], 1)[:live].float() * up.float()).sum().backward()
        return {n: t.grad for n, t in v.items()}, y.detach()

    plain, y = run(live)
    padded, _ = run(live + behind)
    assert all(torch.isfinite(g).all() for g in padded.values())
    assert torch.equal(padded["x"][:live], plain["x"]) and (padded["x"][live:] == 0).all()
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dt]
    xh = f64(y).view(live, 2 * H, D)
    xh = (xh * R.rstd_of(xh, "rms", 1e-6)).abs()
    terms = (f64(up).abs() * xh)
    for n, mag in (("wq", terms[:, :H].sum((0, 1))), ("wk", terms[:, H:].sum((0, 1)))):
        bound = 2 * 300 * 2.0 ** -24 * mag + 2 * half * f64(plain[n]).abs() * (1 + half)
        assert ((f64(padded[n]) - f64(plain[n])).abs() <= bound).all(), n
    assert torch.equal(padded["w"], plain["w"])              # its runs of tokens are the same
