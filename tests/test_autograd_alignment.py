"""Upstream gradients that are contiguous but begin at any element's address, as the backward
of a concatenation along rows hands them out."""
import pytest

torch = pytest.importorskip("torch")


def test_upstream_gradients_are_aligned():
    """What the backward passes hand to the kernels starts at a multiple of 16 bytes."""
    from gated_delta_rule_prologue_amd import autograd as A
    like = torch.zeros(4, 769, dtype=torch.bfloat16)
    base = torch.randn(7, 769, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    cut = base[3:]
    assert cut.is_contiguous() and cut.data_ptr() % 16
    got = A._upstream(cut, like)
    assert got.data_ptr() % 16 == 0 and torch.equal(got, cut)
    fine = base[:4]
    assert A._upstream(fine, like).data_ptr() == fine.data_ptr()       # nothing is copied without need
    assert A._upstream(None, like) is None
    empty = base[3:3]
    assert A._upstream(empty, like).shape == (0, 769)
    assert A._upstream(cut.float().t(), like.float()).is_contiguous()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,width", [("bf16", 769), ("bf16", 61), ("f32", 1001), ("f32", 3)])
def test_norms_behind_a_concatenation(dtype, width):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import autograd as A, binding as B
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(width)

    def r(*shape):
        return torch.randn(shape, generator=gen).to(dt).cuda()

    first, x, y, z = r(3, width), r(5, width), r(5, width), r(5, width)
    w = r(width)
    up = [r(8, width) for _ in range(3)]
    leaves = [t.clone().requires_grad_(True) for t in (x, w, y, z)]
    n, res = A.norm_residual(leaves[0], leaves[1], y=leaves[2])
    out = A.norm_gate(y, leaves[3], w)
    cats = [torch.cat([first, t], 0) for t in (n, res, out)]
    got = torch.autograd.grad(cats, leaves, up)
    cut = [u[3:].clone() for u in up]
    ref = B.norm_residual_bwd(res.detach(), w, cut[0], dr=cut[1])
    gate = B.norm_gate_bwd(y, z, w, cut[2])
    for a, b in zip(got, (ref["x"], ref["w"].to(dt), ref["x"], gate["z"])):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_operator_behind_a_concatenation(dtype):
    """The operator's own backward, for o and the final state behind an odd number of elements."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd.autograd import prism
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(5)

    def r(*shape):
        return torch.randn(shape, generator=gen)

    T, H, L = 20, 2, 2
    unit = torch.nn.functional.normalize
    ins = [unit(r(T, H, 64), dim=-1), unit(r(T, H, 64), dim=-1), r(T, H, 64), unit(r(T, H, 1, 64), dim=-1),
           torch.sigmoid(r(T, H) + 3), torch.sigmoid(r(T, H)), 0.5 * torch.sigmoid(r(T, H, 1, 64)),
           torch.sigmoid(r(T, H, 1, 64)), 0.5 * r(H, 64, 4)]
    ins = [t.to(dt).cuda() for t in ins]
    v = ins[2].clone().requires_grad_(True)
    cu = torch.tensor([0, 13, T], dtype=torch.int32).cuda()
    o, S = prism(ins[0], ins[1], v, *ins[3:], cu, L)
    up_o, up_s = r(3 + o.numel()).to(dt).cuda(), r(1 + S.numel()).cuda()
    ends = [torch.cat([torch.zeros(n, dtype=t.dtype, device="cuda"), t.reshape(-1)]) for n, t in ((3, o), (1, S))]
    got, = torch.autograd.grad(ends, [v], [up_o, up_s])
    o, S = prism(ins[0], ins[1], v, *ins[3:], cu, L)
    ref, = torch.autograd.grad([o, S], [v], [up_o[3:].clone().view_as(o), up_s[1:].clone().view_as(S)])
    assert torch.equal(got, ref)
