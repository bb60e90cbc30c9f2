"""The norm and rotation of queries and keys (prism_qk_norm and its gradients) against the formula in
64 bits, and the gradients against differences.

Tolerances.  An output is rounded once to its type.  Before it, in roundings of 2^-24 on the magnitude of the
terms: a row's sum of squares adds at most 16 terms a lane and 6 across lanes, halved by the
root; root and reciprocal, two products; the rotation two products and an addition, on the sum of
both elements of the pair, with cosines and sines within 4: 40 covers a forward output.  A gradient
holds a second such sum, on the sum of its absolute terms: 128.  A weight's gradient adds the rows of a
lane (at most 64 here), up to 64 groups, a 64th of the workgroups and 6 more: 300 with the 128."""
import pytest

from tests import stack_refs as R
from tests.gpu_common import say
from tests.layer_refs import check, f64

pytestmark = pytest.mark.gpu
FWD, BWD, SUM = 40, 128, 300
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def make(T, hq, hk, d, rot, dtype="bf16", weight=True, fused=False, seed=0, far=1 << 20):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen).to(dt).cuda()
    if fused:                                                # heads beside each other, q, k and v of each in turn
        rows = rand(T, hq + 2 * hk, d + 3)
        q, k = rows[:, :hq, 3:], rows[:, hq:hq + hk, 1:d + 1]
    else:
        q, k = rand(T, hq, d), rand(T, hk, d)
    w = lambda: (1 + 0.3 * torch.randn(d, generator=gen)).to(dt).cuda() if weight else None
    out = {"q": q, "k": k if hk else None, "wq": w(), "wk": w() if hk else None, "dq": rand(T, hq, d),
           "dk": rand(T, hk, d) if hk else None, "positions": None, "freqs": None}
    if rot:
        out["positions"] = torch.randint(-far, far, (T,), generator=gen).int().cuda()
        out["freqs"] = (10000.0 ** (-torch.arange(rot // 2).double() / max(1, rot // 2))).float().cuda()
    return out


def check_all(d, norm, layout, scale=1.0, eps=EPS):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    how = dict(wq=d["wq"], wk=d["wk"], norm=norm, eps=eps, positions=d["positions"], freqs=d["freqs"], layout=layout,
               rot_scale=scale)
    rot = 0 if d["freqs"] is None else 2 * d["freqs"].numel()
    out = dict(zip("qk", B.qk_norm(d["q"], d["k"], **how)))
    g = B.qk_norm_bwd(d["q"], d["dq"], d["k"], d["dk"], **how)
    worst = 0.0
    pos, fr = (None, None) if not rot else (d["positions"].cpu(), d["freqs"].cpu())
    for n in "qk":
        if d[n] is None:
            assert out[n] is None and g[n] is None and g["w" + n] is None
            continue
        x, w, dy = f64(d[n]), f64(d["w" + n]), f64(d["d" + n])
        leaves = [t.requires_grad_(True) for t in (x, w) if t is not None]
        ref = R.qk_norm(x, w, norm, eps, pos, fr, layout, scale)
        grads = torch.autograd.grad((ref * dy).sum(), leaves)
        for t in leaves:
            t.requires_grad_(False)
        rstd = R.rstd_of(x, norm, eps)
        xh = x * rstd
        mag = R.partner_sum(xh if w is None else xh * w, rot, layout, scale)
        worst = max(worst, check(n, out[n], ref.detach(), mag, FWD))
        e = R.partner_sum(dy, rot, layout, scale)
        ew = e if w is None else e * w.abs()
        c = {"none": 0, "rms": 1 / x.shape[-1], "l2": 1}[norm]
        mag = rstd * (ew + xh.abs() * c * (ew * xh.abs()).sum(-1, keepdim=True))
        worst = max(worst, check("d" + n, g[n], grads[0], mag, BWD))
        if w is not None:
            worst = max(worst, check("dw" + n, g["w" + n], grads[1], (e * xh.abs()).sum((0, 1)), SUM))
        else:
            assert g["w" + n] is None
    return worst


# widths and rotated parts: whole vectors, single elements, parts that end inside a vector
SHAPES = [(1, 0), (2, 2), (3, 2), (8, 0), (8, 8), (16, 16), (24, 16), (32, 16), (64, 64), (64, 32), (72, 64), (75, 30),
          (80, 80), (80, 40), (96, 6), (128, 128), (128, 64), (128, 2), (130, 130), (136, 128), (192, 192), (200, 48),
          (256, 256), (257, 256), (384, 128), (511, 510), (512, 512), (512, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
def test_widths(dtype, layout, norm):
    worst = 0.0
    for i, (d, rot) in enumerate(SHAPES):
        T, hq, hk = (7, 3, 1) if i % 2 else (3, 2, 5)
        worst = max(worst, check_all(make(T, hq, hk, d, rot, dtype, weight=i % 3 != 0, seed=d + rot), norm, layout,
                                     scale=1.0 if i % 4 else 1.25))
    say(f"qk_norm {dtype} {layout} {norm}: worst share of the tolerance {worst:.2f}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_heads(dtype):
    """Slices of a fused projection at any element's address, shared keys, no keys, one token."""
    worst = 0.0
    for T in (1, 2, 19):
        for hq, hk in ((1, 1), (8, 2), (6, 6), (3, 0), (17, 1)):
            for d, rot in ((64, 64), (50, 20), (128, 32)):
                worst = max(worst, check_all(make(T, hq, hk, d, rot, dtype, fused=True, seed=T + hq), "l2", "half"))
    say(f"qk_norm strides {dtype}: worst share of the tolerance {worst:.2f}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2047, 2051, 8195, 20011])
def test_many_tokens(dtype, T):
    """Each number of tokens a workgroup takes at once, the last of them cut short; the weights' sums."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    d = make(T, 2, 1, 64, 64, dtype, seed=T)
    check_all(d, "rms", "half")
    how = dict(wq=d["wq"], wk=d["wk"], norm="rms", positions=d["positions"], freqs=d["freqs"])
    a, b = (B.qk_norm_bwd(d["q"], d["dq"], d["k"], d["dk"], **how) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_far_positions():
    """The largest positions an int32 holds, with the fastest frequency."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    pos = [0, 1, -1, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 30 + 1, 2 ** 31 - 1, -2 ** 31]
    d = make(len(pos), 1, 1, 64, 64, "f32")
    d["positions"] = torch.tensor(pos, dtype=torch.int32).cuda()
    d["freqs"] = d["freqs"] * 1.0009765625
    for layout in ("half", "interleaved"):
        check_all(d, "none", layout)


def test_rows_of_zeros_and_extremes():
    """Rows of zeros give zeros; a row that is not finite stays in its own row."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    d = make(6, 2, 2, 64, 64, "f32", weight=False)
    clean, ck = B.qk_norm(d["q"], d["k"], positions=d["positions"], freqs=d["freqs"])
    q = d["q"].clone()
    q[1, 0] = 0
    q[2, 1, 5] = float("nan")
    q[3, 0, 7] = float("inf")
    out, k = B.qk_norm(q, d["k"], positions=d["positions"], freqs=d["freqs"])
    assert (out[1, 0] == 0).all() and torch.isnan(out[2, 1]).any() and torch.equal(k, ck)
    same = torch.ones(6, 2, dtype=torch.bool)
    same[1, 0] = same[2, 1] = same[3, 0] = False
    assert torch.equal(out[same], clean[same])
    g = B.qk_norm_bwd(q, d["dq"], d["k"], d["dk"], positions=d["positions"], freqs=d["freqs"])
    assert torch.isfinite(g["q"][same]).all() and torch.isfinite(g["k"]).all()
    tiny = d["q"] * 1e-22                                    # squares below the smallest normal: eps holds
    out, _ = B.qk_norm(tiny, positions=d["positions"], freqs=d["freqs"])
    ref = R.qk_norm(f64(tiny), None, "l2", EPS, d["positions"].cpu(), d["freqs"].cpu())
    assert (f64(out) - ref).abs().max() <= 64 * 2.0 ** -24 * ref.abs().max()


@pytest.mark.parametrize("d,rot", [(128, 128), (75, 30)])
def test_in_place(d, rot):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    m = make(33, 4, 2, d, rot)
    how = dict(wq=m["wq"], wk=m["wk"], norm="rms", positions=m["positions"], freqs=m["freqs"])
    q, k = B.qk_norm(m["q"], m["k"], **how)
    q2, k2 = m["q"].clone(), m["k"].clone()
    a, b = B.qk_norm(q2, k2, q_out=q2, k_out=k2, **how)
    assert a is q2 and b is k2 and torch.equal(q, q2) and torch.equal(k, k2)


def test_gradients_against_differences():
    import torch
    from gated_delta_rule_prologue_amd.autograd import qk_norm
    for norm, layout, d, rot in (("l2", "half", 10, 8), ("rms", "interleaved", 16, 16), ("none", "half", 8, 4)):
        m = make(4, 2, 1, d, rot, "f32", seed=d, far=50)
        leaves = {n: m[n].clone().requires_grad_(True) for n in ("q", "k", "wq", "wk")}

        def loss(v):
            q, k = qk_norm(v["q"], v["k"], v["wq"], v["wk"], norm=norm, positions=m["positions"], freqs=m["freqs"],
                           layout=layout)
            return (q.double() * m["dq"].double()).sum() + (k.double() * m["dk"].double()).sum()

        grads = torch.autograd.grad(loss(leaves), list(leaves.values()))
        h = 2.0 ** -8                                        # error h^2 of the third derivative, 2^-24 / h of the values
        for name, g in zip(leaves, grads):
            flat = leaves[name].detach().reshape(-1)
            for i in range(0, flat.numel(), max(1, flat.numel() // 9)):
                vals = []
                for sign in (1, -1):
                    v = {n: t.detach() for n, t in leaves.items()}
                    moved = flat.clone()
                    moved[i] += sign * h
                    v[name] = moved.view_as(leaves[name])
                    vals.append(loss(v).item())
                diff = (vals[0] - vals[1]) / (2 * h)
                assert abs(diff - g.reshape(-1)[i].item()) <= 2e-2 * (1 + abs(diff)), (norm, name, i)


def test_autograd_of_projection_slices():
    """q and k as slices of one leaf, weights that are shared, one output unused, gradients of
    gradients refused, frequencies that ask for a gradient refused."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    from gated_delta_rule_prologue_amd.autograd import qk_norm
    m = make(9, 2, 2, 64, 64)
    p = torch.randn(9, 6 * 64, device="cuda").to(torch.bfloat16).requires_grad_(True)
    w = m["wq"].clone().requires_grad_(True)
    cut = lambda t: (t[:, :128].view(9, 2, 64), t[:, 128:256].view(9, 2, 64))
    q, k = qk_norm(*cut(p), w, w, norm="rms", positions=m["positions"], freqs=m["freqs"])
    (q * m["dq"]).sum().backward()                           # k is not used: its gradient is zero
    g = B.qk_norm_bwd(cut(p.detach())[0], m["dq"], cut(p.detach())[1], torch.zeros_like(m["dk"]), m["wq"], m["wq"],
                      norm="rms", positions=m["positions"], freqs=m["freqs"])
    assert torch.equal(p.grad[:, :128].reshape(9, 2, 64), g["q"]) and (p.grad[:, 128:] == 0).all()
    assert torch.equal(w.grad, g["wq"].to(torch.bfloat16))
    only, none = qk_norm(cut(p)[0], norm="l2")
    assert none is None and only.shape == (9, 2, 64)
    with pytest.raises(ValueError, match="freqs"):
        qk_norm(*cut(p), positions=m["positions"], freqs=m["freqs"].clone().requires_grad_(True))
    with pytest.raises(RuntimeError):
        gx, = torch.autograd.grad(qk_norm(cut(p)[0])[0].float().sum(), p, create_graph=True)
        gx.float().sum().backward()


def test_no_tokens():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    d = make(0, 2, 1, 64, 64)
    how = dict(wq=d["wq"], wk=d["wk"], norm="rms", positions=d["positions"], freqs=d["freqs"])
    q, k = B.qk_norm(d["q"], d["k"], **how)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    g = B.qk_norm_bwd(d["q"], d["dq"], d["k"], d["dk"], **how)
    assert (g["wq"] == 0).all() and (g["wk"] == 0).all()


def test_one_query_head_beside_thousands_of_keys():
    assert check_all(make(2050, 1, 4099, 8, 8, seed=13), "rms", "half") <= 1


def test_offsets_past_32_bits():
    """More than 2^31 elements of q, and rows that lie as far apart: the last tokens' values are those that they have
    alone."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    T, H, d, last = 2_100_000, 8, 128, 37
    assert T * H * d > 2 ** 31
    gen = torch.Generator().manual_seed(14)
    rows = torch.zeros(T, H + 1, d, dtype=torch.bfloat16, device="cuda")
    rows[-last:] = torch.randn(last, H + 1, d, generator=gen).to(rows)
    dq, dk = torch.zeros(T, H, d).to(rows), torch.zeros(T, 1, d).to(rows)
    dq[-last:], dk[-last:] = torch.randn(last, H, d, generator=gen).to(rows), torch.randn(last, 1, d, generator=gen).to(rows)
    how = dict(norm="rms", freqs=B.rotary_freqs(64))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    tail = slice(T - last, T)
    own = pos[tail].clone()                                  # int32 arrays begin at 16 bytes
    q, k = B.qk_norm(rows[:, :H], rows[:, H:], positions=pos, **how)
    q1, k1 = B.qk_norm(rows[tail, :H], rows[tail, H:], positions=own, **how)
    assert torch.equal(q[tail], q1) and torch.equal(k[tail], k1)
    del q, k
    g = B.qk_norm_bwd(rows[:, :H], dq, rows[:, H:], dk, positions=pos, **how)
    g1 = B.qk_norm_bwd(rows[tail, :H], dq[tail], rows[tail, H:], dk[tail], positions=own, **how)
    assert torch.equal(g["q"][tail], g1["q"]) and torch.equal(g["k"][tail], g1["k"])
