"""The layer operators together, as a program uses them: a training step of one layer, a
serving step with drafted tokens, captured and replayed, on other streams."""
import numpy as np
import pytest

from tests.gpu_common import say
from tests.layer_refs import f64
from tests import layer_refs as R
from tests.test_gpu_draft import make as make_draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


class Serving:
    """One layer's decoding of drafted tokens: norm, draft, gate, verification, commit."""

    def __init__(self, lens=(5, 1, 3, 0, 4), seed=1, V=700):
        import torch
        self.d, self.cu, self.cu_t, self.S, self.hist = make_draft(list(lens), H=2, dk=64, dv=64, seed=seed)
        T = self.cu[-1]
        gen = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        self.x, self.y = (torch.randn(T, 128, generator=gen).to(bf).cuda() for _ in range(2))
        self.w, self.s = (torch.rand(128, generator=gen).to(bf).cuda() for _ in range(2))
        self.z = torch.randn(T, 2, 64, generator=gen).to(bf).cuda()
        self.wg = torch.rand(2, 64, generator=gen).to(bf).cuda()
        self.head = torch.randn(128, V, generator=gen).cuda()
        self.q = torch.softmax(torch.randn(T, V, generator=gen), -1).cuda()
        self.tokens = torch.randint(0, V, (T,), generator=gen).int().cuda()
        self.ua, self.us = torch.rand(T, generator=gen).cuda(), torch.rand(len(lens), generator=gen).cuda()

    def step(self, S, hist, stream=None):
        import torch
        from gated_delta_rule_prologue_amd import binding as B
        d = self.d
        n, r = B.norm_residual(self.x, self.w, y=self.y, scale=self.s, stream=stream)
        k = n.view(-1, 2, 64)
        o, kw, p = B.decode_draft(d["q"], k, d["v"], d["u"], d["g"], d["b"], d["a"], d["h"], d["conv_w"], self.cu_t, 4,
                                  S, hist, stream=stream)
        out = B.norm_gate(o, self.z, self.wg, stream=stream)
        # the logits' product stands for the rest of the model (fixed order: no library reduction)
        probs = torch.softmax((out.view(-1, 128, 1).float() * self.head).sum(1), -1)
        kept, nxt = B.verify_draft(probs, self.tokens, self.cu_t, self.ua, self.us, q=self.q, stream=stream)
        S_out, h_out = B.decode_commit(k, d["v"], d["g"], d["b"], self.cu_t, kept, kw, p, S, hist,
                                       S_out=torch.empty_like(S), k_hist_out=torch.empty_like(hist), stream=stream)
        return {"n": n, "r": r, "o": o, "out": out, "probs": probs, "kept": kept, "next": nxt, "S": S_out, "hist": h_out}


def same(a, b):
    import torch
    return [k for k in a if not torch.equal(a[k], b[k])]


def test_serving_step_against_reference():
    """Each operator of the step against its 64-bit reference on what it was given."""
    import torch
    m = Serving()
    r = m.step(m.S, m.hist)
    ref_n, ref_r, nm, rm = R.norm_residual(f64(m.x), f64(m.w), f64(m.y), f64(m.s), 1e-6)
    R.check("n", r["n"], ref_n, nm, 64)
    d6 = {k: f64(v) for k, v in m.d.items()}
    d6["k"] = f64(r["n"]).view(-1, 2, 64)
    o, kw, p, states = R.draft(d6, m.cu, 4, f64(m.S), f64(m.hist), "linear")
    # the normalised rows are no unit keys here: the state grows with them, and so does its scale
    scale = o.abs().max()
    assert (f64(r["o"]) - o).abs().max() <= (2.0 ** -8 + 1e-3) * scale
    kept, nxt = R.verify(f64(r["probs"]).numpy(), f64(m.q).numpy(), m.tokens.cpu().numpy(), m.cu,
                         m.ua.cpu().numpy(), m.us.cpu().numpy())
    assert r["kept"].cpu().tolist() == kept and r["next"].cpu().tolist() == nxt
    for n, c in enumerate(kept):
        want = states[m.cu[n] + c - 1] if c else f64(m.S[n])
        assert (f64(r["S"][n]) - want).abs().max() <= 1e-3 * want.abs().max(), n


def test_serving_step_replays_from_graphs():
    """Two captured steps of different batches, replayed in turn with eager work between; every
    replay equals the eager step (their workspaces are their own)."""
    import torch
    ms = [Serving(), Serving(lens=(2, 8, 1), seed=2, V=5000)]
    refs = [m.step(m.S, m.hist) for m in ms]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for m in ms:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.step(m.S, m.hist)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(m.step(m.S, m.hist))
        graphs.append(g)
    for rep in range(4):
        for i in (0, 1):
            for t in outs[i].values():
                t.zero_()
            graphs[i].replay()
            eager = ms[1 - i].step(ms[1 - i].S, ms[1 - i].hist)
            torch.cuda.synchronize()
            assert not same(refs[i], outs[i]), (rep, i, same(refs[i], outs[i]))
            assert not same(refs[1 - i], eager), (rep, i)


def test_two_streams_at_once():
    """Steps of two batches on two streams, by the current stream and by ``stream=``."""
    import torch
    ms = [Serving(), Serving(lens=(6, 3, 16, 1), seed=3)]
    refs = [m.step(m.S, m.hist) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for rep in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(ms[i].step(ms[i].S, ms[i].hist))
    torch.cuda.synchronize()
    for i in (0, 1):
        for r in got[i]:
            assert not same(refs[i], r), (i, same(refs[i], r))


def test_stream_argument():
    """``stream=`` as a torch stream, as a raw handle and as the default stream's 0."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    m = Serving()
    ref = B.norm_residual_bwd(m.x, m.w, m.y, y=m.y, scale=m.s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream()):
        before = torch.cuda.current_stream()
        got = B.norm_residual_bwd(m.x, m.w, m.y, y=m.y, scale=m.s, stream=stream)
        assert torch.cuda.current_stream() == before
        torch.cuda.synchronize()
        assert not same({k: v for k, v in ref.items()}, got)


def layer(leaves, cu, L):
    """One block: norm in front, the operator on the normalised rows, gate behind, residual add."""
    import torch
    from gated_delta_rule_prologue_amd.autograd import norm_gate, norm_residual, prism
    x, y, s, w, q, v, u, g, b, a, h, cw, z, wg, w2 = leaves
    n, r = norm_residual(x, w, y=y, scale=s)
    k = torch.nn.functional.normalize(n.view(n.shape[0], 2, 64).float(), dim=-1).to(n.dtype)
    o, _ = prism(q, k, v, u, g, b, a, h, cw, cu, L)
    out = norm_gate(o, z, wg)
    n2, r2 = norm_residual(r, w2, y=out.view(r.shape))
    return n2, r2


def test_training_step_of_a_layer():
    """Gradients of a whole block, eager twice (same bits but for the operator's db, which is
    summed with atomics) and against differences of the block itself in fp32."""
    import torch
    gen = torch.Generator().manual_seed(2)
    T, L, f32 = 40, 3, torch.float32

    def r(*shape, mul=1.0, add=0.0):
        return (mul * torch.randn(shape, generator=gen) + add).cuda()

    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)
    base = [r(T, 128), r(T, 128), r(128, mul=0.2, add=0.5), r(128, mul=0.2, add=1.0), unit(r(T, 2, 64)), r(T, 2, 64),
            unit(r(T, 2, L - 1, 64)), torch.sigmoid(r(T, 2, add=3.0)), torch.sigmoid(r(T, 2)),
            0.5 * torch.sigmoid(r(T, 2, L - 1, 64)), torch.sigmoid(r(T, 2, L - 1, 64)), r(2, 64, 4, mul=0.5),
            r(T, 2, 64), r(64, mul=0.2, add=1.0), r(128, mul=0.2, add=1.0)]
    cu = torch.tensor([0, 25, 25, T], dtype=torch.int32).cuda()
    dn, dr = r(T, 128), r(T, 128)
    leaves = [t.detach().requires_grad_(True) for t in base]

    def loss_of(ts):
        n2, r2 = layer(ts, cu, L)
        return float((f64(n2) * f64(dn)).sum() + (f64(r2) * f64(dr)).sum())

    grads = torch.autograd.grad(layer(leaves, cu, L), leaves, [dn, dr])
    h = 2.0 ** -7
    for i, t in enumerate(base):
        d = r(*t.shape, mul=float(t.std()) if t.std() > 0 else 1.0)
        with torch.no_grad():
            hi = loss_of([x + h * d if j == i else x for j, x in enumerate(base)])
            lo = loss_of([x - h * d if j == i else x for j, x in enumerate(base)])
        got, want = (hi - lo) / (2 * h), float((f64(grads[i]) * f64(d)).sum())
        scale = float(f64(grads[i]).norm() * f64(d).norm())
        say(f"leaf {i}: {got:.5f} by differences, {want:.5f} (scale {scale:.3f})")
        # h^2 / 6 of the third derivative along d, and 2^-23 n^(1/2) |L's terms| / h of rounding: see
        # the norms' own test; a block chains three such steps
        assert abs(got - want) <= 1e-2 * scale, i


def test_norm_backward_replays_from_a_graph():
    """The norms' forward and backward captured on fresh leaves and replayed several times."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(6)
    bf = torch.bfloat16
    x, y, dn, dr = (torch.randn(3000, 128, generator=gen).to(bf).cuda() for _ in range(4))
    w, s = (torch.rand(128, generator=gen).to(bf).cuda() for _ in range(2))

    def run():
        n, r = B.norm_residual(x, w, y=y, scale=s)
        g = B.norm_residual_bwd(r, w, dn, dr=dr, y=y, scale=s)
        o = n.view(-1, 2, 64)
        gg = B.norm_gate_bwd(o, y.view_as(o), w[:64], dn.view_as(o))
        return {"n": n, "r": r, **{"res " + k: v for k, v in g.items()}, **{"gate " + k: v for k, v in gg.items()}}

    ref = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for rep in range(4):
        for t in out.values():
            t.zero_()
        g.replay()
        eager = run()
        torch.cuda.synchronize()
        assert not same(ref, out) and not same(ref, eager), rep
