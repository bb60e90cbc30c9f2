"""The steps in front of the operator and behind the last product together with it, as a program uses
them: prompts, then tokens one by one, a draft and its verification; a training step; captured and
replayed, on other streams."""
import pytest

from tests import stack_refs as R
from tests.layer_refs import f64

pytestmark = pytest.mark.gpu
H, D, K = 2, 64, 4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


class Layer:
    """Projections (given), short convolution, norm and rotation of q and k, the operator (L = 1), the
    gated norm, logits (given), the token."""

    def __init__(self, seed=0, V=900):
        import torch
        gen = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        rand = lambda *s: torch.randn(s, generator=gen).to(bf).cuda()
        self.w = (0.5 * rand(3 * H * D, K).float()).to(bf)
        self.conv_w = rand(H, D, K)
        self.wg = (1 + 0.1 * rand(H, D).float()).to(bf)
        self.head = rand(H * D, V)
        self.freqs = R_freqs()
        self.gen, self.V = gen, V

    def inputs(self, T):
        import torch
        rand = lambda *s: torch.randn(s, generator=self.gen).to(torch.bfloat16).cuda()
        return {"x": rand(T, 3 * H * D + 32), "g": torch.sigmoid(3 + rand(T, H).float()).to(torch.bfloat16),
                "b": torch.sigmoid(rand(T, H).float()).to(torch.bfloat16), "z": rand(T, H, D)}

    def mix(self, y, pos):
        from gated_delta_rule_prologue_amd import binding as B
        T = y.shape[0]
        q, k, v = (y[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(3))
        q, k = B.qk_norm(q, k, positions=pos, freqs=self.freqs)
        return q, k, v.contiguous()

    def logits(self, o, z):
        from gated_delta_rule_prologue_amd import binding as B
        n = B.norm_gate(o, z, self.wg).view(o.shape[0], -1, 1).float()
        return (n * self.head.float()).sum(1)                # a fixed order: no library product


def R_freqs():
    from gated_delta_rule_prologue_amd import binding as B
    return B.rotary_freqs(D, factor=2.0, trained=2048)


def prompt(m, x, cu, pos, conv_hist, S, k_hist):
    from gated_delta_rule_prologue_amd import binding as B
    y, _ = B.short_conv(x["x"][:, :3 * H * D], m.w, cu, hist=conv_hist, hist_out=conv_hist)
    q, k, v = m.mix(y, pos)
    o, _, _ = B.fwd_resume(q, k, v, None, x["g"], x["b"], None, None, m.conv_w, cu, 1, S_init=S, S_final=S, k_hist=k_hist,
                           k_hist_out=k_hist)
    return o


def token(m, x, pos, conv_hist, S, k_hist):
    from gated_delta_rule_prologue_amd import binding as B
    y, _ = B.short_conv_step(x["x"][:, :3 * H * D], m.w, conv_hist)
    q, k, v = m.mix(y, pos)
    return B.decode_step(q, k, v, None, x["g"], x["b"], None, None, m.conv_w, 1, S, k_hist)


def state(N):
    import torch
    return (torch.zeros(N, K - 1, 3 * H * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, H, D, D, device="cuda"),
            torch.zeros(N, H, 3, D, dtype=torch.bfloat16, device="cuda"))


def test_tokens_continue_prompts():
    """Prompts of several lengths and then single tokens against the whole sequences in one call; the draws
    against the reference on the same logits."""
    import numpy as np
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    m, lens, steps = Layer(), [5, 1, 70], 3
    full = [n + steps for n in lens]
    off = np.concatenate([[0], np.cumsum(full)])
    x = m.inputs(int(off[-1]))
    pos = torch.cat([torch.arange(n) for n in full]).int().cuda()
    whole = prompt(m, x, torch.tensor(off, dtype=torch.int32).cuda(), pos, *state(3))
    pick = lambda rows: {k: v[rows].contiguous() for k, v in x.items()}
    rows = torch.cat([torch.arange(off[i], off[i] + n) for i, n in enumerate(lens)]).cuda()
    st = state(3)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    parts = [(rows, prompt(m, pick(rows), cu, pos[rows], *st))]
    for t in range(steps):
        rows = torch.tensor([off[i] + n + t for i, n in enumerate(lens)]).cuda()
        x1 = pick(rows)
        o = token(m, x1, pos[rows], *st)
        parts.append((rows, o))
        logits = m.logits(o, x1["z"])
        u = torch.rand(3, generator=m.gen)
        t_, p_ = torch.full((3,), 0.8), torch.full((3,), 0.9)
        tokens, probs = B.sample(logits, u.cuda(), temperature=t_.cuda(), top_p=p_.cuda(), want_probs=True)
        for n in range(3):
            row = logits[n].double().cpu().numpy()
            f = dict(t=float(t_[n]), p=float(p_[n]))
            assert tokens[n].item() == R.sample(row, float(u[n]), **f)
            assert abs(probs[n].double().cpu().numpy() - R.probs(row, **f)).max() <= 2.0 ** -23
    for rows, o in parts:                                    # two forms of the operator, bf16 outputs
        ref = whole[rows].float()
        assert (o.float() - ref).abs().max() <= 1e-2 * whole.float().abs().max()


def test_drafts_with_sampled_distributions():
    """The distributions of draft and target feed the verification as they are."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    from tests import layer_refs as L
    gen = torch.Generator().manual_seed(1)
    V, cu = 1000, [0, 4, 4, 9, 10]
    T = cu[-1]
    target = 3 * torch.randn(T, V, generator=gen).cuda()
    draft = target + 0.5 * torch.randn(T, V, generator=gen).cuda()
    p_ = torch.full((T,), 0.9).cuda()
    u = torch.rand(T, generator=gen).cuda()
    drawn, q = B.sample(draft, u, top_p=p_, want_probs=True)
    tokens = torch.roll(drawn, 1).contiguous()               # the token after row t is fed at t + 1
    _, p = B.sample(target, top_p=p_, want_probs=True)
    ua, us = torch.rand(T, generator=gen).cuda(), torch.rand(4, generator=gen).cuda()
    cu_t = torch.tensor(cu, dtype=torch.int32).cuda()
    kept, nxt = B.verify_draft(p, tokens, cu_t, ua, us, q=q)
    want = L.verify(f64(p).numpy(), f64(q).numpy(), tokens.cpu().numpy(), cu, ua.cpu().numpy(), us.cpu().numpy())
    assert kept.cpu().tolist() == want[0] and nxt.cpu().tolist() == want[1]
    assert all(p[c - 1 if c else 0].sum() > 0.999 for c in cu[1:])


def test_training_step():
    """Gradients of the projections through the convolution, the norms and the operator, against the same
    formula in 64 bits (the recurrence token by token); finite and as large as those."""
    import torch
    from gated_delta_rule_prologue_amd import autograd as A
    from tests import layer_refs as L
    m = Layer(seed=2)
    lens = [9, 30]
    T, cu = sum(lens), [0, 9, 39]
    x = m.inputs(T)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    cu_t = torch.tensor(cu, dtype=torch.int32).cuda()
    wq = (1 + 0.1 * torch.randn(D, generator=m.gen)).to(torch.bfloat16).cuda()
    leaves = {"x": x["x"].clone(), "w": m.w.clone(), "wq": wq, "wk": wq.clone()}
    leaves = {n: t.requires_grad_(True) for n, t in leaves.items()}
    y = A.short_conv(leaves["x"][:, :3 * H * D], leaves["w"], cu_t)
    q, k, v = (y[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(3))
    q, k = A.qk_norm(q, k, leaves["wq"], leaves["wk"], positions=pos, freqs=m.freqs)
    o, _ = A.prism(q, k, v.contiguous(), None, x["g"], x["b"], None, None, m.conv_w, cu_t, 1)
    up = torch.randn(T, H, D, generator=m.gen)
    (o.float() * up.cuda()).sum().backward()

    six = {n: f64(t).requires_grad_(True) for n, t in leaves.items()}
    y6, _, _ = R.short_conv(six["x"][:, :3 * H * D], six["w"], cu)
    q6, k6, v6 = (y6[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(3))
    q6 = R.qk_norm(q6, six["wq"], "l2", 1e-6, pos.cpu(), m.freqs.cpu())
    k6 = R.qk_norm(k6, six["wk"], "l2", 1e-6, pos.cpu(), m.freqs.cpu())
    outs = []
    for n in range(len(lens)):
        S = torch.zeros(H, D, D).double()
        for t in range(cu[n], cu[n + 1]):
            b, g = f64(x["b"])[t][:, None], f64(x["g"])[t][:, None, None]
            p = torch.einsum("hij,hi->hj", S, k6[t])
            S = g * (S - (b * k6[t])[:, :, None] * p[:, None]) + (b * k6[t])[:, :, None] * v6[t][:, None]
            outs.append(torch.einsum("hij,hi->hj", S, q6[t]))
    (torch.stack(outs) * up.double()).sum().backward()
    for n in leaves:
        g, r = f64(leaves[n].grad), six[n].grad
        # bf16 storage of y, q, k, o and of their gradients, a few half steps of 2^-8 of the largest
        assert (g - r).abs().max() <= 4e-2 * r.abs().max(), n


@pytest.mark.parametrize("others", [False, True])
def test_captured_and_replayed(others):
    """The whole token step in a graph, replayed on new inputs between eager work, with a second graph beside
    it; on another stream."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    m = Layer(seed=3)
    N = 4
    settings = dict(temperature=torch.full((N,), 0.7).cuda(), top_k=torch.full((N,), 50, dtype=torch.int32).cuda(),
                    top_p=torch.full((N,), 0.9).cuda(), min_p=torch.full((N,), 0.01).cuda())

    def step(x, pos, u, st):
        o = token(m, x, pos, *st)
        logits = m.logits(o, x["z"])
        tokens, probs = B.sample(logits, u, want_probs=True, **settings)
        return o, logits, tokens, probs

    x, pos, u = m.inputs(N), torch.arange(N).int().cuda(), torch.rand(N).cuda()
    st = state(N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, pos, u, [t.clone() for t in st])             # builds what the first call builds
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2 if others else 1):
        own = [t.clone() for t in st]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(x, pos, u, own)
        graphs.append((g, own, outs))
    eager = [t.clone() for t in st]
    for r in range(4):
        new = m.inputs(N)
        for k in x:
            x[k].copy_(new[k])
        pos.add_(1)
        u.copy_(torch.rand(N))
        want = step(x, pos, u, eager)
        for g, own, outs in graphs:
            if others:
                with torch.cuda.stream(side):
                    side.wait_stream(torch.cuda.default_stream())
                    g.replay()
                side.synchronize()
            else:
                g.replay()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), r
            assert all(torch.equal(a, b) for a, b in zip(own, eager)), r
        torch.cuda.synchronize()


def test_captured_training_passes():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
    T, C = 300, 3 * H * D
    x, w, dy, bias = rand(T, C), rand(C, K), rand(T, C), rand(C)
    hist = rand(2, K - 1, C)
    cu = torch.tensor([0, 120, T], dtype=torch.int32).cuda()
    q, k, dq, dk, wq = rand(T, H, D), rand(T, H, D), rand(T, H, D), rand(T, H, D), rand(D)
    pos, freqs = torch.arange(T).int().cuda(), R_freqs()

    def both():
        a = B.short_conv_bwd(x, w, cu, dy, bias=bias, hist=hist)
        b = B.qk_norm_bwd(q, dq, k, dk, wq, wq, norm="rms", positions=pos, freqs=freqs)
        return [*a.values(), *b.values()]

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = both()
    for _ in range(3):
        for t in (x, dy, q, dq):
            t.copy_(rand(*t.shape))
        want = both()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        torch.cuda.synchronize()


def test_streams():
    """Calls given a stream run there, in order behind its other work."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(6)
    s = torch.cuda.Stream()
    big = torch.randn(2000, 2000, device="cuda")
    x = torch.zeros(64, 32, device="cuda")
    src = torch.randn(64, 32, generator=gen).cuda()
    w = torch.randn(32, 4, generator=gen).cuda()
    cu = torch.tensor([0, 64], dtype=torch.int32).cuda()
    u = torch.rand(64, generator=gen).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            big = big @ big * 1e-3
        x.copy_(src)
    y, _ = B.short_conv(x, w, cu, stream=s)
    q, _ = B.qk_norm(y.view(64, 4, 8), stream=s)
    tokens, _ = B.sample(q.view(64, 32), u, stream=s.cuda_stream)
    torch.cuda.synchronize()
    y2, _ = B.short_conv(src, w, cu)
    q2, _ = B.qk_norm(y2.view(64, 4, 8))
    t2, _ = B.sample(q2.view(64, 32), u)
    assert torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(tokens, t2)
