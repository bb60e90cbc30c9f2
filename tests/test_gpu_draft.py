"""Drafted tokens (prism_decode_draft, prism_decode_commit) against the token-by-token
recurrence in 64 bits.

Tolerances.  The records and fp32 outputs come from fp32 sums of dk <= 128 products and
a triangular system over at most 16 tokens (8 a pass) whose couplings b k.k are at most 1 in
size: 128 + 2 x 16 terms' roundings (160 x 2^-24 = 1e-5) times the solve's growth
(below 10 for unit keys and b <= 1) stays under 1e-4 of the largest element, the bound
this operator's fp32 results are held to everywhere.  A bf16 output adds its own
rounding, 2^-8 of the value.  The commit adds up to 2 x 40 products on the state it is given:
(80 + 40) x 2^-24 = 8e-6 of the largest magnitude."""
import numpy as np
import pytest

from tests.gpu_common import say
from tests.layer_refs import HALF_STEP, f64
from tests import layer_refs as R

pytestmark = pytest.mark.gpu
TOL = 1e-4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def make(lens, H=2, dk=64, dv=64, L=4, dtype="bf16", seed=0):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(seed)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, N = cu[-1], len(lens)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    def unit(*shape):
        x = normal(*shape)
        return x / x.norm(dim=-1, keepdim=True)

    d = {"q": unit(T, H, dk), "k": unit(T, H, dk), "v": normal(T, H, dv),
         "u": unit(T, H, L - 1, dk) if L > 1 else None, "g": torch.sigmoid(3 + normal(T, H)),
         "b": torch.sigmoid(normal(T, H)), "a": 0.5 * torch.sigmoid(normal(T, H, L - 1, dk)) if L > 1 else None,
         "h": torch.sigmoid(normal(T, H, L - 1, dk)) if L > 1 else None, "conv_w": 0.5 * normal(H, dk, 4)}
    d = {k: None if v is None else v.to(dt).cuda() for k, v in d.items()}
    S, hist = (0.3 * normal(N, H, dk, dv)).cuda(), unit(N, H, 3, dk).to(dt).cuda()
    return d, cu, torch.tensor(cu, dtype=torch.int32).cuda(), S, hist


def run(d, cu_t, L, S, hist, **kw):
    from gated_delta_rule_prologue_amd import binding as B
    return B.decode_draft(d["q"], d["k"], d["v"], d["u"], d["g"], d["b"], d["a"], d["h"], d["conv_w"], cu_t, L, S,
                          hist, **kw)


def near(name, got, ref, tol=TOL):
    """The error bound above; returns the worst share of it."""
    g, r = f64(got), ref.double()
    assert g.shape == r.shape, name
    if not g.numel():
        return 0.0
    half = HALF_STEP[got.dtype] * r.abs()
    bound = half + tol * r.abs().max()
    assert torch_all_finite(g), name
    share = float(((g - r).abs() / bound).max())
    assert share <= 1, (name, share)
    return share


def torch_all_finite(t):
    import torch
    return bool(torch.isfinite(t).all())


def commit(d, cu_t, kept, kw, p, S, hist, **more):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    n = torch.tensor(kept, dtype=torch.int32, device="cuda")
    return B.decode_commit(d["k"], d["v"], d["g"], d["b"], cu_t, n, kw, p, S, hist, **more)


LENS = [1, 5, 0, 16, 2, 17, 3, 4, 9, 33, 8, 40, 0, 15]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("L,residual", [(1, "linear"), (2, "linear"), (4, "linear"), (4, "gelu"), (8, "gelu")])
def test_draft_and_commit(dtype, dk, dv, L, residual):
    """Outputs and records of ragged drafts, none to 40 tokens; the state after every kind of
    commit (nothing kept, some, all, counts out of range), in place and not."""
    import torch
    d, cu, cu_t, S, hist = make(LENS, dk=dk, dv=dv, L=L, dtype=dtype, seed=dk + dv + L)
    S0, hist0 = S.clone(), hist.clone()
    o, kw, p = run(d, cu_t, L, S, hist, residual=residual)
    assert torch.equal(S, S0) and torch.equal(hist, hist0)        # read only
    d6 = {k: f64(v) for k, v in d.items()}
    ro, rkw, rp, _ = R.draft(d6, cu, L, f64(S), f64(hist), residual)
    share = max(near("o", o, ro), near("kw", kw, rkw), near("p", p, rp))
    kept = [1, 3, 4, 16, -2, 17, 0, 4, 100, 20, 8, 33, 0, 15]
    S_out, h_out = torch.full_like(S, float("nan")), torch.zeros_like(hist)
    commit(d, cu_t, kept, kw, p, S, hist, S_out=S_out, k_hist_out=h_out)
    assert torch.equal(S, S0) and torch.equal(hist, hist0)
    rS, rh = R.commit(f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["b"]), cu, kept, f64(kw), f64(p), f64(S), f64(hist))
    share = max(share, near("S", S_out, rS, 8e-6))
    assert torch.equal(f64(h_out), rh)
    for n in (2, 4, 6, 12):                                        # nothing kept: the same bits
        assert torch.equal(S_out[n], S0[n]) and torch.equal(h_out[n], hist0[n]), n
    got = commit(d, cu_t, kept, kw, p, S, hist)                    # in place
    assert got[0] is S and got[1] is hist
    assert torch.equal(S, S_out) and torch.equal(hist, h_out)
    say(f"draft {dtype} {dk}x{dv} L={L} {residual}: worst share of the tolerance {share:.2f}")


def test_states_follow_the_tokens():
    """The committed state is the recurrence's after that token (from the records alone)."""
    import torch
    d, cu, cu_t, S, hist = make([12] * 12, dk=128, dv=128, dtype="f32", seed=3)
    o, kw, p = run(d, cu_t, 4, S, hist)
    states = R.draft({k: f64(v) for k, v in d.items()}, cu, 4, f64(S), f64(hist), "linear")[3]
    S_out, _ = commit(d, cu_t, list(range(1, 13)), kw, p, S, hist, S_out=torch.empty_like(S),
                      k_hist_out=torch.empty_like(hist))
    for n in range(12):
        near(f"state after {n + 1}", S_out[n], states[cu[n] + n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equals_decode_steps(dtype):
    """A draft and its whole commit against prism_decode_step token by token (both
    within the bound of the exact result, so within twice of each other)."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    M, N = 6, 5
    d, cu, cu_t, S, hist = make([M] * N, H=3, dk=128, dv=64, dtype=dtype, seed=11)
    o, kw, p = run(d, cu_t, 4, S, hist)
    S1, h1 = S.clone(), hist.clone()
    at = torch.tensor(cu[:-1], device="cuda")
    for t in range(M):
        x = {k: v if k == "conv_w" else v[at + t].contiguous() for k, v in d.items()}
        ot = B.decode_step(x["q"], x["k"], x["v"], x["u"], x["g"], x["b"], x["a"], x["h"], x["conv_w"], 4, S1, h1)
        near(f"o {t}", o[at + t], f64(ot), 2 * TOL + HALF_STEP[o.dtype])
    commit(d, cu_t, [M] * N, kw, p, S, hist)
    near("S", S, f64(S1), 2 * TOL)
    assert torch.equal(hist, h1)


def test_extreme_gates():
    """Gates of exactly zero and one, b of zero: no quotient of gate products is formed."""
    import torch
    d, cu, cu_t, S, hist = make([16, 7, 20], dtype="f32", seed=5)
    d["g"][3], d["g"][18], d["g"][30] = 0.0, 0.0, 0.0
    d["g"][5:9] = 1.0
    d["b"][::3] = 0.0
    o, kw, p = run(d, cu_t, 4, S, hist)
    ref = R.draft({k: f64(v) for k, v in d.items()}, cu, 4, f64(S), f64(hist), "linear")
    near("o", o, ref[0]); near("p", p, ref[2])
    kept = [16, 7, 20]
    S_out, _ = commit(d, cu_t, kept, kw, p, S, hist, S_out=torch.empty_like(S), k_hist_out=torch.empty_like(hist))
    for n in range(3):
        near("S", S_out[n], ref[3][cu[n + 1] - 1])


@pytest.mark.parametrize("what", ["v nan", "k inf", "u nan", "g nan", "v huge"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_later_tokens_do_not_reach_earlier_ones(what, dtype):
    """A value of token 5 that is not finite (or overflows products) leaves tokens 0..4
    and other sequences as the recurrence has them, and shows from token 5 on; the commit
    of the first 5 tokens is clean."""
    import torch
    d, cu, cu_t, S, hist = make([9, 9, 18], dk=128, dv=64, dtype=dtype, seed=7)
    name, value = what.split()
    value = {"nan": float("nan"), "inf": float("inf"), "huge": 1e30}[value]
    clean = run(d, cu_t, 4, S, hist)
    for row in (5, 18 + 5):
        if name == "g":
            d[name][row, 0] = value
        elif name == "u":
            d[name][row, 0, 0, 3] = value
        else:
            d[name][row, 0, 3] = value
    o, kw, p = run(d, cu_t, 4, S, hist)
    ref = R.draft({k: f64(v) for k, v in d.items()}, cu, 4, f64(S), f64(hist), "linear")
    early = list(range(5)) + list(range(9, 18)) + list(range(18, 23))
    for got, want in zip((o, kw, p), ref):
        near(f"{what} before", got[early], want[early])
        near(f"{what} other head", got[:, 1], want[:, 1])
    assert torch.equal(torch.isfinite(o[5, 0]).cpu(), torch.isfinite(ref[0][5, 0])) or name == "v"
    if value != 1e30:
        assert not torch.isfinite(o[5:9, 0]).all(1).any()
    kept = [5, 9, 5]
    S_out, _ = commit(d, cu_t, kept, kw, p, S, hist, S_out=torch.empty_like(S), k_hist_out=torch.empty_like(hist))
    rS, _ = R.commit(f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["b"]), cu, kept, f64(kw), f64(p), f64(S), f64(hist))
    near("S", S_out, rS, 8e-6)
    del clean


def test_long_drafts():
    """The longest sequence that is served (gates about 0.95: what a token leaves fades within
    a few passes, so the bound is that of short ones), and one token more, whose outputs and
    records are NaN while its neighbours' are not."""
    import torch
    lens = [3, 1024, 1025, 9]
    d, cu, cu_t, S, hist = make(lens, H=1, dk=64, dv=128, L=3, seed=13)
    o, kw, p = run(d, cu_t, 3, S, hist)
    for x in (o, kw, p):
        assert torch.isnan(x[cu[2]:cu[3]]).all()
    keep = [n for n in range(len(lens)) if n != 2]
    for n in keep:
        at = slice(cu[n], cu[n + 1])
        ref = R.draft({k: f64(v) if k == "conv_w" or v is None else f64(v[at]) for k, v in d.items()}, [0, lens[n]], 3,
                      f64(S[n:n + 1]), f64(hist[n:n + 1]), "linear")
        for name, got, want in zip(("o", "kw", "p"), (o, kw, p), ref):
            near(f"{name} of {lens[n]} tokens", got[at], want)
    S_out, h_out = commit(d, cu_t, [3, 1024, 0, 9], kw, p, S, hist, S_out=torch.empty_like(S),
                          k_hist_out=torch.empty_like(hist))
    assert torch.equal(S_out[2], S[2]) and torch.equal(h_out[2], hist[2])
    rS, _ = R.commit(f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["b"]), cu, [3, 1024, 0, 9], f64(kw).nan_to_num(),
                     f64(p).nan_to_num(), f64(S), f64(hist))
    near("S", S_out, rS, 8e-6)               # 17 roundings a pass of the state, that fade within 3 or 4 passes


def test_rows_behind_the_last_token_stay():
    """Buffers longer than the packed tokens: the rows behind are not written."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    d, cu, cu_t, S, hist = make([3, 0, 4], seed=2)
    T = cu[-1]
    big = {"o": torch.full((T + 5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"),
           "kw": torch.full((T + 5, 2, 64), 7.0, device="cuda"), "p": torch.full((T + 5, 2, 64), 7.0, device="cuda")}
    run(d, cu_t, 4, S, hist, **{k: v[:T] for k, v in big.items()})
    for v in big.values():
        assert (v[T:] == 7.0).all() and (v[:T] != 7.0).any()


def test_no_tokens():
    """A step in which no sequence drafts: the outputs are empty, the commit keeps the state."""
    import torch
    d, cu, cu_t, S, hist = make([0, 0], seed=1)
    o, kw, p = run(d, cu_t, 4, S, hist)
    assert o.shape[0] == kw.shape[0] == p.shape[0] == 0
    S_out, h_out = commit(d, cu_t, [0, 3], kw, p, S, hist, S_out=torch.empty_like(S), k_hist_out=torch.empty_like(hist))
    assert torch.equal(S_out, S) and torch.equal(h_out, hist)


def test_large_batch():
    """The full serving batch, against decode steps' reference on sampled sequences."""
    import torch
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 9, 300)]
    d, cu, cu_t, S, hist = make(lens, H=6, dk=128, dv=128, seed=20)
    o, kw, p = run(d, cu_t, 4, S, hist)
    kept = [int(rng.integers(0, n + 1)) for n in lens]
    S_out, h_out = commit(d, cu_t, kept, kw, p, S, hist, S_out=torch.empty_like(S), k_hist_out=torch.empty_like(hist))
    for n in (0, 77, 150, 299):
        rows = slice(cu[n], cu[n + 1])
        sub = {k: f64(v) if k == "conv_w" else f64(v[rows]) for k, v in d.items()}
        ref = R.draft(sub, [0, lens[n]], 4, f64(S[n:n + 1]), f64(hist[n:n + 1]), "linear")
        near("o", o[rows], ref[0]); near("p", p[rows], ref[2])
        if kept[n]:
            near("S", S_out[n], ref[3][kept[n] - 1])
        else:
            assert torch.equal(S_out[n], S[n])
