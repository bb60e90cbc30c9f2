"""The choice of a token (prism_sample) against a sort in 64 bits.

Tokens have to be the reference's: weights here are exact to 2^-43 of the largest and their
sums exact, the reference's to 2^-53 of each and its sums to some 10^-12, so both choose alike but where u times the
total, or a filter's border, lies within 10^-11 of a running sum; rows of equal logits, where borders are
met, have weights of one and exact sums on both sides.  Probabilities are rounded once to fp32
(2^-24), after a total that is off by at most 2^-44 an entry over at least one."""
import numpy as np
import pytest

from tests import stack_refs as R
from tests.gpu_common import say

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def settings(n, seed):
    """Per-row settings, each filter off in some rows."""
    r = np.random.default_rng(seed)
    off = lambda x, o, p: np.where(r.random(n) < p, o, x)
    return {"t": off(0.3 + 1.5 * r.random(n), 0.0, 0.1).astype(np.float32),
            "k": off(np.exp(r.random(n) * 6).astype(np.int32), 0, 0.5).astype(np.int32),
            "p": off(r.random(n), 1.0, 0.4).astype(np.float32),
            "m": off(0.3 * r.random(n), 0.0, 0.5).astype(np.float32)}


def run(logits, u=None, t=None, k=None, p=None, m=None, **kw):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    dev = lambda x, dt: None if x is None else torch.as_tensor(np.asarray(x), dtype=dt).cuda()
    tokens, probs = B.sample(logits, dev(u, torch.float32), dev(t, torch.float32), dev(k, torch.int32),
                             dev(p, torch.float32), dev(m, torch.float32), **kw)
    return (None if tokens is None else tokens.cpu().numpy(), None if probs is None else probs.cpu().numpy())


def check(logits, u, f, rows=None, probs=True):
    """Tokens and distributions of every row against the reference."""
    l = logits.double().cpu().numpy()
    tokens, pr = run(logits, u, want_probs=probs, **f)
    for n in range(len(l)) if rows is None else rows:
        one = {name: v[n] for name, v in f.items()}
        want = R.sample(l[n], u[n], **{a: float(b) if a != "k" else int(b) for a, b in one.items()})
        assert tokens[n] == want, (n, one, u[n], tokens[n], want)
        if probs:
            ref = R.probs(l[n], **{a: float(b) if a != "k" else int(b) for a, b in one.items()})
            assert ((pr[n] > 0) == (ref > 2.0 ** -149)).all() or (np.abs(pr[n] - ref) < 2.0 ** -126).all(), (n, one)
            assert (np.abs(pr[n] - ref) <= 2.0 ** -23 * ref + 2.0 ** -126).all(), (n, one)
    return tokens, pr


VOCABS = [1, 2, 3, 7, 8, 9, 63, 64, 100, 1000, 1023, 1024, 1025, 2049, 4095, 4096, 4097, 4104, 16384, 16385, 32000,
          32768, 32769, 50001, 65536, 65543, 70000, 131072, 131073, 200001]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_vocabularies(dtype):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    for V in VOCABS:
        N = 24 if V < 5000 else 8
        gen = torch.Generator().manual_seed(V)
        logits = (3 * torch.randn(N, V, generator=gen)).to(dt).cuda()
        check(logits, np.random.default_rng(V).random(N).astype(np.float32), settings(N, V))


@pytest.mark.parametrize("filters", ["", "k", "p", "m", "kp", "km", "pm", "kpm"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_filters(dtype, filters):
    """Every combination, with rows from one token to a batch; settings left out are off."""
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    for N in (1, 3, 300):
        gen = torch.Generator().manual_seed(N)
        logits = (2 * torch.randn(N, 777, generator=gen)).to(dt).cuda()
        f = {n: v for n, v in settings(N, N + 1).items() if n in "t" + filters}
        check(logits, np.random.default_rng(N).random(N).astype(np.float32), f)


def test_no_settings_at_all():
    import torch
    logits = torch.randn(5, 333, generator=torch.Generator().manual_seed(0)).cuda()
    check(logits, np.array([0, 0.2, 0.5, 0.8, 1 - 2.0 ** -24], dtype=np.float32), {})


@pytest.mark.parametrize("V", [1000, 5000, 40000, 140000])
def test_equal_logits(V):
    """Rows of one value: the order is the index alone, over far more entries than a list holds, and
    every border falls on a running sum exactly."""
    import torch
    N = 16
    u = (np.arange(N) / N).astype(np.float32)
    for value in (0.0, -7.25, LOWEST):
        logits = torch.full((N, V), value).cuda()
        for f in ({}, {"k": np.arange(N, dtype=np.int32) * (V // N) + 1}, {"p": ((1 + np.arange(N)) / N).astype(np.float32)},
                  {"k": np.full(N, V // 2, np.int32), "p": np.full(N, 0.5, np.float32)}, {"m": np.full(N, 1.0, np.float32)}):
            check(logits, u, f, probs=V < 50000)
    half = torch.full((N, V), 1.0).cuda()                    # two values: the ties of the lower one are cut
    half[:, ::2] = 0.5
    check(half, u, {"k": np.full(N, V // 2 + V // 4 + 1, np.int32)})


def test_signed_zeros_are_equal():
    import torch
    logits = torch.tensor([[0.0, -0.0, 0.0, -0.0], [-0.0, 0.0, -1.0, 0.0]]).cuda()
    for u, want in ((0.1, [0, 0]), (0.3, [1, 0]), (0.6, [2, 1]), (0.9, [3, 3])):
        tokens, _ = run(logits, [u, u], k=[4, 3])
        assert tokens.tolist() == want
    tokens, _ = run(logits, [0.9, 0.9], t=[0, 0])
    assert tokens.tolist() == [0, 0]


@pytest.mark.parametrize("V", [37, 3000, 70001])
def test_masked_and_extreme_entries(V):
    """-infinity, NaN, +infinity and the type's lowest value, alone and beside others; rows with nothing left."""
    import torch
    inf, nan = float("inf"), float("nan")
    rng = np.random.default_rng(V)
    base = rng.standard_normal((12, V)).astype(np.float32)
    base[0] = -inf
    base[1] = nan
    base[2, rng.random(V) < 0.5] = -inf
    base[3, rng.random(V) < 0.5] = nan
    base[4] = -inf
    base[4, V // 2] = -3.0
    base[5, [1, V - 2]] = inf
    base[6] = inf
    base[7] = LOWEST
    base[8, : V - 3] = LOWEST
    base[9, ::2] = 3e38
    base[9, 1::2] = -3e38
    base[10, 1:] = LOWEST
    base[11, ::3] = nan
    base[11, 1::3] = -inf
    logits = torch.from_numpy(base).cuda()
    u = rng.random(12).astype(np.float32)
    for f in ({}, {"t": np.full(12, 0.7, np.float32)}, {"k": np.full(12, 5, np.int32), "p": np.full(12, 0.9, np.float32)},
              {"m": np.full(12, 0.05, np.float32)}, {"t": np.zeros(12, np.float32)}, {"p": np.full(12, 0.2, np.float32)}):
        tokens, pr = check(logits, u, f)
        assert tokens[0] == tokens[1] == -1 and (pr[0] == 0).all() and (pr[1] == 0).all()


@pytest.mark.parametrize("t", [1e-38, 1e-30, 1e-6, 1e-2, 30.0, 1e6, 1e30, float("inf")])
def test_temperatures(t):
    """From where the largest alone has weight to where all weigh the same."""
    import torch
    gen = torch.Generator().manual_seed(3)
    logits = (4 * torch.randn(6, 9000, generator=gen)).cuda()
    u = np.array([0, 0.1, 0.4, 0.7, 0.95, 1 - 2.0 ** -24], dtype=np.float32)
    tt = np.full(6, t, np.float32)
    for f in ({}, {"k": np.full(6, 3000, np.int32)}, {"p": np.full(6, 0.6, np.float32)}, {"m": np.full(6, 0.9, np.float32)}):
        check(logits, u, {"t": tt, **f}, probs=False)


def test_settings_at_and_beyond_their_ends():
    import torch
    nan, inf = float("nan"), float("inf")
    gen = torch.Generator().manual_seed(4)
    V = 500
    logits = torch.randn(8, V, generator=gen).cuda()
    u = np.linspace(0.05, 0.95, 8).astype(np.float32)
    check(logits, u, {"k": np.array([0, -1, -2 ** 31, 1, V - 1, V, V + 1, 2 ** 31 - 1], dtype=np.int64).astype(np.int32)})
    check(logits, u, {"p": np.array([0, -1, -inf, 1e-30, 1, 2, inf, 1 - 2.0 ** -24], np.float32)})
    check(logits, u, {"m": np.array([0, -1, -inf, 1e-45, 1, 2, inf, 1 - 2.0 ** -24], np.float32)})
    check(logits, u, {"t": np.array([0, -1, -inf, -0.0, 1, 2, 1e-45, 0.5], np.float32)})
    one = {"t": nan, "p": nan, "m": nan}
    for name in one:
        tokens, _ = run(logits, u, **{name: np.full(8, nan, np.float32)})
        off = {"t": 0.0, "p": 1.0, "m": 0.0}[name]
        want, _ = run(logits, u, **{name: np.full(8, off, np.float32)})
        assert (tokens == want).all()
    # random numbers outside [0, 1) count as the nearest inside
    tokens, _ = run(logits, np.array([-1, nan, -inf, 0, 1, 2, inf, 1 - 2.0 ** -24], np.float32))
    want, _ = run(logits, np.array([0, 0, 0, 0] + [1 - 2.0 ** -24] * 4, np.float32))
    assert (tokens == want).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(dtype):
    """Columns of a padded table, rows at any element's address, every row the same."""
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(6)
    wide = (3 * torch.randn(9, 5011, generator=gen)).to(dt).cuda()
    u = np.random.default_rng(6).random(9).astype(np.float32)
    for cut in (wide[:, :5000], wide[:, 1:4998], wide[:, 7:], wide[:1].expand(9, -1)):
        check(cut, u, settings(9, 7))


def test_the_same_bits_again():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(8)
    logits = torch.randn(40, 60000, generator=gen).to(torch.bfloat16).cuda()     # many ties
    u = torch.rand(40, generator=gen).cuda()
    p = torch.full((40,), 0.9).cuda()
    first = B.sample(logits, u, top_p=p, want_probs=True)
    for _ in range(5):
        again = B.sample(logits, u, top_p=p, want_probs=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_draws_follow_the_distribution():
    """Evenly spaced u draw every entry as often as its probability says, to one draw."""
    import torch
    N, V = 4000, 50
    row = torch.randn(1, V, generator=torch.Generator().manual_seed(9)).cuda()
    u = ((np.arange(N) + 0.5) / N).astype(np.float32)
    tokens, _ = run(row.expand(N, -1), u)
    pr = R.probs(row[0].double().cpu().numpy())
    assert (np.abs(np.bincount(tokens, minlength=V) - N * pr) <= 1.01).all()


def test_given_outputs_and_none():
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    logits = torch.randn(3, 100, device="cuda")
    u = torch.rand(3, device="cuda")
    tokens, probs = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, 100, device="cuda")
    a, b = B.sample(logits, u, tokens=tokens, probs=probs)
    assert a is tokens and b is probs
    only, none = B.sample(logits, u)
    assert none is None and torch.equal(only, tokens)
    none, only = B.sample(logits, want_probs=True)
    assert none is None and torch.equal(only, probs)
    a, b = B.sample(logits[:0], u[:0], want_probs=True)
    assert a.shape == (0,) and b.shape == (0, 100)


def test_the_largest_vocabulary():
    import torch
    gen = torch.Generator().manual_seed(10)
    logits = (3 * torch.randn(2, 1 << 20, generator=gen)).cuda()
    u = np.array([0.3, 0.97], dtype=np.float32)
    for f in ({}, {"p": np.full(2, 0.95, np.float32)}, {"k": np.full(2, 500000, np.int32)}):
        check(logits, u, f)


@pytest.mark.parametrize("V", [41000, 50001, 98304, 131073])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_cut_and_whole_ones(dtype, V):
    """Batches that are worked on in chunks of either size, and as whole rows, choose alike to the bit, from a
    workspace that holds anything; parts of rows are masked away."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(V)
    N = 110
    logits = (2 * torch.randn(N, V, generator=gen)).to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype]).cuda()
    logits[1, : V // 2] = float("-inf")
    logits[2, V // 3:] = float("nan")
    logits[3] = float("-inf")
    logits[4, 1:] = float("-inf")
    logits[5, [V // 2, V - 1]] = float("inf")
    u = np.random.default_rng(V).random(N).astype(np.float32)
    f = settings(N, V)
    tokens, pr = check(logits, u, f, rows=range(0, N, 9))
    for rows in (80, 12):
        d = B.SampleDims(rows, V, B._dtype_code(logits), V)
        ws = torch.full((B.sample_workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0
        for from_ in (0, N - rows):
            at = slice(from_, from_ + rows)
            some, some_pr = run(logits[at], u[at], want_probs=True, workspace=ws, **{n: v[at] for n, v in f.items()})
            assert (some == tokens[at]).all() and (some_pr == pr[at]).all()
            some, _ = run(logits[at], u[at], workspace=ws, **{n: v[at] for n, v in f.items()})
            assert (some == tokens[at]).all()


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last rows choose as they do alone."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    N, V = 22_000, 100_003
    assert N * V > 2 ** 31
    logits = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    logits[-9:] = (3 * torch.randn(9, V, generator=torch.Generator().manual_seed(15))).to(logits)
    u = torch.rand(N, generator=torch.Generator().manual_seed(16)).cuda()
    p = torch.full((N,), 0.9, device="cuda")
    tokens, _ = B.sample(logits, u, top_p=p)
    alone, probs = B.sample(logits[-9:], u[-9:].clone(), top_p=p[-9:].clone(), want_probs=True)
    assert torch.equal(tokens[-9:], alone)
    assert (probs.gather(1, alone[:, None].long()) > 0).all()
    # rows of equal logits: the kept ones are the first 0.9 V
    assert (tokens[:-9] == (u[:-9].double() * np.ceil(np.float64(np.float32(0.9)) * V)).floor().int()).all()


@pytest.mark.parametrize("N,V", [(3, 60_000), (70, 60_000), (100, 60_000), (3, 1000)])
def test_captured_and_beside_each_other(N, V):
    """Two graphs over the same inputs, replayed on two streams at once between eager calls on new inputs."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(N)
    new = lambda: (2 * torch.randn(N, V, generator=gen)).cuda()
    logits, u = new(), torch.rand(N, generator=gen).cuda()
    k, p = torch.full((N,), 400, dtype=torch.int32).cuda(), torch.full((N,), 0.95).cuda()
    B.sample(logits, u, None, k, p, want_probs=True)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graphs = []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = B.sample(logits, u, None, k, p, want_probs=True)
        graphs.append((g, out))
    for _ in range(4):
        logits.copy_(new())
        u.copy_(torch.rand(N, generator=gen))
        want = B.sample(logits, u, None, k, p, want_probs=True)
        torch.cuda.synchronize()
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("V", [8193, 16385, 32771])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_and_few(dtype, V):
    """Many rows, worked on by smaller workgroups, choose as they do in small batches, to the bit."""
    import torch
    gen = torch.Generator().manual_seed(V)
    N = 520
    logits = (2 * torch.randn(N, V, generator=gen)).to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype]).cuda()
    logits[7, V // 3:] = float("-inf")
    logits[8] = float("nan")
    u = np.random.default_rng(V).random(N).astype(np.float32)
    f = settings(N, V)
    tokens, pr = check(logits, u, f, rows=range(0, N, 37))
    for at in (slice(0, 200), slice(200, 400), slice(400, N)):
        some, some_pr = run(logits[at], u[at], want_probs=True, **{n: v[at] for n, v in f.items()})
        assert (some == tokens[at]).all() and (some_pr == pr[at]).all()
