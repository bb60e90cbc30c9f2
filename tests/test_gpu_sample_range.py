"""The choice of a token (prism_sample) from rows whose logits lie too far apart for an fp32 difference, or nearer
together than fp32 can invert, against a sort in 64 bits.

Tokens have to be the reference's, and inside the vocabulary.  Probabilities are rounded once to fp32 (2^-24),
after weights of 10^-12 and a total that is off by at most 2^-44 an entry over at least one; what is below
fp32's normal numbers, 2^-126."""
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


def check(rows, u, name, **f):
    """Rows [N, V] (fp32 or bf16 values) with settings, one for all or one each: tokens and distributions."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    N, V = rows.shape
    f = {n: np.broadcast_to(np.asarray(v, dtype=np.int32 if n == "k" else np.float32), (N,)).copy() for n, v in f.items()}
    args = [torch.from_numpy(f[n]).cuda() if n in f else None for n in "tkpm"]
    u = np.asarray(u, dtype=np.float32)
    tokens, probs = B.sample(rows.cuda(), torch.from_numpy(u).cuda(), *args, want_probs=True)
    _, alone = B.sample(rows.cuda(), None, *args, want_probs=True)           # no draw: fewer places are looked up
    tokens, probs, alone = tokens.cpu().numpy(), probs.cpu().numpy(), alone.cpu().numpy()
    l = rows.double().numpy()
    for n in range(N):
        one = {a: v[n].item() for a, v in f.items()}
        at = (name, V, n, one, u[n])
        assert tokens[n] == R.sample(l[n], float(u[n]), **one), (at, tokens[n])
        ref = R.probs(l[n], **one)
        for got in (probs[n], alone[n]):
            assert (np.abs(got - ref) <= 2.0 ** -23 * ref + 2.0 ** -126).all(), at


def spread(V, values, seed):
    """[1, V] of the values: each once, the last but one everywhere else, in any order."""
    import torch
    rng = np.random.default_rng(seed)
    row = np.full(V, values[-2], dtype=np.float32)
    row[rng.permutation(V)[:len(values)]] = np.asarray(values, dtype=np.float32)
    return torch.from_numpy(row)[None]


@pytest.mark.parametrize("V", [60, 3000, 20000, 70001])
def test_draws_among_entries_far_below_an_overflowing_maximum(V):
    """1e38 beside many 8.3e37 at a temperature of 1e36, where they weigh e^-17 each, and one entry so low
    that the difference overflows: a draw behind the largest finds one of them."""
    row = spread(V, [1e38, 8.3e37, -3e38], V)
    rest = (V - 2) * np.exp(-17.0)
    total = 1 + rest
    for share in (0.1, 0.5, 0.9):
        u = (1 + share * rest) / total
        if np.float32(u) < 1:
            check(row, [u], "far", t=1e36)
    check(row, [0.5], "far", t=1e36)


@pytest.mark.parametrize("V", [5, 3000, 70001])
def test_counts_among_entries_far_below_an_overflowing_maximum(V):
    for top in (1e37, 1e32, 2e31):
        values = [top, 2.0, 1.0, 0.0, LOWEST]
        for k in (2, 3, 4):
            check(spread(V, values, V + k), [0.3], "few", k=k)


@pytest.mark.parametrize("V", [60, 3000, 70001])
def test_min_p_among_entries_far_below_an_overflowing_maximum(V):
    """min_p ends among the entries of 8.3e37, some of which lie beside the maximum: their weight counts."""
    for near in (9.99999e37, 9e37):
        row = spread(V, [1e38, near, 8.3e37, -3e38], V)
        for m in (1e-7, 3e-8, 1e-8):                          # above and below e^-17
            for u in (0.4, 0.8):
                check(row, [u], "least", t=1e36, m=m)


def any_rows(N, V, rng):
    """Rows of every magnitude that fp32 holds: of one sign or both, a row's all alike or not, with a lowest value."""
    biggest = np.finfo(np.float32).max
    out = np.empty((N, V))
    for n in range(N):
        kind = n % 4
        if kind == 0:
            out[n] = rng.choice([-1, 1], V) * 10.0 ** rng.uniform(-45, 38.5, V)
        elif kind == 1:
            out[n] = rng.standard_normal(V) * 10.0 ** rng.uniform(-44, 38)
        elif kind == 2:
            out[n] = 10.0 ** rng.uniform(-10, 38) * (1 + rng.standard_normal(V) * 10.0 ** rng.uniform(-8, 0))
            if rng.random() < 0.5:
                out[n, V // 2] = -biggest
        else:
            out[n] = rng.standard_normal(V) * 10.0 ** rng.uniform(-3, 3)
            out[n, [V // 3, V // 2]] = 10.0 ** rng.uniform(25, 38.5), -biggest
    return np.clip(out, -biggest, biggest).astype(np.float32)


@pytest.mark.parametrize("filters", ["", "k", "p", "m", "kpm"])
@pytest.mark.parametrize("V,N", [(60, 400), (2500, 40), (70001, 12)])
def test_rows_of_any_magnitude(V, N, filters):
    """Temperatures from the smallest number to the largest beside logits of all magnitudes."""
    import torch
    rng = np.random.default_rng(V + len(filters))
    for dt in (torch.float32, torch.bfloat16):
        rows = torch.from_numpy(any_rows(N, V, rng))
        if dt == torch.bfloat16:
            rows = torch.clamp(rows, -3.3e38, 3.3e38).to(dt)
        t = np.where(rng.random(N) < 0.6, 10.0 ** rng.uniform(-44.8, 38.4, N), 10.0 ** rng.uniform(-1, 1, N))
        f = {"t": t, "k": rng.integers(1, V // 2, N), "p": rng.uniform(0.05, 0.999, N), "m": 10.0 ** rng.uniform(-9, 0, N)}
        check(rows, rng.random(N).astype(np.float32), f"any {dt}", **{n: f[n] for n in "t" + filters})


def test_rows_nearer_than_fp32_inverts():
    """Differences of 1e-37 and of fp32's smallest numbers, alone and with temperatures as small."""
    import torch
    tiny = 2.0 ** -149
    for values in ([1e-37, 0.0], [0.0, -1e-37, -2e-37], [3 * tiny, tiny, 0.0], [1e-38, 1.1e-38, 0.9e-38, -1e-38], [tiny, 0.0]):
        row = torch.tensor([values], dtype=torch.float64).float()
        for u in (0.05, 0.45, 0.7, 0.95):
            for t in (1.0, 1e-37, 1e-38, tiny):
                check(row, [u], "near", t=t)
                check(row, [u], "near", t=t, k=2)
                check(row, [u], "near", t=t, p=0.6)
                check(row, [u], "near", t=t, m=0.3)
