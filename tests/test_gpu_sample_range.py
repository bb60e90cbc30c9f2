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
    """Rows [N, V] (fp32 or bf16 values) with one set of settings: tokens and distributions."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    N, V = rows.shape
    each = {n: None if v is None else torch.full((N,), v, dtype=torch.int32 if n == "k" else torch.float32).cuda()
            for n, v in {"t": None, "k": None, "p": None, "m": None, **f}.items()}
    args = (each["t"], each["k"], each["p"], each["m"])
    tokens, probs = B.sample(rows.cuda(), torch.tensor(u, dtype=torch.float32).cuda(), *args, want_probs=True)
    _, alone = B.sample(rows.cuda(), None, *args, want_probs=True)           # no draw: fewer places are looked up
    tokens, probs, alone = tokens.cpu().numpy(), probs.cpu().numpy(), alone.cpu().numpy()
    l = rows.double().numpy()
    f = {n: int(v) if n == "k" else float(np.float32(v)) for n, v in f.items()}
    for n in range(N):
        at = (name, V, n, f, u[n])
        assert tokens[n] == R.sample(l[n], float(np.float32(u[n])), **f), (at, tokens[n])
        ref = R.probs(l[n], **f)
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
