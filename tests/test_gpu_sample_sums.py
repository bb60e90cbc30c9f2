"""How near the sums of sampled weights are to exact ones (prism_sample), where entries are alike and round alike.

A weight is off by half a step of 2^-43 of the largest, so a sum over V entries by V 2^-44 at most, and the goal of a
draw or of top_p, a share of such a sum, by as much.  A choice's place is therefore within V 2^-43 of where
exact sums have it (and 10^-11 of the total for the weights' own series and this test's sums)."""
import numpy as np
import pytest

from tests.gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


@pytest.mark.parametrize("V", [1000, 32_000, 128_000, 1 << 20])
@pytest.mark.parametrize("below", [3.0, 20.3, 28.7, 29.41, 29.9, 30.4, 31.0])
def test_one_entry_above_equal_ones(V, below):
    """One weight of 1 at index 0 and V - 1 equal ones behind it."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    row = torch.full((1, V), -below)
    row[0, 0] = 0
    w = np.exp(np.float64(row[0, 1].item()))
    total = 1 + (V - 1) * w
    off = V * 2.0 ** -43 + 1e-11 * total
    shares = [1 - 2.0 ** -24, 1 - 2.0 ** -20, 0.99, 0.6, 0.5]
    u = torch.tensor(shares, dtype=torch.float32).cuda()
    logits = row.expand(len(shares), -1).cuda()
    tokens, _ = B.sample(logits, u)
    # `u`: a share of the weight; the token is the first at which the running weight exceeds it
    worst = 0.0
    for goal, token in zip(u.double().cpu().numpy() * total, tokens.cpu().numpy()):
        assert 0 <= token < V
        before, upto = (0.0, 1.0) if token == 0 else (1 + (token - 1) * w, 1 + token * w)
        far = max(before - goal, goal - upto, 0.0)
        worst = max(worst, far / off)
        assert far <= off, (goal, token, far)
    p = torch.full((1,), 1 - 2.0 ** -24).cuda()
    _, probs = B.sample(logits[:1], None, top_p=p, want_probs=True)
    n = int((probs > 0).sum())                               # the entries before which less than p has passed
    goal = (1 - 2.0 ** -24) * total
    last = (0.0, 1.0) if n == 1 else (1 + (n - 2) * w, 1 + (n - 1) * w)
    far = max(last[0] - goal, goal - last[1], 0.0)
    assert far <= off, (n, far)
    say(f"sample, {V} entries, {below} below: worst share of the bound {max(worst, far / off):.2f}")
