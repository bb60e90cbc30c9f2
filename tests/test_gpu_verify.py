"""prism_verify_draft against a sequential 64-bit reference: whole numbers, so every value
has to be equal.  Sums of up to 10^5 weights in 64 bits differ by 1e-13 between orders, so a
threshold would have to be drawn that near a border to tell them apart."""
import numpy as np
import pytest

from tests.gpu_common import say
from tests import layer_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def make(lens, V, dtype="f32", seed=0, near=0.7):
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    gen = torch.Generator().manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(int).tolist()
    T = cu[-1]
    logits = 2 * torch.randn(T, V, generator=gen)
    p = torch.softmax(logits, -1).to(dt)
    q = torch.softmax(logits + near * torch.randn(T, V, generator=gen), -1).to(dt)
    tokens = torch.zeros(T, dtype=torch.int32)
    if T > 1:
        tokens[1:] = torch.multinomial(q[:-1].float(), 1, generator=gen)[:, 0].int()
    return {"p": p, "q": q, "tokens": tokens, "cu": cu, "u_accept": torch.rand(T, generator=gen),
            "u_sample": torch.rand(len(lens), generator=gen)}


def both(m, use_q=True):
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    cu_t = torch.tensor(m["cu"], dtype=torch.int32)
    q = m["q"].cuda() if use_q else None
    n, t = B.verify_draft(m["p"].cuda(), m["tokens"].cuda(), cu_t.cuda(), m["u_accept"].cuda(), m["u_sample"].cuda(),
                          q=q)
    assert n.dtype == t.dtype == torch.int32
    ref = R.verify(m["p"].double().numpy(), m["q"].double().numpy() if use_q else None, m["tokens"].numpy(), m["cu"],
                   m["u_accept"].numpy(), m["u_sample"].numpy())
    assert n.cpu().tolist() == ref[0], (n.cpu().tolist(), ref[0])
    assert t.cpu().tolist() == ref[1], (t.cpu().tolist(), ref[1])
    return ref


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("use_q", [True, False])
@pytest.mark.parametrize("V", [1, 2, 5, 8, 255, 1000, 1023, 1025, 4095, 4096, 4097, 8200, 32768, 32769, 36857, 36860, 36864,
                               50001])
def test_vocabularies(dtype, use_q, V):
    m = make([5, 1, 0, 3, 6, 2, 9, 4], V, dtype, seed=V)
    kept, nxt = both(m, use_q)
    say(f"V={V} {dtype} q={use_q}: kept {kept} next {nxt}")


def test_more_chunks_than_lanes():
    """A vocabulary of more than 64 chunks of 4096."""
    m = make([3, 2], 64 * 4096 + 1500, seed=3)
    both(m)
    m["u_sample"][:] = 0.9999999
    both(m)


def test_long_drafts():
    """More drafted tokens than a wavefront tests at once; all kept, and a rejection at each end
    of the groups of 64."""
    import torch
    m = make([200, 66, 1, 130, 65, 64], 50, seed=4)
    m["q"] = m["p"].clone()
    m["u_accept"][:] = 0.5                               # u q < p always holds
    kept, _ = both(m)
    assert kept == [200, 66, 1, 130, 65, 64]
    for at in (1, 63, 64, 65, 128, 129, 199):
        tok = m["tokens"].clone()
        m["tokens"][at] = -1
        kept, _ = both(m)
        assert kept[0] == at
        m["tokens"] = tok


def test_tokens_outside_the_vocabulary():
    m = make([4, 4, 4], 33, seed=5)
    m["u_accept"][:] = 0.0
    m["tokens"][1], m["tokens"][6], m["tokens"][11] = 33, -7, 2 ** 31 - 1
    for use_q in (True, False):
        kept, _ = both(m, use_q)
        assert kept == [1, 2, 3]


def test_rows_without_weight():
    """Zero rows, equal distributions after a rejection, NaN, infinities and negative entries."""
    import torch
    m = make([2, 2, 2, 2, 1, 2, 1], 300, seed=6)
    p, q = m["p"], m["q"]
    m["u_accept"][:] = 0.999999
    m["tokens"][1::2] = 7
    p[0] = 0.0                                           # no probability at all: -1
    q[2] = p[2]
    q[2, 7] = p[2, 7] * 1.5                              # rejected, and max(p - q, 0) is empty: p
    p[4, 10:200] = float("nan")
    q[4, 7], p[4, 7] = 0.9, 0.1
    p[6, 3], p[6, 5], q[6, 9] = float("inf"), -1.0, float("nan")
    q[6, 7], p[6, 7] = 0.9, 0.1
    p[8] = 0.0
    p[8, 299] = 1e-30                                    # one weight, the last
    p[9] = float("nan")
    p[9, 17] = 0.25
    q[9] = 0.0
    for s in (0.0, 0.3, 0.99999994):
        m["u_sample"][:] = s
        kept, nxt = both(m)
        assert nxt[0] == -1 and nxt[4] == 299
        both(m, use_q=False)


def test_random_numbers_at_the_ends():
    """u_sample of 0, the last value below 1, and outside: the first and the last weight."""
    import torch
    m = make([3, 3, 1, 1], 5000, seed=7)
    m["p"][:, :40] = 0.0
    m["p"][:, -3:] = 0.0
    for s in (0.0, float(np.nextafter(np.float32(1), np.float32(0))), 1.0, 2.0, -1.0, float("nan")):
        m["u_sample"][:] = s
        kept, nxt = both(m, use_q=False)
        assert all(40 <= t < 4997 for t in nxt)
        both(m)


def test_greedy_target():
    """One-hot target rows (greedy decoding): drafts are kept while they are the argmax."""
    import torch
    m = make([5] * 20, 1000, seed=8)
    best = m["p"].argmax(1)
    m["p"] = torch.nn.functional.one_hot(best, 1000).float()
    m["tokens"][1:] = torch.where(torch.rand(99) < 0.7, best[:-1].int(), m["tokens"][1:])
    kept, nxt = both(m, use_q=False)
    for n in range(20):
        assert nxt[n] == best[5 * n + kept[n] - 1]


def test_many_sequences():
    """More sequences than one grid dimension of 65,536."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    N = 70000
    p = torch.tensor([[0.25, 0.75]]).repeat(N, 1).cuda()
    cu = torch.arange(N + 1, dtype=torch.int32).cuda()
    s = (torch.arange(N) % 2).float().cuda() * 0.5
    n, t = B.verify_draft(p, torch.zeros(N, dtype=torch.int32).cuda(), cu, torch.zeros(N).cuda(), s)
    assert (n == 1).all() and torch.equal(t.cpu(), (torch.arange(N) % 2).int())


def test_the_drawn_tokens_follow_the_target():
    """The kept tokens and the next one together are distributed as the target's: the first
    token after the prefix over 40,000 independent sequences, against p within 6 standard
    deviations of a count (a probability of 2e-9 an entry)."""
    import torch
    from gated_delta_rule_prologue_amd import binding as B
    gen = torch.Generator().manual_seed(12)
    N, V = 40000, 12
    p1, q1 = torch.softmax(torch.randn(V, generator=gen), 0), torch.softmax(torch.randn(V, generator=gen), 0)
    draft = torch.multinomial(q1, N, replacement=True, generator=gen).int()
    tokens = torch.stack([torch.zeros(N, dtype=torch.int32), draft], 1).reshape(-1)
    p, q = p1.repeat(2 * N, 1), q1.repeat(2 * N, 1)
    cu = torch.arange(0, 2 * N + 1, 2, dtype=torch.int32)
    n, t = B.verify_draft(p.cuda(), tokens.cuda(), cu.cuda(), torch.rand(2 * N, generator=gen).cuda(),
                          torch.rand(N, generator=gen).cuda(), q=q.cuda())
    first = torch.where(n.cpu() == 2, draft, t.cpu())
    count = torch.bincount(first, minlength=V).double()
    want = p1.double() * N
    assert ((count - want).abs() <= 6 * torch.sqrt(want * (1 - p1.double()))).all(), (count, want)
