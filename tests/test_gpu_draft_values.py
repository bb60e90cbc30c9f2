"""Drafted tokens with values that are not finite or whose products overflow: every output and
record against the token-by-token recurrence in 64 bits wherever a value does not reach
it.  Tolerances as in test_gpu_draft.py (the same sums), per row where rows differ in scale."""
import pytest

from tests.layer_refs import f64
from tests import layer_refs as R
from tests.test_gpu_draft import commit, make, near, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_delta_rule_prologue_amd import binding
    binding.lib()


def reference(d, cu, L, S, hist, residual="linear"):
    return R.draft({k: f64(v) for k, v in d.items()}, cu, L, f64(S), f64(hist), residual)


def commit_near(d, cu, cu_t, kept, kw, p, S, hist):
    """The state moved by `kept` tokens, from the records, is finite and the reference's."""
    import torch
    S_out, _ = commit(d, cu_t, kept, kw, p, S, hist, S_out=torch.empty_like(S), k_hist_out=torch.empty_like(hist))
    want, _ = R.commit(f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["b"]), cu, kept, f64(kw), f64(p), f64(S), f64(hist))
    for n in range(len(kept)):
        near(f"S of {n}", S_out[n], want[n], 8e-6)


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("single", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_query_stays_in_its_row(value, single, dtype):
    """A q that is not finite shows in its own row of o: the records (its own token's too) and every
    other output stay, in blocks of 8 and where a later value (`single`) makes a sequence's
    tokens go one at a time; the commit may keep that token."""
    import torch
    d, cu, cu_t, S, hist = make([9, 9, 18], dk=128, dv=64, dtype=dtype, seed=7)
    rows = (5, 18 + 5, 18 + 10)
    for row in rows:
        d["q"][row, 0, 3] = float(value)
    last = cu[-1]
    if single:
        d["v"][18 + 12, 0, 7] = 1e30                     # beyond what a block takes
        last = 18 + 12
    o, kw, p = run(d, cu_t, 4, S, hist)
    ro, rkw, rp, _ = reference(d, cu, 4, S, hist)
    for row in rows:
        assert not torch.isfinite(o[row, 0]).any() and not torch.isfinite(ro[row, 0]).any()
    clean = [t for t in range(last) if t not in rows]
    near("o", o[clean], ro[clean])
    near("o of the other head", o[:, 1], ro[:, 1])
    near("kw", kw[:last], rkw[:last])
    near("p", p[:last], rp[:last])
    commit_near(d, cu, cu_t, [6, 9, 12], kw, p, S, hist)


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("name", ["v", "u"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_write_stays_out_of_its_own_record(name, value, dtype):
    """p of a token is formed from the state before it: its own v and write key, finite or not, are no
    part of it."""
    d, cu, cu_t, S, hist = make([9, 18], dk=64, dv=128, dtype=dtype, seed=17)
    rows = (4, 9 + 12)
    for row in rows:
        d[name][(row, 0, 3) if name == "v" else (row, 0, 1, 3)] = float(value)
    o, kw, p = run(d, cu_t, 4, S, hist)
    ro, rkw, rp, _ = reference(d, cu, 4, S, hist)
    upto = list(range(5)) + list(range(9, 9 + 13))
    near("p", p[upto], rp[upto])
    before = [t for t in upto if t not in rows]
    near("o", o[before], ro[before])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_later_gates_that_overflow(dtype):
    """Each gate is in range, their product over tokens 2..7 is 2^180: tokens before them stay."""
    d, cu, cu_t, S, hist = make([9, 5, 18], dk=64, dv=64, dtype=dtype, seed=21)
    d["g"][2:8, 0] = 2.0 ** 30
    d["g"][14 + 10:14 + 16, 0] = 2.0 ** 30
    o, kw, p = run(d, cu_t, 4, S, hist)
    ro, rkw, rp, _ = reference(d, cu, 4, S, hist)
    near("kw", kw, rkw)
    for first, n in ((0, 2), (9, 5), (14, 10)):
        near("o", o[first:first + n], ro[first:first + n])
        near("p", p[first:first + n], rp[first:first + n])
    near("o of the other head", o[:, 1], ro[:, 1])
    near("p of the other head", p[:, 1], rp[:, 1])
    commit_near(d, cu, cu_t, [2, 5, 10], kw, p, S, hist)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_later_keys_that_overflow_with_the_state(dtype):
    """A state of 1e30 and a later key of 4e8, whose product is beyond fp32: tokens before it stay."""
    d, cu, cu_t, S, hist = make([9, 5, 18], dk=64, dv=64, dtype=dtype, seed=22)
    S *= 3e30
    for row in (6, 14 + 12):
        d["k"][row, 0, 3] = 4e8
    o, kw, p = run(d, cu_t, 4, S, hist)
    ro, rkw, rp, _ = reference(d, cu, 4, S, hist)
    assert (rp[6].abs() > 3.5e38).any()
    for first, n in ((0, 6), (9, 5), (14, 12)):
        near("o", o[first:first + n], ro[first:first + n])
        near("p", p[first:first + n], rp[first:first + n])
    commit_near(d, cu, cu_t, [6, 5, 12], kw, p, S, hist)


@pytest.mark.parametrize("name,value", [("k", 1e25), ("k", -1e38), ("b", float("inf")), ("b", float("nan")), ("b", 1e30),
                                        ("g", float("inf")), ("g", 1e38), ("v", 3e38)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_later_values_beyond_products(name, value, dtype):
    """A value of a later token that is not finite or overflows any product with it, twice in a
    sequence: tokens before the first one stay, and so does the other head."""
    d, cu, cu_t, S, hist = make([8, 9, 20], dk=128, dv=128, dtype=dtype, seed=23)
    for row in (5, 6, 17 + 11, 17 + 14):
        d[name][(row, 0, 3) if d[name].dim() == 3 else (row, 0)] = value
    o, kw, p = run(d, cu_t, 4, S, hist)
    ro, rkw, rp, _ = reference(d, cu, 4, S, hist)
    for first, n in ((0, 5), (8, 9), (17, 11)):
        near("o", o[first:first + n], ro[first:first + n])
        near("p", p[first:first + n], rp[first:first + n])
        near("kw", kw[first:first + n], rkw[first:first + n])
    near("o of the other head", o[:, 1], ro[:, 1])
    near("p of the other head", p[:, 1], rp[:, 1])
    commit_near(d, cu, cu_t, [5, 9, 11], kw, p, S, hist)


@pytest.mark.parametrize("L,residual", [(2, "linear"), (3, "linear"), (4, "linear"), (6, "linear"), (8, "linear"),
                                        (9, "linear"), (12, "linear"), (2, "gelu"), (3, "gelu"), (6, "gelu")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_keys_of_infinite_keys(dtype, L, residual):
    """An infinite k (positive levels and taps) gives the infinities and NaN that the recurrence
    has, in its channel of four tokens: no level beyond the last one takes part.  12 tokens: the
    second pass forms its write keys elsewhere."""
    import torch
    d, cu, cu_t, S, hist = make([12, 3], dk=64, dv=64, L=L, dtype=dtype, seed=31)
    for name in ("u", "conv_w"):
        d[name] = d[name].abs() + 2.0 ** -6
    for row, value in ((2, "inf"), (8, "-inf")):
        d["k"][row, 0, 5] = float(value)
    kw = run(d, cu_t, L, S, hist, residual=residual)[1].cpu().double()
    want = reference(d, cu, L, S, hist, residual)[1]
    assert torch.equal(torch.isnan(kw), torch.isnan(want))
    assert torch.equal(torch.isinf(kw) * torch.sign(kw).nan_to_num(), torch.isinf(want) * torch.sign(want).nan_to_num())
    fine = torch.isfinite(want)
    assert (~fine).sum() == 8
    assert ((kw - want)[fine].abs().max() <= 1e-5 * want[fine].abs().max())
