"""Arguments that the layer operators refuse, before anything is launched: the C
entry points' return codes and the binding's exceptions.  No GPU needed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
FAKE = 0x10000          # aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def B():
    from gated_delta_rule_prologue_amd import binding
    binding.lib()
    return binding


def nd(B, rows=8, heads=1, width=64, dtype=1):
    return ctypes.byref(B.NormDims(rows, heads, width, dtype))


def test_norm_workspace_bytes(B):
    """Per workgroup (one a row or token up to 512 in all, 256 of rows beyond 4096) an fp32 partial: dw and dscale
    of width, or dw of heads rows."""
    up = lambda x: (x + 255) // 256 * 256
    b = lambda *a: B.norm_workspace_bytes(B.NormDims(*a))
    assert b(8, 1, 64, 1) == up(2 * 8 * 64 * 4)
    assert b(100000, 1, 768, 1) == up(2 * 512 * 768 * 4)
    assert b(0, 1, 64, 0) == up(2 * 64 * 4)
    assert b(100000, 1, 8000, 0) == 2 * 256 * 8000 * 4
    assert b(6000, 6, 128, 1) == up(2 * 512 * 128 * 4)         # the residual norm's is larger
    assert b(3 * 5000, 5000, 8, 1) == up(5000 * 8 * 4)
    for bad in ((-1, 1, 64, 1), (8, 0, 64, 1), (8, 3, 64, 1), (8, 1, 0, 1), (8, 1, 64, 2),
                (1 << 61, 1, 64, 1), (1 << 30, 1 << 30, 64, 1)):
        assert b(*bad) == 0, bad


def test_norm_residual_refuses(B):
    f = B.lib().prism_norm_residual

    def call(d=None, x=FAKE, y=FAKE, scale=FAKE, w=FAKE, eps=1e-6, r=FAKE, n=FAKE):
        return f(d if d is not None else nd(B), x, y, scale, w, eps, r, n, None)

    for kw in (dict(x=None), dict(x=FAKE + 2), dict(w=None), dict(n=None), dict(n=FAKE + 8),
               dict(y=FAKE + 4), dict(scale=FAKE + 2), dict(r=FAKE + 8), dict(y=None),       # scale without y
               dict(r=None),                                                                # y without r
               dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**kw) == B.PRISM_EINVAL, kw
    for d in (nd(B, rows=-1), nd(B, width=0), nd(B, dtype=3), nd(B, heads=2)):
        assert call(d) == B.PRISM_EINVAL
    assert f(None, *[FAKE] * 4, 1e-6, FAKE, FAKE, None) == B.PRISM_EINVAL
    assert call(nd(B, width=8193)) == B.PRISM_EUNSUPPORTED


def test_norm_residual_bwd_refuses(B):
    f = B.lib().prism_norm_residual_bwd

    def call(d=None, r=FAKE, y=FAKE, scale=FAKE, w=FAKE, eps=1e-6, dn=FAKE, dr=None, dx=FAKE, dy=FAKE,
             dw=FAKE, ds=FAKE, ws=FAKE, nb=1 << 30):
        return f(d if d is not None else nd(B), r, y, scale, w, eps, dn, dr, dx, dy, dw, ds, ws, nb, None)

    for kw in (dict(r=None), dict(w=None), dict(dn=None), dict(dx=None), dict(dw=None), dict(ws=None),
               dict(nb=16), dict(y=None), dict(scale=None), dict(dr=FAKE + 2), dict(dy=FAKE + 2),
               dict(ds=FAKE + 4), dict(eps=-1.0)):
        assert call(**kw) == B.PRISM_EINVAL, kw
    assert call(nd(B, heads=2)) == B.PRISM_EINVAL
    assert call(nd(B, width=9000)) == B.PRISM_EUNSUPPORTED


def test_norm_gate_refuses(B):
    fwd, bwd = B.lib().prism_norm_gate, B.lib().prism_norm_gate_bwd

    def call(d=None, o=FAKE, z=FAKE, w=FAKE, eps=1e-6, gate=0, y=FAKE):
        return fwd(d if d is not None else nd(B), o, z, w, eps, gate, y, None)

    def grad(d=None, o=FAKE, z=FAKE, w=FAKE, eps=1e-6, gate=1, dy=FAKE, do=FAKE, dz=FAKE, dw=FAKE, ws=FAKE,
             nb=1 << 30):
        return bwd(d if d is not None else nd(B), o, z, w, eps, gate, dy, do, dz, dw, ws, nb, None)

    for kw in (dict(o=None), dict(z=None), dict(w=None), dict(y=None), dict(z=FAKE + 2), dict(gate=2),
               dict(gate=-1), dict(eps=-1.0)):
        assert call(**kw) == B.PRISM_EINVAL, kw
    for kw in (dict(o=None), dict(dy=None), dict(do=None), dict(dz=None), dict(dw=None), dict(ws=None),
               dict(nb=16), dict(gate=2)):
        assert grad(**kw) == B.PRISM_EINVAL, kw
    for d in (nd(B, rows=7, heads=2), nd(B, heads=0), nd(B, width=0)):
        assert call(d) == B.PRISM_EINVAL and grad(d) == B.PRISM_EINVAL
    assert call(nd(B, width=1025)) == B.PRISM_EUNSUPPORTED
    assert grad(nd(B, width=1025)) == B.PRISM_EUNSUPPORTED


def test_decode_draft_refuses(B):
    f = B.lib().prism_decode_draft
    names = ["q", "k", "v", "u", "g", "b", "a", "h", "conv_w", "cu"]
    outs = ["S", "hist", "o", "kw", "p"]

    def call(d=None, L=3, residual=0, **over):
        a = {n: FAKE for n in names + outs}
        a.update(over)
        return f(ctypes.byref(d or B.make_dims(4, 12, 2, 64, 64, 1)), *(a[n] for n in names), L, residual,
                 *(a[n] for n in outs), None)

    for n in names + outs:
        assert call(**{n: None}) == B.PRISM_EINVAL, n
        assert call(**{n: FAKE + 2}) == B.PRISM_EINVAL, n
    for kw in (dict(L=0), dict(L=17), dict(residual=2), dict(residual=-1)):
        assert call(**kw) == B.PRISM_EINVAL, kw
    assert call(B.make_dims(0, 12, 2, 64, 64, 1)) == B.PRISM_EINVAL
    assert call(B.make_dims(4, -1, 2, 64, 64, 1)) == B.PRISM_EINVAL
    assert call(B.make_dims(4, 12, 2, 96, 64, 1)) == B.PRISM_EUNSUPPORTED
    assert call(B.make_dims(4, 12, 2, 64, 256, 0)) == B.PRISM_EUNSUPPORTED
    assert call(B.make_dims(1 << 20, 12, 1 << 20, 64, 64, 0)) == B.PRISM_EUNSUPPORTED
    # no tokens: nothing to do, and nothing is launched
    none = {n: None for n in ("q", "k", "v", "u", "g", "b", "a", "h", "o", "kw", "p")}
    assert call(B.make_dims(4, 0, 2, 64, 64, 1), **none) == B.PRISM_OK


def test_decode_commit_refuses(B):
    f = B.lib().prism_decode_commit
    names = ["k", "v", "g", "b", "cu", "n_accept", "kw", "p", "S", "hist", "S_out", "hist_out"]

    def call(d=None, **over):
        a = {n: FAKE for n in names}
        a.update(over)
        return f(ctypes.byref(d or B.make_dims(4, 12, 2, 64, 64, 1)), *(a[n] for n in names), None)

    for n in names:
        assert call(**{n: None}) == B.PRISM_EINVAL, n
        assert call(**{n: FAKE + 4}) == B.PRISM_EINVAL, n
    assert call(B.make_dims(4, 12, 2, 64, 32, 1)) == B.PRISM_EUNSUPPORTED
    assert call(B.make_dims(4, 12, 0, 64, 64, 1)) == B.PRISM_EINVAL


def test_verify_refuses(B):
    f = B.lib().prism_verify_draft
    names = ["p", "q", "tokens", "cu", "u_accept", "u_sample", "n_accept", "next", "ws"]

    def call(d=(4, 12, 100000, 0), nb=1 << 30, **over):
        a = {n: FAKE for n in names}
        a.update(over)
        return f(ctypes.byref(B.VerifyDims(*d)), *(a[n] for n in names), nb, None)

    for n in names:
        if n != "q":
            assert call(**{n: None}) == B.PRISM_EINVAL, n
        assert call(**{n: FAKE + 4}) == B.PRISM_EINVAL, n
    assert call(nb=16) == B.PRISM_EINVAL
    for d in ((0, 12, 100000, 0), (4, -1, 100000, 0), (4, 12, 0, 0), (4, 12, 100000, 2)):
        assert call(d) == B.PRISM_EINVAL, d
        assert B.verify_workspace_bytes(B.VerifyDims(*d)) == 0
    assert call((1, 1, (1 << 28) + 1, 0)) == B.PRISM_EUNSUPPORTED
    # two fp64 sums per 4096 entries (and up to 7 for the row's offset) beyond 32,768 entries
    assert B.verify_workspace_bytes(B.VerifyDims(3, 9, 32768, 0)) == 0
    assert B.verify_workspace_bytes(B.VerifyDims(3, 9, 32769, 0)) == 3 * 9 * 16 // 256 * 256 + 256
    assert B.verify_workspace_bytes(B.VerifyDims(64, 99, 128000, 1)) == 64 * 32 * 16


def far(count):
    """Addresses that no two arrays of these sizes reach from one to the other."""
    return [FAKE + (i + 1 << 32) for i in range(count)]


def test_outputs_that_overlap_are_refused(B):
    """An output on an input, another output or the workspace: refused wherever it begins, but for
    whole buffers that may be both.  Every call here is refused (a call with nothing wrong would
    launch)."""
    L = B.lib()
    row, t = 64 * 2, 8 * 64 * 2                              # bytes of a row and of a tensor

    names = ["x", "y", "scale", "w", "r", "n"]
    at = dict(zip(names, far(6)))

    def norm(**over):
        a = {**at, **over}
        return L.prism_norm_residual(nd(B), a["x"], a["y"], a["scale"], a["w"], 1e-6, a["r"], a["n"], None)

    for over in (dict(r=at["n"]), dict(r=at["x"] + row), dict(n=at["y"] + t - 16), dict(n=at["x"] - t + 16),
                 dict(r=at["w"]), dict(n=at["scale"] - 16), dict(r=at["n"] + t - row)):
        assert norm(**over) == B.PRISM_EINVAL, over

    names = ["r", "y", "scale", "w", "dn", "dr", "dx", "dy", "dw", "ds", "ws"]
    at = dict(zip(names, far(11)))
    for over in (dict(dx=at["dy"]), dict(dx=at["dn"] + row), dict(dy=at["w"]), dict(dw=at["ds"]), dict(dw=at["w"]),
                 dict(ds=at["r"]), dict(ws=at["dn"]), dict(ws=at["dx"] + row), dict(dw=at["ws"] + 256)):
        a = {**at, **over}
        assert L.prism_norm_residual_bwd(nd(B), a["r"], a["y"], a["scale"], a["w"], 1e-6, a["dn"], a["dr"], a["dx"],
                                         a["dy"], a["dw"], a["ds"], a["ws"], 1 << 30, None) == B.PRISM_EINVAL, over

    names = ["o", "z", "w", "dy", "do", "dz", "dw", "ws"]
    at = dict(zip(names, far(8)))
    for over in (dict(do=at["dz"]), dict(do=at["o"] + row), dict(dz=at["w"]), dict(dw=at["dy"]), dict(ws=at["do"])):
        a = {**at, **over}
        assert L.prism_norm_gate_bwd(nd(B, heads=2), a["o"], a["z"], a["w"], 1e-6, 0, a["dy"], a["do"], a["dz"], a["dw"],
                                     a["ws"], 1 << 30, None) == B.PRISM_EINVAL, over
    for over in (at["o"] + row, at["z"] - 16, at["w"]):
        assert L.prism_norm_gate(nd(B), at["o"], at["z"], at["w"], 1e-6, 0, over, None) == B.PRISM_EINVAL

    dims = ctypes.byref(B.make_dims(4, 12, 2, 64, 64, 0))
    names = ["q", "k", "v", "u", "g", "b", "a", "h", "conv_w", "cu"]
    outs = ["S", "hist", "o", "kw", "p"]
    at = dict(zip(names + outs, far(15)))
    for out in ("o", "kw", "p"):
        for other in names + outs:
            if other != out:
                a = {**at, out: at[other]}
                assert L.prism_decode_draft(dims, *(a[n] for n in names), 3, 0, *(a[n] for n in outs),
                                            None) == B.PRISM_EINVAL, (out, other)

    names = ["k", "v", "g", "b", "cu", "n_accept", "kw", "p", "S", "hist", "S_out", "hist_out"]
    at = dict(zip(names, far(12)))
    for out in ("S_out", "hist_out"):
        for other in names:
            if other != out:
                same = other == out[:-4]                     # the whole buffer may be both, a part of it not
                a = {**at, out: at[other] + (16 if same else 0)}
                assert L.prism_decode_commit(dims, *(a[n] for n in names), None) == B.PRISM_EINVAL, (out, other)

    names = ["p", "q", "tokens", "cu", "u_accept", "u_sample", "n_accept", "next", "ws"]
    at = dict(zip(names, far(9)))
    for out in ("n_accept", "next", "ws"):
        for other in names:
            if other != out:
                a = {**at, out: at[other]}
                assert L.prism_verify_draft(ctypes.byref(B.VerifyDims(4, 12, 100000, 0)), *(a[n] for n in names),
                                            1 << 30, None) == B.PRISM_EINVAL, (out, other)


def test_grids_beyond_a_launch_are_refused(B):
    """Chains, sequences and heads that one launch cannot hold (2^32 threads)."""
    at = far(15)
    L = B.lib()
    for n, H, dv in ((1 << 20, 16, 128), (1 << 20, 32, 64)):
        d = ctypes.byref(B.make_dims(n, 12, H, 64, dv, 1))
        assert L.prism_decode_draft(d, *at[:10], 3, 0, *at[10:], None) == B.PRISM_EUNSUPPORTED
        assert L.prism_decode_commit(d, *at[:12], None) == B.PRISM_EUNSUPPORTED
    for n, vocab in ((1 << 22, 1000), (1 << 19, 40000)):
        assert L.prism_verify_draft(ctypes.byref(B.VerifyDims(n, 12, vocab, 0)), *at[:9], 1 << 40,
                                    None) == B.PRISM_EUNSUPPORTED
    d = nd(B, rows=65536, heads=65536, width=8)
    assert L.prism_norm_gate(d, *at[:3], 1e-6, 0, at[3], None) == B.PRISM_EUNSUPPORTED
    assert L.prism_norm_gate_bwd(d, *at[:3], 1e-6, 0, *at[3:8], 1 << 40, None) == B.PRISM_EUNSUPPORTED


def test_drafts_longer_than_served_are_refused(B):
    f = B.lib().prism_decode_draft
    at = far(15)
    assert f(ctypes.byref(B.make_dims(3, 3 * 1024 + 1, 2, 64, 64, 1)), *at[:10], 3, 0, *at[10:],
             None) == B.PRISM_EUNSUPPORTED


def test_binding_refuses_before_calling(B):
    """What the binding refuses by itself: host tensors, and the arguments it looks at
    before any address."""
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    with pytest.raises(ValueError, match="device"):
        B.norm_residual(x, w)
    with pytest.raises(ValueError, match="heads"):
        B.norm_gate(torch.zeros(4, 3, 64, dtype=bf), torch.zeros(4, 3, 64, dtype=bf), torch.zeros(2, 64, dtype=bf))
    with pytest.raises(ValueError, match="gate"):
        B.norm_gate(x, x, w, gate="tanh")
    with pytest.raises(ValueError, match="scale without y"):
        B.norm_residual(x, w, scale=w)
    with pytest.raises(ValueError, match="scale without y"):
        B.norm_residual_bwd(x, w, x, scale=w)
    with pytest.raises(ValueError, match="same buffer"):
        B.norm_residual(x, w, y=x.clone(), r=(r := torch.zeros_like(x)), n=r)
    with pytest.raises(TypeError, match="unsupported dtype"):
        B.norm_residual(x.half(), w)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    q, v = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, 2, 128, dtype=bf)
    th, cw = torch.zeros(4, 2, dtype=bf), torch.zeros(2, 64, 4, dtype=bf)
    S, hist = torch.zeros(1, 2, 64, 128), torch.zeros(1, 2, 3, 64, dtype=bf)
    with pytest.raises(ValueError, match="residual"):
        B.decode_draft(q, q, v, None, th, th, None, None, cw, cu, 1, S, hist, residual="relu")
    with pytest.raises(ValueError, match="L must"):
        B.decode_draft(q, q, v, None, th, th, None, None, cw, cu, 17, S, hist)
    with pytest.raises(ValueError, match="cu_seqlens"):
        B.decode_commit(q, v, th, th, cu.long(), cu[:1], S, S, S, hist)
    p = torch.zeros(4, 10)
    with pytest.raises(ValueError, match="p must be"):
        B.verify_draft(p[0], cu, cu, p[:, 0], p[0, :1])
    with pytest.raises(ValueError, match="same buffer"):
        B.verify_draft(p, cu, cu, p[:, 0], p[0, :1], n_accept=(m := torch.zeros(1, dtype=torch.int32)), next_token=m)
