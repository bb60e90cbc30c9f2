"""Arguments that the short convolution, the norm and rotation of queries and keys, and the choice of a
token refuse, before anything is launched: the C entry points' return codes and the binding's
exceptions.  No GPU needed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
FAKE = 0x10000          # aligned, never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def B():
    from gated_delta_rule_prologue_amd import binding
    binding.lib()
    return binding


def far(count):
    """Addresses that no two arrays of these sizes reach from one to the other."""
    return [FAKE + (i + 1 << 34) for i in range(count)]


CONV = ["x", "w", "bias", "hist", "cu", "y", "hist_out"]


def conv(B, d=None, act=1, **over):
    a = {**dict(zip(CONV, far(7))), **over}
    return B.lib().prism_short_conv(ctypes.byref(d or B.ConvDims(4, 20, 64, 4, 1, 64)), a["x"], a["w"], a["bias"],
                                    a["hist"], a["cu"], act, a["y"], a["hist_out"], None)


def step(B, d=None, act=1, **over):
    a = {**dict(zip(CONV, far(7))), **over}
    return B.lib().prism_short_conv_step(ctypes.byref(d or B.ConvDims(4, 4, 64, 4, 1, 64)), a["x"], a["w"], a["bias"],
                                         a["hist"], act, a["y"], a["hist_out"], None)


GRAD = ["x", "w", "bias", "hist", "cu", "dy", "dx", "dw", "db", "dh", "ws"]


def grad(B, d=None, act=1, nb=1 << 30, **over):
    a = {**dict(zip(GRAD, far(11))), **over}
    return B.lib().prism_short_conv_bwd(ctypes.byref(d or B.ConvDims(4, 20, 64, 4, 1, 64)), a["x"], a["w"], a["bias"],
                                        a["hist"], a["cu"], act, a["dy"], a["dx"], a["dw"], a["db"], a["dh"], a["ws"],
                                        nb, None)


def test_conv_refuses(B):
    bad = [B.ConvDims(*v) for v in ((0, 20, 64, 4, 1, 64), (4, -1, 64, 4, 1, 64), (4, 20, 0, 4, 1, 64),
                                    (4, 20, 64, 0, 1, 64), (4, 20, 64, 9, 1, 64), (4, 20, 64, 4, 2, 64),
                                    (4, 20, 64, 4, 1, -64), (4, 20, 64, 4, 1, 1 << 62))]
    for call in (conv, grad):
        for d in bad:
            assert call(B, d) == B.PRISM_EINVAL
        for name in ("x", "w", "cu"):
            assert call(B, **{name: None}) == B.PRISM_EINVAL, name
        for name in ("w", "bias", "hist", "cu"):
            assert call(B, **{name: far(1)[0] + 2}) == B.PRISM_EINVAL, name
        assert call(B, x=far(1)[0] + 1) == B.PRISM_EINVAL            # an odd address
        assert call(B, act=2) == B.PRISM_EINVAL and call(B, act=-1) == B.PRISM_EINVAL
        assert call(B, B.ConvDims(4, 20, (1 << 22) + 1, 4, 1, 1 << 23)) == B.PRISM_EUNSUPPORTED
    for kw in (dict(y=None), dict(y=FAKE + 2), dict(hist_out=FAKE + 8)):
        assert conv(B, **kw) == B.PRISM_EINVAL, kw
    for kw in (dict(dy=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(nb=16), dict(dh=FAKE + 2),
               dict(db=FAKE + 4), dict(dx=FAKE + 2)):
        assert grad(B, **kw) == B.PRISM_EINVAL, kw
    L = B.lib()
    assert L.prism_short_conv(None, *far(5), 1, *far(2), None) == B.PRISM_EINVAL
    assert all(B.conv_workspace_bytes(d) == 0 for d in bad)
    for call in (conv, grad):
        many = dict(zip(CONV if call is conv else GRAD, [FAKE + (i << 48) for i in range(11)]))
        assert call(B, B.ConvDims(4, (1 << 30) + 1, 1, 4, 1, 1), **many) == B.PRISM_EUNSUPPORTED
    # a launch holds 2^32 threads: a billion tokens of 2^15 channels are more
    assert conv(B, B.ConvDims(4, 1 << 30, 1 << 15, 4, 1, 1 << 15), **dict(zip(CONV, [FAKE + (i << 48) for i in range(7)]))) \
        == B.PRISM_EUNSUPPORTED


def test_conv_step_refuses(B):
    for d in (B.ConvDims(4, 5, 64, 4, 1, 64), B.ConvDims(0, 0, 64, 4, 1, 64)):
        assert step(B, d) == B.PRISM_EINVAL
    for name in ("x", "w", "hist", "y", "hist_out"):
        assert step(B, **{name: None}) == B.PRISM_EINVAL, name
    assert step(B, act=5) == B.PRISM_EINVAL
    assert step(B, y=far(1)[0]) == B.PRISM_EINVAL                    # y on x


def test_conv_overlaps_are_refused(B):
    at = dict(zip(CONV, far(7)))
    for out in ("y", "hist_out"):
        for other in CONV:
            if other != out:
                same = (out, other) == ("hist_out", "hist")          # the whole buffer may be both
                assert conv(B, **{out: at[other] + (16 if same else 0)}) == B.PRISM_EINVAL, (out, other)
    at = dict(zip(GRAD, far(11)))
    for out in GRAD[6:]:
        for other in GRAD:
            if other != out:
                assert grad(B, **{out: at[other]}) == B.PRISM_EINVAL, (out, other)
    # y within the rows of a wider tensor that x is columns of
    d = B.ConvDims(4, 20, 64, 4, 1, 128)
    assert conv(B, d, y=far(1)[0] + 128) == B.PRISM_EINVAL


def test_conv_workspace(B):
    """Per workgroup along the tokens an fp32 partial of C (K + 1)."""
    up = lambda x: (x + 255) // 256 * 256
    b = lambda *a: B.conv_workspace_bytes(B.ConvDims(*a))
    assert b(1, 0, 64, 4, 1, 64) == up(64 * 5 * 4)
    assert b(3, 2048, 512, 4, 1, 512) % up(512 * 5 * 4) == 0


QK = ["q", "k", "wq", "wk", "pos", "freqs", "qo", "ko"]


def qd(B, T=10, hq=4, hk=2, d=64, rot=32, dt=1, st=None):
    return B.QkDims(T, hq, hk, d, rot, dt, *(st or (hq * d, d, hk * d, d)))


def qk(B, d=None, norm=1, eps=1e-6, layout=0, **over):
    a = {**dict(zip(QK, far(8))), **over}
    return B.lib().prism_qk_norm(ctypes.byref(d or qd(B)), a["q"], a["k"], a["wq"], a["wk"], norm, eps, a["pos"],
                                 a["freqs"], layout, 1.0, a["qo"], a["ko"], None)


QKG = ["q", "k", "wq", "wk", "pos", "freqs", "dqo", "dko", "dq", "dk", "dwq", "dwk", "ws"]


def qk_grad(B, d=None, norm=1, eps=1e-6, layout=0, nb=1 << 30, **over):
    a = {**dict(zip(QKG, far(13))), **over}
    return B.lib().prism_qk_norm_bwd(ctypes.byref(d or qd(B)), a["q"], a["k"], a["wq"], a["wk"], norm, eps, a["pos"],
                                     a["freqs"], layout, 1.0, *(a[n] for n in QKG[6:]), nb, None)


def test_qk_refuses(B):
    for call in (qk, qk_grad):
        for d in (qd(B, T=-1), qd(B, hq=0), qd(B, hk=-1), qd(B, d=0), qd(B, rot=31), qd(B, rot=66), qd(B, rot=-2),
                  qd(B, dt=2), qd(B, st=(-1, 64, 128, 64)), qd(B, st=(256, 64, 128, -64)), qd(B, st=(1 << 62, 64, 128, 64))):
            assert call(B, d) == B.PRISM_EINVAL
        for kw in (dict(norm=3), dict(norm=-1), dict(layout=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q=None),
                   dict(k=None), dict(wq=None), dict(wk=None), dict(pos=None), dict(freqs=None), dict(q=FAKE + 1),
                   dict(wq=FAKE + 2), dict(pos=FAKE + 4), dict(freqs=FAKE + 4)):
            assert call(B, **kw) == B.PRISM_EINVAL, kw
        assert call(B, qd(B, hk=0)) == B.PRISM_EINVAL                # k and wk without heads of k
        for d in (qd(B, d=513, rot=0), qd(B, hq=65536, st=(0, 0, 0, 0)), qd(B, T=1 << 25, st=(0, 0, 0, 0))):
            a = dict(zip(QK if call is qk else QKG, [FAKE + (i + 1 << 48) for i in range(13)]))
            assert call(B, d, **a) == B.PRISM_EUNSUPPORTED
    for kw in (dict(qo=None), dict(ko=None), dict(qo=FAKE + 2)):
        assert qk(B, **kw) == B.PRISM_EINVAL, kw
    for kw in (dict(dqo=None), dict(dko=None), dict(dq=None), dict(dk=None), dict(dwq=None), dict(dwk=None), dict(ws=None),
               dict(nb=16)):
        assert qk_grad(B, **kw) == B.PRISM_EINVAL, kw
    assert B.qk_workspace_bytes(qd(B, rot=3)) == 0
    assert B.qk_workspace_bytes(qd(B, T=0)) == 512 and B.qk_workspace_bytes(qd(B, T=0, hk=0)) == 256


def test_qk_overlaps_are_refused(B):
    at = dict(zip(QK, far(8)))
    for out in ("qo", "ko"):
        for other in QK:
            if other != out:
                same = out[0] == other                               # whole dense buffers may be both
                assert qk(B, **{out: at[other] + (16 if same else 0)}) == B.PRISM_EINVAL, (out, other)
    assert qk(B, qd(B, st=(2 * 256, 64, 128, 64)), qo=at["q"]) == B.PRISM_EINVAL       # not dense
    assert qk(B, qd(B, st=(64, 640, 128, 64)), qo=at["q"]) == B.PRISM_EINVAL           # dense, heads first
    assert qk(B, qd(B, hk=4, st=(256, 64, 256, 64)), qo=at["k"]) == B.PRISM_EINVAL     # as large as k
    at = dict(zip(QKG, far(13)))
    for out in QKG[8:]:
        for other in QKG:
            if other != out and other != out + "o":
                assert qk_grad(B, **{out: at[other]}) == B.PRISM_EINVAL, (out, other)
    assert qk_grad(B, qd(B, hk=4, st=(256, 64, 256, 64)), dq=at["dko"]) == B.PRISM_EINVAL


SAM = ["logits", "t", "k", "p", "m", "u", "tokens", "probs", "ws"]


def sam(B, d=None, nb=1 << 40, **over):
    a = {**dict(zip(SAM, far(9))), **over}
    return B.lib().prism_sample(ctypes.byref(d or B.SampleDims(4, 1000, 0, 1000)), *(a[n] for n in SAM), nb, None)


def test_sample_refuses(B):
    for d in (B.SampleDims(-1, 1000, 0, 1000), B.SampleDims(4, 0, 0, 1000), B.SampleDims(4, 1000, 2, 1000),
              B.SampleDims(4, 1000, 0, -1), B.SampleDims(4, 1000, 0, 1 << 62)):
        assert sam(B, d) == B.PRISM_EINVAL
        assert B.sample_workspace_bytes(d) == 0
    for kw in (dict(logits=None), dict(logits=FAKE + 2), dict(u=None), dict(tokens=None, probs=None),
               *({n: FAKE + 4} for n in SAM[1:-1])):
        assert sam(B, **kw) == B.PRISM_EINVAL, kw
    assert sam(B, B.SampleDims(4, (1 << 20) + 1, 0, 1 << 21)) == B.PRISM_EUNSUPPORTED
    at = dict(zip(SAM, [FAKE + (i + 1 << 48) for i in range(9)]))
    assert sam(B, B.SampleDims(1 << 23, 1000, 0, 1000), **at) == B.PRISM_EUNSUPPORTED
    at = dict(zip(SAM, far(9)))
    for out in ("tokens", "probs"):
        for other in SAM[:-1]:
            if other != out:
                assert sam(B, **{out: at[other]}) == B.PRISM_EINVAL, (out, other)


def test_sample_workspace(B):
    need = lambda *a: B.sample_workspace_bytes(B.SampleDims(*a))
    assert need(0, 200000, 0, 0) == 0 and need(1, 40960, 0, 0) == 0 and need(200, 200000, 0, 0) == 0
    assert need(1, 131072, 0, 0) > 8 * 1024 * 20 and need(64, 131072, 0, 0) > 64 * 4 * 1024 * 20
    d = B.SampleDims(4, 131072, 0, 131072)
    at = dict(zip(SAM, far(9)))
    n = need(4, 131072, 0, 131072)
    assert sam(B, d, nb=n - 1) == sam(B, d, ws=None) == sam(B, d, ws=FAKE + 8) == B.PRISM_EINVAL
    for other in SAM[:-1]:
        assert sam(B, d, ws=at[other]) == B.PRISM_EINVAL, other
    assert sam(B, d, ws=at["probs"] - n + 256) == B.PRISM_EINVAL


def test_binding_refuses_before_calling(B):
    bf = torch.bfloat16
    x, w, cu = torch.zeros(8, 16, dtype=bf), torch.zeros(16, 4, dtype=bf), torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        B.short_conv(x, w, cu)
    with pytest.raises(ValueError, match="activation"):
        B.short_conv(x, w, cu, activation="gelu")
    with pytest.raises(ValueError, match="channels, taps"):
        B.short_conv(x, w[:8], cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        B.short_conv(x, w, cu.long())
    with pytest.raises(ValueError, match="x must"):
        B.short_conv(x[0], w, cu)
    with pytest.raises(TypeError, match="unsupported dtype"):
        B.short_conv_step(x.half(), w, x)
    with pytest.raises(ValueError, match="n_seqs >= 1"):
        B.short_conv_step(x[:0], w, x)
    q = torch.zeros(8, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="norm"):
        B.qk_norm(q, norm="layer")
    with pytest.raises(ValueError, match="layout"):
        B.qk_norm(q, layout="pairs")
    with pytest.raises(ValueError, match="device"):
        B.qk_norm(q, q)
    with pytest.raises(ValueError, match="logits must"):
        B.sample(x[0])
    with pytest.raises(ValueError, match="device"):
        B.sample(x, want_probs=True)
    with pytest.raises(ValueError, match="even"):
        B.rotary_freqs(7, device="cpu")
    with pytest.raises(ValueError, match="positive"):
        B.rotary_freqs(8, factor=0, device="cpu")


def test_rotary_freqs(B):
    import math
    f = B.rotary_freqs(64, base=500.0, device="cpu")
    assert f.dtype == torch.float32 and f.shape == (32,)
    assert all(abs(f[i].item() - 500.0 ** (-i / 32)) <= 2.0 ** -24 * 500.0 ** (-i / 32) for i in range(32))
    assert torch.equal(B.rotary_freqs(64, base=500.0, factor=4.0, device="cpu"), f / 4)
    g = B.rotary_freqs(64, factor=4.0, trained=4096, low=1.0, high=32.0, device="cpu")
    f = B.rotary_freqs(64, device="cpu")
    for i in range(32):
        turns = 4096 * 10000.0 ** (-i / 32) / (2 * math.pi)
        if turns >= 32:
            assert g[i] == f[i]
        elif turns <= 1:
            assert g[i] == f[i] / 4
        else:
            assert f[i] / 4 < g[i] < f[i]
    assert B.rotary_freqs(0, device="cpu").shape == (0,)
