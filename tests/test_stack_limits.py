"""Refusals and workspace sizes at the limits of the short convolution, the norm and rotation of queries and
keys, and the choice of a token.  No GPU needed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
FAR = [0x10000 + (i + 1 << 34) for i in range(13)]           # aligned, apart, never dereferenced


@pytest.fixture(scope="module")
def B():
    from gated_delta_rule_prologue_amd import binding
    binding.lib()
    return binding


def test_rows_behind_are_cleared_or_not(B):
    """prism_short_conv_ex refuses what prism_short_conv does, and any other choice than 0 and 1."""
    def call(clear, d=B.ConvDims(4, 20, 64, 4, 1, 64), y=FAR[5]):
        return B.lib().prism_short_conv_ex(ctypes.byref(d), *FAR[:5], 1, clear, y, FAR[6], None)

    for clear in (-1, 2, 256):
        assert call(clear) == B.PRISM_EINVAL
    for clear in (0, 1):
        assert call(clear, y=None) == B.PRISM_EINVAL and call(clear, y=FAR[0]) == B.PRISM_EINVAL
        assert call(clear, d=B.ConvDims(4, 20, 64, 9, 1, 64)) == B.PRISM_EINVAL
        assert call(clear, d=B.ConvDims(4, 20, (1 << 22) + 1, 4, 1, 1 << 23)) == B.PRISM_EUNSUPPORTED


BIG = 2 ** 31 - 1


def test_workspaces_of_refused_dims_are_empty(B):
    """Nothing is asked for, whatever a caller would allocate, and the call says that the dims are unsupported."""
    wide = [0x10000 + (i + 1 << 50) for i in range(13)]
    for c in ((1 << 22) + 1, 1 << 30, BIG - 8, BIG):
        d = B.ConvDims(4, 20, c, 4, 1, c)
        assert B.conv_workspace_bytes(d) == 0
        assert B.lib().prism_short_conv_bwd(ctypes.byref(d), *wide[:5], 1, *wide[5:10], None, 0, None) == B.PRISM_EUNSUPPORTED
    assert B.conv_workspace_bytes(B.ConvDims(4, (1 << 30) + 1, 1, 4, 1, 1)) == 0
    for T, width in ((10, 513), (10, BIG), (1 << 23, 64)):
        d = B.QkDims(T, 1, 1, width, 0, 1, 0, 0, 0, 0)
        assert B.qk_workspace_bytes(d) == 0
        assert B.lib().prism_qk_norm_bwd(ctypes.byref(d), *wide[:4], 1, 1e-6, None, None, 0, 1.0, *wide[4:10], None, 0,
                                         None) == B.PRISM_EUNSUPPORTED
    for rows, vocab in ((8, (1 << 20) + 1), (8, 1 << 30), (8, BIG), (1, BIG), (1 << 22, 100), (1 << 40, 100)):
        d = B.SampleDims(rows, vocab, 0, 0)
        assert B.sample_workspace_bytes(d) == 0
        assert B.lib().prism_sample(ctypes.byref(d), *wide[:7], None, None, 0, None) == B.PRISM_EUNSUPPORTED


def test_workspaces_at_the_limits(B):
    assert B.conv_workspace_bytes(B.ConvDims(4, 20, 1 << 22, 8, 1, 1 << 22)) >= (1 << 22) * 9 * 4
    assert B.qk_workspace_bytes(B.QkDims((1 << 23) - 1, 1, 1, 512, 0, 1, 0, 0, 0, 0)) == 1024 * 2 * 512 * 4
    assert 0 < B.sample_workspace_bytes(B.SampleDims(80, 1 << 20, 0, 0)) < 80 * 64 * 21_000
