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
