"""The norm refuses an eps whose square root has no FP32 reciprocal (CPU only:
the addresses are never dereferenced)."""
import ctypes

import pytest

ns = pytest.importorskip("newton_schulz_amd")


def at(i):
    return (i + 1) * (1 << 40)


@pytest.mark.parametrize("eps", [5e-324, 1e-300, 1e-78, 2.0 ** -255, 2.0 ** -254 * (1 - 2.0 ** -53)])
def test_an_eps_that_leaves_fp32(eps):
    """A row of zeros would be 0 * infinity."""
    a = ns.MxNormArgs()
    a.x, a.weight, a.y, a.T, a.C, a.eps = at(0), at(1), at(2), 8, 64, eps
    assert ns._lib.mx_rms_norm(ctypes.byref(a), None) == ns.NS_ERR_ARG
