"""The norm where its inputs leave the ordinary: weights without a value, and
rows that pass through a workgroup one after the other."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402
from oracle import layer as L  # noqa: E402
from oracle import mxfp4 as M4  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("types", ["f32 f32", "bf16 bf16", "f32 bf16"])
@pytest.mark.parametrize("T,C", [(1, 70), (31, 33), (32, 40), (40, 256), (224, 129), (256, 48), (257, 64), (300, 300), (5, 4100)])
def test_weights_that_are_not_finite(T, C, types):
    """A column of NaN or infinities: its blocks are NaN, what lies behind the
    last token or column stays zero, in every operand."""
    ht, wt = (TYPES[t] for t in types.split())
    g = np.random.default_rng(T + C)
    x = torch.from_numpy(g.standard_normal((T, C)).astype(np.float32)).to(ht).to(DEV)
    w = torch.from_numpy((1 + 0.2 * g.standard_normal(C)).astype(np.float32)).to(wt).to(DEV)
    w[0], w[C // 2], w[C - 1] = float("inf"), float("nan"), -float("inf")
    n = ns.mx_rms_norm(x, w, y=True, mxfp8=True, mxfp4=True, kept=True, rstd=True)
    with np.errstate(invalid="ignore"):
        y = (host(x).astype(np.float32) * host(n.rstd).astype(np.float32)[:, None]) * host(w).astype(np.float32)
    assert torch.equal(n.y.cpu().isnan(), torch.from_numpy(np.isnan(y)))
    for got, (codes, scales) in ((n.mxfp8, L.mx8_quantize(y)), (n.mxfp4, M4.quantize(y)), (n.kept, M4.quantize(y.T))):
        assert np.array_equal(host(got[0]), codes) and np.array_equal(host(got[1]), scales)


@pytest.mark.parametrize("C", [9, 64, 300, 5000])
def test_the_smallest_eps(C):
    """2^-254: rows without values are zero, the smallest values meet r = 2^127."""
    x = torch.zeros(3, C, device=DEV)
    x[1], x[2] = 2.0 ** -149, 3.0
    n = ns.mx_rms_norm(x, torch.ones(C, device=DEV), 2.0 ** -254, y=True, rstd=True, mxfp8=True)
    y, r = host(n.y), host(n.rstd)
    assert not y[0].any() and not host(n.mxfp8[0])[:, 0].any() and not host(n.mxfp8[1])[:, 0].any()
    assert np.all(y[1] == 2.0 ** -22) and np.all(r[:2] == 2.0 ** 127)
    assert np.all(np.abs(y[2] - 1.0) <= 3 * 2.0 ** -24)
