"""Tensors of the caller's that a call writes show to autograd as written."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV  # noqa: E402

QUINTIC = synth.QUINTIC


def test_an_update_shows_to_autograd():
    """A weight saved for a backward pass and updated before it is reported, as
    with torch's own updates in place."""
    w = torch.nn.Parameter(torch.randn(64, 80, device=DEV))
    mom, g = torch.zeros(64, 80, device=DEV), torch.randn(64, 80, device=DEV)
    loss = (w * w).sum()
    before = w._version, mom._version, g._version
    ns.ns_muon_step([w], [mom], [g], [QUINTIC] * 5, lr=0.1)
    assert w._version > before[0] and mom._version > before[1] and g._version == before[2]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():                      # tensors without a counter
        ns.ns_muon_step([w.clone()], [mom.clone()], [g], [QUINTIC] * 5, lr=0.1)


def test_outputs_given_to_a_call_show_to_autograd():
    x = torch.randn(64, 96, device=DEV)
    q = ns.mxfp4_quantize(x)
    wt = ns.mxfp4_quantize(x, ns.NVFP4_COLS)
    y, dx, dw, o = (torch.zeros(*s, device=DEV) for s in ((64, 64), (64, 96), (64, 96), (64, 96)))
    kept = tuple(t.clone() for t in wt)
    for given, call in (
            (q, lambda: ns.mxfp4_quantize(x, codes=q[0], scales=q[1])),
            (q + wt, lambda: ns.mxfp4_quantize_both(x, along=q, down=wt)),
            ((o,), lambda: ns.mxfp4_dequantize(*q, 64, 96, out=o)),
            ((y,), lambda: ns.mxfp4_gemm(q, q, 64, 64, 96, out=y)),
            ((y,) + kept, lambda: ns.mxfp4_linear(x, q, 64, out=y, kept=kept)),
            ((dx, dw), lambda: ns.mxfp4_linear_backward(y, wt, kept, 96, dx=dx, dw=dw)),
            ((o,), lambda: ns.ns_orthogonalize_f16(x, [QUINTIC], out=o)),
            ((o, dx), lambda: ns.ns_orthogonalize_f16_grouped([x, dw], [QUINTIC], outs=[o, dx]))):
        before = [t._version for t in given]
        call()
        assert all(t._version > v for t, v in zip(given, before))
