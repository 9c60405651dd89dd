"""MXFP4 operands of other shapes than the call's."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV  # noqa: E402

def _x(rows, cols, seed, ty=torch.float32):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    return (x * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=gen, device=DEV).float())).to(ty)


def test_operands_of_other_shapes_are_refused():
    x = _x(128, 600, 1)
    q, t = ns.mxfp4_quantize(x), ns.mxfp4_quantize(x, ns.NVFP4_COLS)
    y = torch.randn(128, 100, device=DEV)
    for call in (lambda: ns.mxfp4_gemm(q, q, 64, 128, 600),                   # fewer rows than the panels have
                 lambda: ns.mxfp4_gemm(q, q, 128, 64, 600),
                 lambda: ns.mxfp4_gemm(q, q, 128, 128, 300),                  # fewer panels
                 lambda: ns.mxfp4_linear(x, q, 100),
                 lambda: ns.mxfp4_dequantize(*q, 100, 600),
                 lambda: ns.mxfp4_dequantize(*t, 128, 300, ns.NVFP4_COLS),
                 lambda: ns.mxfp4_linear_backward(y, t, t, 500, need_dw=False),
                 lambda: ns.mxfp4_linear_backward(y, None, t, 500, need_dx=False),
                 lambda: ns.mxfp4_quantize(x, codes=torch.empty(3, 130, 128, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call()
