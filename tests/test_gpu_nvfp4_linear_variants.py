"""The linear layer on NVFP4 weights: groups of rows and tokens that its other
tests do not meet, with the bounds of test_gpu_nvfp4_linear.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV  # noqa: E402

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [
    (33, 11001, 512), (40, 11008, 64), (50, 6000, 4096),      # BF16: pairs of rows' groups and of tokens', K whole lanes
    (4200, 16, 64), (4113, 10, 48), (8200, 1, 16),            # one group of rows, FP32 tokens beyond 256 workgroups
    (1500, 300, 144), (3000, 64, 1024)])
def test_sums(T, N, K, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(T + N)
    W = torch.zeros(-(-N // 16) * 16, K, device=DEV)
    W[:N] = torch.randn(N, K, generator=g, device=DEV) * torch.exp2(torch.randint(-3, 4, (N, K), generator=g, device=DEV).float())
    codes, scales, sg = ns.nvfp4_quantize(W)
    op = codes[:N].contiguous(), scales[:N].contiguous(), sg
    # codes times block scales are exact in FP32, so s_g is applied in 64 bits
    w = ns.nvfp4_dequantize(codes, scales, torch.ones_like(sg), W.shape[0], K)[:N].double() * sg.double()
    x = torch.randn(T, K, generator=g, device=DEV).to(TYPES[dtype])
    wt, X = w.T.contiguous(), x.double()
    n = K + 3 if dtype == "bf16" else 3 * K + 5
    want, bound = X @ wt, n * U * (X.abs() @ wt.abs())
    for kind, half in ((torch.float32, U), (torch.bfloat16, 2.0 ** -8)):
        out = torch.full((T, N), float("nan"), dtype=kind, device=DEV)
        y = ns.nvfp4_linear(x, op, N, out=out).double()
        assert bool(((y - want).abs() <= bound + half * (want.abs() + bound)).all())
    # the last elements of K one by one: each meets its own
    for k in range(max(0, K - 34), K, 3):
        e = torch.zeros(T, K, device=DEV)
        e[:, k] = 3.0
        y = ns.nvfp4_linear(e.to(TYPES[dtype]), op, N, out=torch.empty(T, N, device=DEV)).double()
        assert bool(((y - 3.0 * w[:, k]).abs() <= 3 * U * (3.0 * w[:, k]).abs()).all())
