"""Mixed products on every shape of tile: one unit or several a workgroup, K
whole or in parts, one panel or many, rows and columns that end inside a tile.

Bounds as in test_gpu_mxfp8.py.  They grow with K and would hide one lost
element of many, so every size is also multiplied by rows of a single element,
whose products are exact in either output type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV  # noqa: E402

U = 2.0 ** -24

# tiles taken (rows x columns) for BF16 | FP32 outputs, with a workspace
SIZES = [
    (18, 18, 17),         # 64x64 | 64x64
    (22, 17, 2145),       # 64x64 in parts | the same
    (71, 8405, 23),       # 64x128 | the same
    (292, 4001, 62),      # 64x128 | the same
    (805, 4637, 1546),    # 64x128, several a workgroup
    (1439, 2703, 890),    # FP32: the same
    (34, 3011, 4094),     # 64x128 in parts
    (328, 330, 4059),     # 64x128 in parts
    (597, 415, 1914),     # FP32: 64x128 in parts
    (1067, 1940, 19),     # 128x128 | the same
    (5744, 265, 29),      # 128x128 | the same
    (5651, 1352, 536),    # 128x128, several a workgroup
    (4172, 1880, 279),    # FP32: the same
    (74, 2053, 5188),     # 128x128 in parts
    (372, 1436, 3669),    # FP32: 128x128 in parts
    (774, 283, 5344),     # FP32: 128x128 in parts
    (390, 8378, 25),      # 128x256 | the same
    (2016, 2264, 165),    # 128x256 | the same
    (1805, 8210, 39),     # 128x256, several a workgroup | the same
    (2178, 140, 13638),   # 128x256 in parts
    (636, 782, 11429),    # FP32: 128x256 in parts
    (798, 9251, 17),      # 256x256 | the same
    (6574, 2357, 21),     # 256x256, several a workgroup
    (5059, 7363, 300),    # 256x256, several a workgroup | the same
]
TYPES = {"f32": (torch.float32, ns.NS_F32), "bf16": (torch.bfloat16, ns.NS_BF16)}


def operands(seed, M, N, K):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    spread = lambda rows: torch.exp2(torch.randint(-3, 4, (rows, K), generator=g, device=DEV).float())  # noqa: E731
    p = ns.mxfp8_quantize(torch.randn(M, K, generator=g, device=DEV) * spread(M))
    q = ns.mxfp4_quantize(torch.randn(N, K, generator=g, device=DEV) * spread(N))
    return p, q, ns.mxfp8_dequantize(*p, M, K).double(), ns.mxfp4_dequantize(*q, N, K).double()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sums(M, N, K, dtype):
    kind, code = TYPES[dtype]
    p, q, P, Q = operands(M + N + K, M, N, K)
    Qt = Q.T.contiguous()
    sums, size = P @ Qt, P.abs() @ Qt.abs()
    lost = torch.zeros((), device=DEV, dtype=torch.float64)
    if dtype == "bf16":       # the window's share
        A, B = P.abs(), Q.abs()
        for k in range(0, K, 8):
            lost = lost + A[:, k:k + 8].amax(1)[:, None] * B[:, k:k + 8].amax(1)
        lost = 7 * 2.0 ** -13 * lost
    half = U if dtype == "f32" else 2.0 ** -8
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    add = torch.randn(M, N, generator=g, device=DEV)
    for alpha, beta, split in ((1.0, 0.0, True), (-0.5, 2.0, True), (1.0, 0.0, False)):
        out = torch.full((M, N), float("nan"), dtype=kind, device=DEV)
        got = ns.mxfp8_gemm(p, q, M, N, K, alpha=alpha, beta=beta, addend=add if beta else None, out=out, split=split).double()
        want = alpha * sums + beta * add.double()
        bound = (K + 2) * U * (abs(alpha) * size + abs(beta) * add.double().abs()) + abs(alpha) * lost
        assert bool(((got - want).abs() <= bound + half * (want.abs() + bound)).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_rows_of_a_single_element(M, N, K, dtype):
    """Row m of P holds element (m + shift) % K alone: every product comes out as
    it is, whatever the tile, the panel, the part or the place in it."""
    kind, code = TYPES[dtype]
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N)
    q = ns.mxfp4_quantize(torch.randn(N, K, generator=g, device=DEV))
    Q = ns.mxfp4_dequantize(*q, N, K)
    rows = torch.arange(M, device=DEV)
    times = -(-K // M)
    for shift in range(0, K, M * max(1, times // (128 if M * N < 200000 else 6))):
        at = (rows + shift) % K
        x = torch.zeros(M, K, device=DEV)
        x[rows, at] = torch.randn(M, generator=g, device=DEV)
        p = ns.mxfp8_quantize(x)
        held = ns.mxfp8_dequantize(*p, M, K)[rows, at]
        got = ns.mxfp8_gemm(p, q, M, N, K, out_dtype=code)
        assert got.dtype == kind and torch.equal(got.float(), held[:, None] * Q[:, at].T)
