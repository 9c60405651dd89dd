"""MXFP4 paths of their own: products of few rows whose waves pass over K more
than once, wide odd rows through the quantizers, operands of other shapes."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402

U32, UBF = 2.0 ** -24, 2.0 ** -8


def _x(rows, cols, seed, ty=torch.float32):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    return (x * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=gen, device=DEV).float())).to(ty)


# few_kernel with 16 waves of one panel at a time (fewer than 512 groups of 16
# weight rows, 16 panels or more) and with 4 waves of four (more rows); rows of
# x by 16-byte loads or by elements; one pass over K or several, the last of
# them with fewer panels
FEW = [(1, 4096, 4096), (7, 4096, 4096), (16, 4096, 4096), (1, 1000, 11008), (7, 1000, 11008), (16, 1000, 11008),
       (1, 300, 9999), (5, 300, 9999), (16, 300, 9999), (17, 500, 9000), (32, 500, 9000), (31, 500, 9002), (25, 300, 9999),
       (1, 8200, 5000), (16, 8200, 5000), (3, 8195, 9001), (16, 8179, 4700), (31, 8180, 2040), (20, 600, 3800)]


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", FEW)
def test_few_rows(T, N, K, ty):
    assert ns.mxfp4_linear_workspace_bytes(T, N, K) == 0              # that kernel
    x, w = _x(T, K, T + N, ty), _x(N, K, N + K)
    wq = ns.mxfp4_quantize(w)
    xq = O.quantize(x.double().cpu().numpy())
    xv = torch.from_numpy(O.dequantize(*xq, K)).to(DEV)
    wv = ns.mxfp4_dequantize(*wq, N, K).double()
    want = xv @ wv.t()
    # exact products, at most K roundings of sums below the sum of magnitudes
    tol = (K + 4) * U32 * (xv.abs() @ wv.abs().t())
    u = UBF if ty == torch.bfloat16 else U32
    y = ns.mxfp4_linear(x, wq, N)
    assert bool(((y - want).abs() <= tol + u * (want.abs() + tol)).all())
    held = tuple(torch.from_numpy(a).to(DEV) for a in xq)
    out = torch.full((T * N + 64,), 5.0, device=DEV)
    ns.mxfp4_gemm(held, wq, T, N, K, out=out)
    assert bool(((out[:T * N].view(T, N) - want).abs() <= tol + U32 * (want.abs() + tol)).all())
    assert bool((out[T * N:] == 5.0).all())
    add = _x(T, N, 9)
    got = ns.mxfp4_gemm(held, wq, T, N, K, alpha=0.5, beta=-1.0, addend=add)
    ref = 0.5 * want - add.double()
    assert bool(((got - ref).abs() <= 0.5 * tol + 4 * U32 * (want.abs() + add.abs())).all())


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(37, 4095), (4095, 37), (5, 8193), (300, 1021), (3, 2047), (257, 4097), (1000, 999),
                                       (40, 2050), (9, 2052)])
def test_quantizers_on_wide_odd_rows(rows, cols, ty):
    x = torch.from_numpy(synth.student_t(rows, cols, rows + cols)).to(ty).to(DEV)
    xv = x.double().cpu().numpy()
    along, down = O.quantize(xv), O.quantize(xv.T)
    same = lambda got, want: all(np.array_equal(host(g), w) for g, w in zip(got, want))  # noqa: E731
    a, d = ns.mxfp4_quantize_both(x)
    assert same(a, along) and same(d, down)
    assert same(ns.mxfp4_quantize(x), along) and same(ns.mxfp4_quantize(x, ns.NVFP4_COLS), down)
    for ot in (ns.NS_F32, ns.NS_BF16):
        assert np.array_equal(host(ns.mxfp4_dequantize(*a, rows, cols, out_dtype=ot)), O.dequantize(*along, cols))
        assert np.array_equal(host(ns.mxfp4_dequantize(*d, rows, cols, ns.NVFP4_COLS, ot)), O.dequantize(*down, rows).T)


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


@pytest.mark.parametrize("M,N,K", [(5, 100, 700), (300, 333, 1000), (1024, 1024, 256), (4096, 4096, 512)])
def test_products_of_far_scales_are_exact(M, N, K):
    """Powers of two on the operands are powers of two on the product, to the
    bit, subnormal results included (their sums have bits to spare)."""
    x, y = _x(M, K, 1), _x(N, K, 2)
    base = ns.mxfp4_gemm(ns.mxfp4_quantize(x), ns.mxfp4_quantize(y), M, N, K).double()
    for ex, ey in ((100, -100), (-60, -50), (60, 40), (110, -112), (-112, 110), (-90, -40)):
        p, q = (ns.mxfp4_quantize(torch.ldexp(t, torch.tensor(e, device=DEV))) for t, e in ((x, ex), (y, ey)))
        want = torch.ldexp(base, torch.tensor(ex + ey, device=DEV)).float()
        assert torch.equal(ns.mxfp4_gemm(p, q, M, N, K), want), (ex, ey)
