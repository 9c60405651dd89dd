"""The operators between 4-bit layers on tensors inside larger buffers: what lies
around an output stays as it is, what lies around an input (NaN, or codes of
them) does not show, and results are those of tensors by themselves, bit for bit."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV  # noqa: E402

PAD = 1024
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class Guards:
    def __init__(self):
        self.all = []

    def out(self, *shape, dtype=torch.uint8):
        fill, n = 85 if dtype == torch.uint8 else 7.25, math.prod(shape)
        b = torch.full((n + 2 * PAD,), fill, dtype=dtype, device=DEV)
        self.all.append((b, n, fill))
        return b[PAD:PAD + n].view(shape)

    def pair(self, rows, cols, width):
        p = -(-cols // 256)
        return self.out(p, rows, width), self.out(p, rows, 8)

    def untouched(self):
        return all(bool((b[:PAD] == f).all()) and bool((b[PAD + n:] == f).all()) for b, n, f in self.all)


def inside(t):
    fill = 127 if t.dtype == torch.uint8 else float("nan") if t.is_floating_point() else -1
    b = torch.full((t.numel() + 2 * PAD,), fill, dtype=t.dtype, device=DEV)
    v = b[PAD:PAD + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def same(a, b):
    return same(a[0], b[0]) and same(a[1], b[1]) if isinstance(a, tuple) else torch.equal(a, b)


@pytest.mark.parametrize("types", ["f32 f32", "bf16 bf16", "bf16 f32"])
@pytest.mark.parametrize("T,C", [(1, 1), (5, 7), (33, 64), (40, 100), (9, 250), (70, 500), (31, 1001), (300, 1111), (3, 4097), (2, 8190),
                                 (300, 8195), (2, 32767)])
def test_norm(T, C, types):
    xt, ht = (TYPES[t] for t in types.split())
    x, r, w, dy, din = rand(1, T, C, dtype=xt), rand(2, T, C, dtype=ht), rand(3, C, dtype=xt), rand(4, T, C, dtype=xt), rand(5, T, C, dtype=ht)
    rng = torch.tensor([3, 4], device=DEV)
    g = Guards()
    a = ns.mx_rms_norm(x, w, residual=r, drop=0.3, rng=rng, y=True, mxfp8=True, mxfp4=True, kept=True, rstd=True)
    b = ns.mx_rms_norm(inside(x), inside(w), residual=inside(r), drop=0.3, rng=inside(rng), h=g.out(T, C, dtype=ht), y=g.out(T, C, dtype=xt),
                       mxfp8=g.pair(T, C, 256), mxfp4=g.pair(T, C, 128), kept=g.pair(C, T, 128), rstd=g.out(T, dtype=torch.float32))
    assert g.untouched() and all(same(p, q) for p, q in zip(a, b))
    a = ns.mx_rms_norm_backward(dy, a.h, a.rstd, w, dh=din, drop=0.3, rng=rng)
    b = ns.mx_rms_norm_backward(inside(dy), inside(b.h), inside(b.rstd), inside(w), dh=inside(din), drop=0.3, rng=inside(rng),
                                out=g.out(T, C, dtype=ht), dx=g.out(T, C, dtype=xt), dw=g.out(C, dtype=torch.float32),
                                workspace=g.out(ns.mx_rms_norm_backward_workspace_bytes(T, C)))
    assert g.untouched() and all(same(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(1, 1), (7, 5), (300, 9), (33, 255), (70, 1501), (5, 8199)])
def test_dropout_and_mxfp8(T, C, dtype):
    x, rng, g = rand(1, T, C, dtype=TYPES[dtype]), torch.tensor([3, 4], device=DEV), Guards()
    assert same(ns.mx_dropout(x, 0.3, rng), ns.mx_dropout(inside(x), 0.3, inside(rng), out=g.out(T, C, dtype=x.dtype)))
    q = g.pair(T, C, 256)
    assert same(ns.mxfp8_quantize(x), ns.mxfp8_quantize(inside(x), *q))
    code = ns.NS_F32 if dtype == "f32" else ns.NS_BF16
    assert same(ns.mxfp8_dequantize(*q, T, C, code), ns.mxfp8_dequantize(*map(inside, q), T, C, out=g.out(T, C, dtype=x.dtype)))
    assert g.untouched()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 21, 300), (16, 1000, 4095), (17, 33, 70), (100, 130, 2600), (34, 3011, 4094), (300, 777, 1501),
                                   (1067, 1940, 19), (390, 8378, 25), (2100, 2300, 515), (798, 9251, 17)])
def test_mixed_product(M, N, K, dtype):
    p, q, add, g = ns.mxfp8_quantize(rand(1, M, K)), ns.mxfp4_quantize(rand(2, N, K)), rand(3, M, N), Guards()
    code = ns.NS_F32 if dtype == "f32" else ns.NS_BF16
    need = ns.mxfp8_gemm_workspace_bytes(M, N, K)
    for beta in (0.0, 1.5):
        a = ns.mxfp8_gemm(p, q, M, N, K, beta=beta, addend=add, out_dtype=code)
        b = ns.mxfp8_gemm(tuple(map(inside, p)), tuple(map(inside, q)), M, N, K, beta=beta, addend=inside(add), out=g.out(M, N, dtype=TYPES[dtype]),
                          workspace=g.out(need) if need else None)
        assert g.untouched() and same(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 33, 4112), (2, 1000, 2080), (2, 9, 48), (5, 30, 1040), (16, 4113, 160), (33, 100, 272), (40, 9000, 64)])
def test_nvfp4_linear(T, N, K, dtype):
    codes, scales, sg = ns.nvfp4_quantize(rand(1, -(-N // 16) * 16, K))
    w, x, g = (codes[:N].contiguous(), scales[:N].contiguous(), sg), rand(2, T, K, dtype=TYPES[dtype]), Guards()
    assert same(ns.nvfp4_linear(x, w, N), ns.nvfp4_linear(inside(x), tuple(map(inside, w)), N, out=g.out(T, N, dtype=x.dtype)))
    assert g.untouched()
