"""The operators between 4-bit layers beyond 2^31 elements and 4 GiB of codes:
stretches of rows from the start, the middle and the end against calls on these
rows alone (bit for bit where a row does not depend on the others)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402
from oracle import layer as L  # noqa: E402

U = 2.0 ** -24
T, C = 2100003, 1031          # 2.165e9 elements


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def stretches(rows, n=512, step=256):
    """[a, b): the first rows, those around element 2^31 and byte 2^32, the last."""
    marks = {0, rows // 2 // step * step, (rows - 1) // step * step, (1 << 31) // C // step * step, (1 << 32) // C // 2 // step * step}
    return sorted((a, min(a + n, rows)) for a in marks if a < rows)


def rows_of(op, a, b):
    return op[0][:, a:b], op[1][:, a:b]


def same(p, q):
    return torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


def test_dropout():
    x = torch.randn(T, C, generator=gen(1), device=DEV, dtype=torch.bfloat16)
    seed, offset = 5, 6
    y = ns.mx_dropout(x, 0.5, torch.tensor([seed, offset], device=DEV))
    c = np.arange(C)
    for t in (0, 1, (1 << 31) // C - 1, (1 << 31) // C, (1 << 31) // C + 1, (1 << 32) // C // 2, T - 2, T - 1):
        w = np.stack([np.broadcast_to(v, c.shape) for v in L.philox((c // 8, t, offset, 0), (seed, 0))])
        bits = (w[c // 2 % 4, c] >> (16 * (c % 2)).astype(np.uint64)) & np.uint64(0xFFFF)
        want = host(x[t]) * np.where(bits >= 32768, 2.0, 0.0)
        assert np.array_equal(host(y[t]), want)
    kept = sum(int((y[a:a + 100000] != 0).sum()) for a in range(0, T, 100000))
    assert abs(kept - T * C / 2) < 1e-3 * T * C


def test_norm_and_gradients():
    g = gen(2)
    x, r, dy = (torch.randn(T, C, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    w = 1 + 0.2 * torch.randn(C, generator=g, device=DEV)
    n = ns.mx_rms_norm(x, w, residual=r, y=True, mxfp8=True, mxfp4=True, kept=True, rstd=True)
    b = ns.mx_rms_norm_backward(dy, n.h, n.rstd, w, dh=r, x_dtype=torch.float32)
    for s, e in stretches(T):
        m = ns.mx_rms_norm(x[s:e].clone(), w, residual=r[s:e].clone(), y=True, mxfp8=True, mxfp4=True, kept=True, rstd=True)
        assert torch.equal(n.h[s:e], m.h) and torch.equal(n.y[s:e], m.y) and torch.equal(n.rstd[s:e], m.rstd)
        assert same(rows_of(n.mxfp8, s, e), m.mxfp8) and same(rows_of(n.mxfp4, s, e), m.mxfp4)
        assert same((n.kept[0][s // 256:-(-e // 256)], n.kept[1][s // 256:-(-e // 256)]), m.kept)
        d = ns.mx_rms_norm_backward(dy[s:e].clone(), m.h, m.rstd, w, dh=r[s:e].clone(), x_dtype=torch.float32)
        assert torch.equal(b.dh[s:e], d.dh) and torch.equal(b.dx[s:e], d.dx)
    want, size = torch.zeros(C, device=DEV, dtype=torch.float64), torch.zeros(C, device=DEV, dtype=torch.float64)
    for a in range(0, T, 100000):
        p = dy[a:a + 100000].double() * (n.h[a:a + 100000].double() * n.rstd[a:a + 100000].double()[:, None])
        want += p.sum(0)
        size += p.abs().sum(0)
    # a lane's rows, 768 workgroups by 32, 32 threads, and 4 for the products
    assert bool(((b.dw.double() - want).abs() <= (-(-T // 768) + 24 + 32 + 4) * U * size).all())


def test_mxfp8():
    rows, cols = T, 2100       # 4.4e9 elements, 4.8 GB of codes
    x = torch.randn(rows, cols, generator=gen(3), device=DEV, dtype=torch.bfloat16)
    q = ns.mxfp8_quantize(x)
    assert q[0].numel() > 1 << 32
    back = ns.mxfp8_dequantize(*q, rows, cols, ns.NS_BF16)
    for s, e in stretches(rows):
        p = ns.mxfp8_quantize(x[s:e].clone())
        assert same(rows_of(q, s, e), p)
        assert torch.equal(back[s:e], ns.mxfp8_dequantize(*p, e - s, cols, ns.NS_BF16))


def random_operand(seed, rows, cols, width):
    """Codes and scales of any values (E4M3's NaN excepted), zeros behind a row's end."""
    g = gen(seed)
    p = -(-cols // 256)
    codes = torch.randint(0, 256, (p, rows, width), generator=g, device=DEV, dtype=torch.uint8)
    if width == 256:
        codes -= (codes & 127) // 127
    scales = torch.randint(120, 131, (p, rows, 8), generator=g, device=DEV, dtype=torch.uint8)
    last = cols - 256 * (p - 1)
    assert last % 32 == 0
    codes[-1, :, last * width // 256:] = 0
    scales[-1, :, last // 32:] = 0
    return codes, scales


def picked(op, rows):
    return op[0][:, rows].contiguous(), op[1][:, rows].contiguous()


def check(got, p, q, K, dtype):
    """The product of a few rows of each operand, as in test_gpu_mxfp8_tiles.py."""
    M, N = got.shape
    P, Q = ns.mxfp8_dequantize(*p, M, K).double(), ns.mxfp4_dequantize(*q, N, K).double()
    want, size = P @ Q.T.contiguous(), P.abs() @ Q.abs().T.contiguous()
    bound = (K + 2) * U * size
    if dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -13 * sum(P[:, k:k + 8].abs().amax(1)[:, None] * Q[:, k:k + 8].abs().amax(1) for k in range(0, K, 8))
    half = U if dtype == torch.float32 else 2.0 ** -8
    assert bool(((got.double() - want).abs() <= bound + half * (want.abs() + bound)).all())


@pytest.mark.parametrize("M,N,K", [(1100001, 33, 4064), (70001, 33001, 64), (1, 2200003, 4064), (19, 2200003, 4064)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mixed_product(M, N, K, dtype):
    """P's codes, the outputs, or Q's codes beyond 4 GiB."""
    kind, code = (torch.float32, ns.NS_F32) if dtype == "f32" else (torch.bfloat16, ns.NS_BF16)
    p, q = random_operand(4, M, K, 256), random_operand(5, N, K, 128)
    assert max(p[0].numel(), q[0].numel(), 4 * M * N) > 1 << 32
    out = torch.full((M, N), float("nan"), dtype=kind, device=DEV)
    ns.mxfp8_gemm(p, q, M, N, K, out=out)
    some = lambda n: torch.tensor(sorted({*range(min(n, 40)), *(i for a in (n // 2, n - 40) for i in range(max(a, 0), min(max(a, 0) + 40, n)))}), device=DEV)  # noqa: E731
    r, c = some(M), some(N)
    check(out[r][:, c], picked(p, r), picked(q, c), K, kind)
    assert all(bool(torch.isfinite(out.view(-1)[a:a + (1 << 28)]).all()) for a in range(0, M * N, 1 << 28))


@pytest.mark.parametrize("tokens", [1, 2, 5, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nvfp4_linear(tokens, dtype):
    """4.3 GB of codes."""
    N, K = 2100005, 4112
    g = gen(6)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(0x20, 0x48, (N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
    sg = torch.tensor([0.01], device=DEV)
    x = torch.randn(tokens, K, generator=g, device=DEV).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    y = ns.nvfp4_linear(x, (codes, scales, sg), N, out=torch.full((tokens, N), float("nan"), device=DEV))
    assert bool(torch.isfinite(y).all())
    for a in (0, (1 << 32) // (K // 2) - 32, N // 2, N - 64):
        part = codes[a:a + 64].clone(), scales[a:a + 64].clone()
        if tokens <= 2:
            assert torch.equal(y[:, a:a + 64], ns.nvfp4_linear(x, (*part, sg), 64, out=torch.empty(tokens, 64, device=DEV)))
        w = ns.nvfp4_dequantize(*part, torch.ones_like(sg), 64, K).double() * sg.double()
        want, size = x.double() @ w.T.contiguous(), x.double().abs() @ w.abs().T.contiguous()
        bound = (K + 3 if dtype == "bf16" else 3 * K + 5) * U * size
        assert bool(((y[:, a:a + 64].double() - want).abs() <= bound + U * (want.abs() + bound)).all())
