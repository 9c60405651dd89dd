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


@pytest.mark.parametrize("types", ["f32 f32", "bf16 bf16"])
@pytest.mark.parametrize("T,C", [(1, 70), (5, 8), (31, 33), (32, 40), (33, 128), (40, 256), (249, 129), (256, 48), (257, 64), (300, 300)])
def test_negative_weights(T, C, types):
    """What lies behind the last token or column is zero to the bit."""
    ht, wt = (TYPES[t] for t in types.split())
    g = np.random.default_rng(T + C)
    x = torch.from_numpy(g.standard_normal((T, C)).astype(np.float32)).to(ht).to(DEV)
    w = torch.from_numpy(g.standard_normal(C).astype(np.float32)).to(wt).to(DEV)
    n = ns.mx_rms_norm(x, w, mxfp8=True, mxfp4=True, kept=True, rstd=True)
    y = (host(x).astype(np.float32) * host(n.rstd).astype(np.float32)[:, None]) * host(w).astype(np.float32)
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


U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def weight_depth(T, C):
    """FP32 additions behind a column's dw: the rows of a workgroup that a lane
    takes, those that share it, the workgroups of a thread of the last sum and its
    32 threads; and 4 for the products."""
    rows, most = (1, 256) if C > 8192 else (32 if C <= 64 else 16 if C <= 128 else 8 if C <= 256 else 4 if C <= 1024 else 1, 768)
    groups = min(most, -(-T // rows))
    return -(-T // (rows * groups)) + rows + -(-groups // 32) + 32 + 4


@pytest.mark.parametrize("types", ["f32 f32 f32", "bf16 bf16 bf16", "bf16 f32 bf16"])
@pytest.mark.parametrize("T,C", [(50000, 24), (25601, 63), (26000, 100), (13000, 255), (6500, 200), (7000, 700), (3500, 1024), (1600, 1500),
                                 (1537, 2049), (800, 4099), (2400, 6000), (770, 8192), (257, 8193), (600, 8200), (513, 16384), (600, 16385),
                                 (520, 32768)])
def test_gradients_of_more_rows_than_workgroups(T, C, types):
    """Every workgroup walks over rows, with and without the stream's gradient in
    place and dropout; FP64 on the device, dropout's factors from mx_dropout."""
    xt, ht, wt = (TYPES[t] for t in types.split())
    g = torch.Generator(device=DEV)
    g.manual_seed(T + C)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    h, dy, din = rand(T, C).to(ht), (1e-2 * rand(T, C)).to(xt), (1e-2 * rand(T, C)).to(ht)
    w = (1 + 0.2 * rand(C)).to(wt)
    rstd = ns.mx_rms_norm(h, w, rstd=True).rstd
    r = rstd.double()[:, None]
    u, G = h.double() * r, dy.double() * w.double()
    m, size = (G * u).mean(1, keepdim=True), (G * u).abs().mean(1, keepdim=True)
    dh = r * (G - u * m)
    # products of up to four roundings, and a row's sum of depth 70: 32 values a
    # lane, a wave's tree and up to 16 waves
    bound = r * (6 * U * (G.abs() + u.abs() * size) + 75 * U * u.abs() * size)
    dw = (dy.double() * u).sum(0)
    bw = weight_depth(T, C) * U * (dy.double() * u).abs().sum(0)
    near = lambda got, want, b: bool(((got.double() - want).abs() <= b).all())  # noqa: E731
    a = ns.mx_rms_norm_backward(dy, h, rstd, w)
    assert near(a.dh, dh, bound + HALF[ht] * (dh.abs() + bound))
    assert near(a.dw, dw, bw)
    b = ns.mx_rms_norm_backward(dy, h, rstd, w)
    assert torch.equal(a.dh, b.dh) and torch.equal(a.dw, b.dw)
    rng = torch.tensor([T, C], dtype=torch.int64, device=DEV)
    f = ns.mx_dropout(torch.ones(T, C, device=DEV), 0.25, rng).double()
    acc, stream = torch.full((C,), 0.5, device=DEV), din.clone()
    c = ns.mx_rms_norm_backward(dy, h, rstd, w, dh=stream, out=stream, drop=0.25, rng=rng, dw=acc, beta=2.0)
    want = din.double() + dh
    bound = bound + U * want.abs()
    assert c.dh is stream and near(stream, want, bound + HALF[ht] * (want.abs() + bound))
    assert near(c.dx, f * want, f * (bound + U * want.abs()) + HALF[xt] * f * (want.abs() + bound))
    assert c.dw is acc and near(acc, dw + 1.0, bw + U * (dw.abs() + 1.0))


@pytest.mark.parametrize("T,C", [(50000, 24), (3500, 700), (800, 4099), (600, 8200), (520, 32768)])
def test_a_row_without_values_among_many(T, C):
    """A NaN or an infinity in one row stays there, and in its own columns of dw."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    h, dy, w = torch.randn(T, C, generator=g, device=DEV), torch.randn(T, C, generator=g, device=DEV), torch.ones(C, device=DEV)
    clean = ns.mx_rms_norm_backward(dy, h, ns.mx_rms_norm(h, w, rstd=True).rstd, w)
    at = T - 2
    dy[at, C // 2] = float("nan")
    got = ns.mx_rms_norm_backward(dy, h, ns.mx_rms_norm(h, w, rstd=True).rstd, w)
    rest = torch.arange(T, device=DEV) != at
    assert torch.isnan(got.dh[at]).all() and torch.equal(got.dh[rest], clean.dh[rest])
    bad = torch.isnan(got.dw)
    assert bool(bad[C // 2]) and int(bad.sum()) == 1 and torch.equal(got.dw[~bad], clean.dw[~bad])
