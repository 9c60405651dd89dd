"""The norm with residual and dropout, its gradients and dropout by itself,
against float64 on the host.

Tolerances count roundings.  One FP32 rounding is off by at most 2^-24, the
rounding to an output type by its half step (2^-8 BF16)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402
from oracle import layer as L  # noqa: E402
from oracle import mxfp4 as M4  # noqa: E402

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def heavy(seed, rows, cols, dtype, scale=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_t(3, (rows, cols)) * scale
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)


def weight(seed, cols, dtype):
    g = np.random.default_rng(seed)
    return torch.from_numpy((1 + 0.2 * g.standard_normal(cols)).astype(np.float32)).to(dtype).to(DEV)


def f64(t):
    return host(t).astype(np.float64)


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


def check_rstd(rstd, h):
    want = L.rms(f64(h), EPS)
    assert np.all(np.abs(f64(rstd) - want) <= 1.001 * U * want)


def y32(h, rstd, w):
    """y as defined: two FP32 products."""
    return (host(h).astype(np.float32) * host(rstd).astype(np.float32)[:, None]) * host(w).astype(np.float32)


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 256), (4, 257), (33, 512), (9, 513), (2, 1024), (7, 1111), (300, 2048), (6, 2049),
          (3, 4099), (2, 8192), (2, 8200), (3, 11008), (2, 16384), (1, 20001), (2, 32768)]


@pytest.mark.parametrize("types", ["f32 f32 f32", "bf16 bf16 bf16", "bf16 f32 bf16", "f32 bf16 f32", "bf16 bf16 f32"])
@pytest.mark.parametrize("T,C", SHAPES)
def test_forward(T, C, types):
    xt, ht, wt = (TYPES[t] for t in types.split())
    x, r, w = heavy(1, T, C, xt, 0.3), heavy(2, T, C, ht), weight(3, C, wt)
    n = ns.mx_rms_norm(x, w, EPS, residual=r, y=True, mxfp8=True, mxfp4=True, kept=True, rstd=True)
    h64 = f64(r) + f64(x)
    assert n.h.dtype == ht and np.all(np.abs(f64(n.h) - h64) <= (HALF[ht] + U) * np.abs(h64))
    check_rstd(n.rstd, n.h)
    y = y32(n.h, n.rstd, w)
    assert n.y.dtype == xt
    # y is one rounding (to its type) from the FP32 product
    assert torch.equal(n.y.cpu(), torch.from_numpy(y).to(xt))
    want = L.norm(f64(n.h), f64(w), EPS)
    assert np.all(np.abs(y - want) <= 3.01 * U * np.abs(want))
    for got, (codes, scales) in ((n.mxfp8, L.mx8_quantize(y)), (n.mxfp4, M4.quantize(y)), (n.kept, M4.quantize(y.T))):
        assert np.array_equal(host(got[0]), codes) and np.array_equal(host(got[1]), scales)


@pytest.mark.parametrize("T,C", [(1, 4096), (5, 333), (70, 1111), (2, 16384)])
@pytest.mark.parametrize("types", ["f32 f32", "bf16 bf16", "bf16 f32"])
@pytest.mark.parametrize("p", [0.1, 0.5, 0.999])
def test_forward_with_dropout(T, C, types, p):
    xt, ht = (TYPES[t] for t in types.split())
    x, r, w = heavy(1, T, C, xt, 0.3), heavy(2, T, C, ht), weight(3, C, xt)
    seed, offset = -0x123456789ABCDEF, (7 << 40) + 3
    n = ns.mx_rms_norm(x, w, EPS, residual=r, drop=p, rng=rng_of(seed, offset), y=True, rstd=True)
    f = L.drop_factors(T, C, p, seed, offset)
    h64 = f64(r) + f * f64(x)
    assert np.all(np.abs(f64(n.h) - h64) <= (HALF[ht] + U) * np.abs(h64))
    assert np.array_equal(f64(n.h)[f == 0], f64(r)[f == 0])
    check_rstd(n.rstd, n.h)
    assert torch.equal(n.y.cpu(), torch.from_numpy(y32(n.h, n.rstd, w)).to(xt))
    # without a residual the dropped branch is the stream
    m = ns.mx_rms_norm(x, w, EPS, drop=p, rng=rng_of(seed, offset))
    assert torch.equal(m.h, ns.mx_dropout(x, p, rng_of(seed, offset)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(1, 1), (3, 5), (1, 4096), (64, 1111), (5, 16384), (2, 32768)])
def test_without_residual(T, C, dtype):
    x, w = heavy(4, T, C, TYPES[dtype]), weight(5, C, TYPES[dtype])
    n = ns.mx_rms_norm(x, w, EPS, rstd=True)
    assert n.h is x and n.mxfp8 is None and n.kept is None
    check_rstd(n.rstd, x)
    assert torch.equal(n.y.cpu(), torch.from_numpy(y32(x, n.rstd, w)).to(x.dtype))
    o = ns.mx_rms_norm(x, w, EPS, mxfp8=True)
    assert o.y is None and np.array_equal(host(o.mxfp8[0]), L.mx8_quantize(y32(x, n.rstd, w))[0])


def test_rows_without_values():
    """Zero rows, infinities, NaN, and numbers whose squares leave FP32."""
    C = 600
    x = torch.zeros(6, C, device=DEV)
    x[1, 5] = float("inf")
    x[2, 300] = float("nan")
    x[3] = 1e30
    x[4] = 1e-30
    x[5, 0] = -0.0
    w = torch.ones(C, device=DEV)
    n = ns.mx_rms_norm(x, w, EPS, y=True, mxfp8=True, mxfp4=True, kept=True, rstd=True)
    y = host(n.y)
    assert not y[0].any() and np.signbit(y[5, 0]) and not y[5].any()
    assert np.isnan(y[1, 5]) and not np.delete(y[1], 5).any()
    assert np.isnan(y[2]).all()
    assert np.all(np.abs(y[3] - 1.0) <= 3 * U)
    want = L.norm(f64(x)[4:5], np.ones(C), EPS)[0]
    assert np.all(np.abs(y[4] - want) <= 4 * U * want)
    full = y32(x, n.rstd, w)
    for got, (codes, scales) in ((n.mxfp8, L.mx8_quantize(full)), (n.mxfp4, M4.quantize(full)), (n.kept, M4.quantize(full.T))):
        assert np.array_equal(host(got[0]), codes) and np.array_equal(host(got[1]), scales)
    # a tiny eps, whose rstd is huge: what lies behind the row's end stays out
    z = ns.mx_rms_norm(torch.zeros(2, 33, device=DEV), torch.ones(33, device=DEV), 1e-40, mxfp8=True, y=True)
    assert not host(z.y).any() and not host(z.mxfp8[0]).any() and not host(z.mxfp8[1]).any()


def backward_bounds(dy, h, rstd, w, C, T):
    """Absolute bounds on dh (before its rounding) and dw: products of up to four
    FP32 roundings, sums of depth 70 along a row (32 values a lane, a wave's
    tree, up to 16 waves) and of ceil(T / 1024) + 1024 / 32 + 32 down a column."""
    u, g = np.abs(h * rstd[:, None]), np.abs(dy * w)
    m = np.mean(g * u, axis=1, keepdims=True)
    dh = rstd[:, None] * (6 * U * (g + u * m) + 75 * U * u * m)
    dw = (-(-T // 1024) + 32 + 128 + 4) * U * np.sum(np.abs(dy) * u, axis=0)
    return dh, dw


@pytest.mark.parametrize("types", ["f32 f32 f32", "bf16 bf16 bf16", "bf16 f32 bf16", "f32 bf16 f32"])
@pytest.mark.parametrize("T,C", SHAPES + [(5000, 24), (2100, 1500)])
def test_backward(T, C, types):
    xt, ht, wt = (TYPES[t] for t in types.split())
    h, w, dy, din = heavy(1, T, C, ht), weight(2, C, wt), heavy(3, T, C, xt, 1e-2), heavy(4, T, C, ht, 1e-2)
    rstd = ns.mx_rms_norm(h, w, EPS, rstd=True).rstd
    H, W, D, R = f64(h), f64(w), f64(dy), f64(rstd)
    dh, dw = L.norm_backward(D, H, W, EPS)
    bh, bw = backward_bounds(D, H, R, W, C, T)
    # without what comes by other ways
    g = ns.mx_rms_norm_backward(dy, h, rstd, w)
    assert g.dh.dtype == ht and g.dw.dtype == torch.float32 and (g.dx is g.dh) == (xt == ht) and g.dx.dtype == xt
    assert np.all(np.abs(f64(g.dh) - dh) <= bh + HALF[ht] * (np.abs(dh) + bh))
    assert np.all(np.abs(f64(g.dx) - dh) <= bh + HALF[xt] * (np.abs(dh) + bh))
    assert np.all(np.abs(f64(g.dw) - dw) <= bw)
    # with it, dropout, and an accumulated weight gradient
    p, seed, offset = 0.25, 99, 1 << 33
    f = L.drop_factors(T, C, p, seed, offset) if T * C < 200000 else None
    if f is not None:
        acc = torch.full((C,), 0.5, device=DEV)
        g = ns.mx_rms_norm_backward(dy, h, rstd, w, dh=din, drop=p, rng=rng_of(seed, offset), dw=acc, beta=2.0)
        want = f64(din) + dh
        bound = bh + U * np.abs(want)
        assert np.all(np.abs(f64(g.dh) - want) <= bound + HALF[ht] * (np.abs(want) + bound))
        assert np.all(np.abs(f64(g.dx) - f * want) <= f * (bound + U * np.abs(want)) + HALF[xt] * f * (np.abs(want) + bound))
        assert g.dw is acc and np.all(np.abs(f64(g.dw) - (dw + 1.0)) <= bw + U * (np.abs(dw) + 1.0))
    n = ns.mx_rms_norm_backward(dy, h, rstd, w, need_dw=False)
    assert n.dw is None and torch.equal(n.dh, ns.mx_rms_norm_backward(dy, h, rstd, w).dh)


def test_gradients_against_differences():
    """The formula's gradients of a sum, from differences of the GPU's own
    forward pass in FP32: steps of 2^-6 leave a cubic error of about 1e-4 and a
    rounding of 2^-24 * 20 / 2^-5."""
    T, C = 3, 40
    x, r, w, dy = heavy(1, T, C, torch.float32), heavy(2, T, C, torch.float32), weight(3, C, torch.float32), heavy(4, T, C, torch.float32)
    rng = rng_of(5, 6)
    f = lambda a, b, c: float((ns.mx_rms_norm(a, c, EPS, residual=b, drop=0.3, rng=rng).y.double() * dy.double()).sum())  # noqa: E731
    n = ns.mx_rms_norm(x, w, EPS, residual=r, drop=0.3, rng=rng, rstd=True)
    g = ns.mx_rms_norm_backward(dy, n.h, n.rstd, w, drop=0.3, rng=rng)
    step = 2.0 ** -6
    for t, c in ((0, 0), (1, 7), (2, 39), (0, 20), (1, 31)):
        e = torch.zeros(T, C, device=DEV)
        e[t, c] = step
        assert abs((f(x + e, r, w) - f(x - e, r, w)) / (2 * step) - float(g.dx[t, c])) < 3e-3
        assert abs((f(x, r + e, w) - f(x, r - e, w)) / (2 * step) - float(g.dh[t, c])) < 3e-3
        assert abs((f(x, r, w + e[t]) - f(x, r, w - e[t])) / (2 * step) - float(g.dw[c])) < 3e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(1, 1), (1, 9), (1, 4096), (700, 1), (333, 7), (257, 8), (129, 100), (50, 1501), (3, 8192),
                                 (2, 8193), (2, 20000)])
def test_dropout(T, C, dtype):
    x = heavy(1, T, C, TYPES[dtype])
    seed, offset = (1 << 62) + 12345, -5
    for p in (0.0, 0.1, 0.5, 0.9999):
        f = L.drop_factors(T, C, p, seed, offset)
        want = torch.from_numpy(host(x).astype(np.float32) * f.astype(np.float32)).to(x.dtype)
        got = ns.mx_dropout(x, p, rng_of(seed, offset)).cpu()
        assert torch.equal(got, want)
    y = x.clone()
    assert ns.mx_dropout(y, 0.5, rng_of(seed, offset), out=y) is y
    assert torch.equal(y, ns.mx_dropout(x, 0.5, rng_of(seed, offset)))


def test_dropped_values_are_zero_whatever_they_were():
    x = torch.full((8, 256), float("nan"), device=DEV)
    y = host(ns.mx_dropout(x, 0.5, rng_of(1, 2)))
    f = L.drop_factors(8, 256, 0.5, 1, 2)
    assert np.isnan(y[f != 0]).all() and not y[f == 0].any()


def test_in_place_and_given_outputs():
    T, C = 40, 700
    x, r, w = heavy(1, T, C, torch.bfloat16), heavy(2, T, C, torch.bfloat16), weight(3, C, torch.bfloat16)
    a = ns.mx_rms_norm(x, w, EPS, residual=r, mxfp8=True, mxfp4=True, kept=True, rstd=True, y=True)
    stream = r.clone()
    given = dict(y=torch.empty(T, C, device=DEV), mxfp8=tuple(torch.empty_like(t) for t in a.mxfp8),
                 mxfp4=tuple(torch.empty_like(t) for t in a.mxfp4), kept=tuple(torch.empty_like(t) for t in a.kept),
                 rstd=torch.empty(T, device=DEV))
    flat = [stream, given["y"], given["rstd"], *given["mxfp8"], *given["mxfp4"], *given["kept"]]
    before = [t._version for t in flat]
    b = ns.mx_rms_norm(x, w, EPS, residual=stream, h=stream, **given)
    assert all(t._version > v for t, v in zip(flat, before))
    assert b.h is stream and torch.equal(b.h, a.h) and torch.equal(b.rstd, a.rstd)
    assert b.y is given["y"] and torch.equal(b.y.bfloat16(), a.y)
    for p, q in ((a.mxfp8, b.mxfp8), (a.mxfp4, b.mxfp4), (a.kept, b.kept)):
        assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
    dy, din = heavy(5, T, C, torch.bfloat16), heavy(6, T, C, torch.bfloat16)
    g = ns.mx_rms_norm_backward(dy, a.h, a.rstd, w, dh=din)
    d = din.clone()
    k = ns.mx_rms_norm_backward(dy, a.h, a.rstd, w, dh=d, out=d)
    assert k.dh is d and torch.equal(d, g.dh) and torch.equal(k.dw, g.dw)


def test_graph_replays_draw_anew():
    """A captured step follows its generator's words, and replays equal eager calls."""
    T, C = 64, 1000
    x, r, w, dy = (heavy(i, T, C, torch.bfloat16) for i in (1, 2, 3, 4))
    w = weight(3, C, torch.bfloat16)
    rng = rng_of(11, 0)

    def step():
        n = ns.mx_rms_norm(x, w, EPS, residual=r, drop=0.2, rng=rng, mxfp4=True, kept=True, rstd=True)
        g = ns.mx_rms_norm_backward(dy, n.h, n.rstd, w, drop=0.2, rng=rng)
        return [n.h, *n.mxfp4, *n.kept, g.dh, g.dx, g.dw, ns.mx_dropout(x, 0.2, rng)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    seen = []
    for k in range(4):
        rng[1] = k % 3
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        seen.append(outs[0].clone())
    assert not torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[3])


def test_other_streams():
    T, C = 128, 4096
    x, r, w = heavy(1, T, C, torch.bfloat16), heavy(2, T, C, torch.bfloat16), weight(3, C, torch.bfloat16)
    want = ns.mx_rms_norm(x, w, EPS, residual=r, y=True, kept=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [ns.mx_rms_norm(x, w, EPS, residual=r, y=True, kept=True, stream=s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g.y, want.y) and torch.equal(g.kept[0], want.kept[0]) and torch.equal(g.h, want.h)


NARROW = [(1, 2), (37, 8), (300, 9), (65, 40), (33, 63), (64, 64), (31, 65), (300, 100), (17, 127), (16, 128), (15, 129), (9, 200), (70, 255), (8, 256)]


@pytest.mark.parametrize("types", ["f32 f32 f32", "bf16 f32 bf16"])
@pytest.mark.parametrize("T,C", NARROW)
def test_several_rows_a_wave(T, C, types):
    """Widths around 64, 128 and 256, the last workgroup part full."""
    test_forward(T, C, types)
    test_forward_with_dropout(T, C, " ".join(types.split()[:2]), 0.25)
    test_backward(T, C, types)


@pytest.mark.parametrize("T,C", [(1, 9), (300, 15), (7, 63), (300, 257), (7, 1001), (300, 2049), (7, 4095), (2, 8195), (1, 20001)])
def test_in_place_at_widths_that_end_inside_eight(T, C):
    """The residual stream and its gradient overwritten: what is written is what
    apart tensors hold, bit for bit."""
    x, r, w = heavy(1, T, C, torch.bfloat16), heavy(2, T, C, torch.float32), weight(3, C, torch.bfloat16)
    apart = ns.mx_rms_norm(x, w, EPS, residual=r, y=True, rstd=True, mxfp8=True)
    h = r.clone()
    n = ns.mx_rms_norm(x, w, EPS, residual=h, h=h, y=True, rstd=True, mxfp8=True)
    assert n.h is h and torch.equal(h, apart.h) and torch.equal(n.y, apart.y) and torch.equal(n.mxfp8[0], apart.mxfp8[0])
    dy, dh = heavy(4, T, C, torch.bfloat16), heavy(5, T, C, torch.float32)
    a = ns.mx_rms_norm_backward(dy, h, n.rstd, w, dh=dh)
    b = ns.mx_rms_norm_backward(dy, h, n.rstd, w, dh=dh, out=dh)
    assert b.dh is dh and torch.equal(a.dh, dh) and torch.equal(a.dx, b.dx) and torch.equal(a.dw, b.dw)
