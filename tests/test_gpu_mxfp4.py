"""MXFP4 on the GPU against the float64 oracle: codes and scales byte for
byte, products within the rounding of FP32 sums, the linear layer's gradients
against the formula and against differences."""
import numpy as np
import pytest
import torch

import synth
from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
U32 = 2.0 ** -24
U16 = 2.0 ** -8


def _x(rows, cols, seed, ty):
    """Heavy-tailed values over many binades, with zeros of both signs."""
    x = synth.student_t(rows, cols, seed) if rows * cols >= 1000 else synth.gaussian(rows, cols, seed)
    g = synth.rng(seed + 1)
    x = x * np.exp2(g.integers(-6, 7, size=(rows, 1))).astype(np.float32)
    x[g.random((rows, cols)) < 0.02] = 0.0
    x[g.random((rows, cols)) < 0.02] = -0.0
    t = torch.from_numpy(x.astype(np.float32)).to(TYPES[ty])
    return t.to(DEV), t.double().numpy()


def _dev(q):
    return tuple(torch.from_numpy(a).to(DEV) for a in q)


def _same(got, want):
    return all(np.array_equal(host(g), w) for g, w in zip(got, want))


SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (1, 255), (5, 256), (7, 257), (31, 8), (32, 40), (33, 512),
          (255, 130), (256, 128), (257, 129), (300, 700), (65, 1024), (1000, 18)]


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_matches_oracle(rows, cols, ty):
    x, xv = _x(rows, cols, rows * 1000 + cols, ty)
    along, down = O.quantize(xv), O.quantize(xv.T)
    assert _same(ns.mxfp4_quantize(x, ns.NVFP4_ROWS), along)
    assert _same(ns.mxfp4_quantize(x, ns.NVFP4_COLS), down)
    a, d = ns.mxfp4_quantize_both(x)
    assert _same(a, along) and _same(d, down)
    for ot, name in ((ns.NS_F32, "f32"), (ns.NS_BF16, "bf16")):
        for q, axis in ((along, ns.NVFP4_ROWS), (down, ns.NVFP4_COLS)):
            v = O.dequantize(*q, cols if axis == ns.NVFP4_ROWS else rows)
            v = v if axis == ns.NVFP4_ROWS else v.T
            got = host(ns.mxfp4_dequantize(*_dev(q), rows, cols, axis, ot))
            assert np.array_equal(got, v) and np.array_equal(np.signbit(got), np.signbit(v)), (axis, name)


@pytest.mark.parametrize("axis", [0, 1])
def test_nothing_is_written_behind_the_outputs(axis):
    rows, cols = 33, 70
    x, _ = _x(rows, cols, 5, "f32")
    r, c = (rows, cols) if axis == 0 else (cols, rows)
    codes = torch.full((r * 128 * O.panels(c) + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((r * 8 * O.panels(c) + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    ns.mxfp4_quantize(x, axis, codes=codes, scales=scales)
    assert (host(codes)[-64:] == 0xA5).all() and (host(scales)[-64:] == 0xA5).all()
    out = torch.full((rows * cols + 64,), 7.0, device=DEV)
    ns.mxfp4_dequantize(codes, scales, rows, cols, axis, out=out)
    assert (host(out)[-64:] == 7.0).all()


def test_quantize_extremes():
    """Midpoints and their neighbours at every binade, subnormals, the largest
    values, blocks of zeros, NaN and infinities (one per block)."""
    mags = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float32)
    near = np.concatenate((mags, np.nextafter(mags, np.float32(0)), np.nextafter(mags, np.float32(9))))
    rows = []
    for e in list(range(-149, -120)) + [-60, -1, 0, 1, 60, 124, 125]:
        row = np.zeros(32, np.float64)
        row[:27] = near * 2.0 ** min(e, 125)
        row[27] = 4.0 * 2.0 ** e if e < 126 else 0.0
        rows.append(row)
    rows += [np.zeros(32), -np.zeros(32), np.full(32, 3.4e38)]
    for bad in (np.nan, np.inf, -np.inf):
        row = np.linspace(-1, 1, 32)
        row[11] = bad
        rows.append(row)
    with np.errstate(over="ignore"):
        x = np.array(rows).astype(np.float32)
    x = x[~np.isinf(x).any(1) | (np.isinf(x).sum(1) == 1)]
    t = torch.from_numpy(x).to(DEV)
    want = O.quantize(x.astype(np.float64))
    assert _same(ns.mxfp4_quantize(t), want)
    a, d = ns.mxfp4_quantize_both(t)
    assert _same(a, want) and _same(d, O.quantize(x.astype(np.float64).T))
    assert _same(ns.mxfp4_quantize(t.t().contiguous(), ns.NVFP4_COLS), want)
    for ot in (ns.NS_F32, ns.NS_BF16):
        got = host(ns.mxfp4_dequantize(*_dev(want), *x.shape, out_dtype=ot))
        assert np.array_equal(got, O.dequantize(*want, 32), equal_nan=True)


# every tile size, its edges one less and one more, K inside and across panels
GEMM = [(1, 1, 1), (1, 64, 256), (17, 33, 100), (63, 65, 257), (64, 64, 512), (65, 130, 1000), (5, 700, 300),
        (128, 128, 256), (255, 300, 511), (256, 257, 768), (300, 1000, 1024), (513, 384, 2000),
        (1024, 1024, 256), (1025, 1100, 1300), (1300, 1027, 513), (2048, 1536, 300), (16, 4096, 4096), (1, 1000, 2100)]


def _bound(pv, qv, K):
    """FP32 accumulation of exact products: at most K roundings of partial
    sums, each of which is at most the sum of magnitudes."""
    return (K + 4) * U32 * (np.abs(pv) @ np.abs(qv).T)


@pytest.mark.parametrize("M,N,K", GEMM)
def test_gemm_matches_float64(M, N, K):
    p, q = O.quantize(_x(M, K, M + K, "f32")[1]), O.quantize(_x(N, K, N + K + 1, "f32")[1])
    pv, qv = O.dequantize(*p, K), O.dequantize(*q, K)
    want, tol = pv @ qv.T, _bound(pv, qv, K)
    for split in (True, False):
        got = host(ns.mxfp4_gemm(_dev(p), _dev(q), M, N, K, split=split))
        assert np.all(np.abs(got - want) <= tol), (split, float(np.max(np.abs(got - want) / (tol + 1e-300))))
    add = synth.gaussian(M, N, 3)
    out = torch.from_numpy(add).to(DEV)
    ns.mxfp4_gemm(_dev(p), _dev(q), M, N, K, alpha=-0.5, beta=2.0, addend=out, out=out)      # in place
    w = 2.0 * add - 0.5 * want
    assert np.all(np.abs(host(out) - w) <= 0.5 * tol + 4 * U32 * (np.abs(w) + np.abs(2.0 * add) + np.abs(want)))
    b = host(ns.mxfp4_gemm(_dev(p), _dev(q), M, N, K, out_dtype=ns.NS_BF16))
    assert np.all(np.abs(b - want) <= tol + U16 * (np.abs(want) + tol))


# 64-, 128- and 256-wide tiles over several rounds of workgroups, and each with
# leftover tiles split along K
LARGE = [(330, 330, 5000), (200, 1760, 5000), (2100, 2050, 2100), (2410, 3450, 2000), (2020, 4100, 2000),
         (8190, 4090, 300), (3970, 4100, 5000)]


@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_gemm_matches_float64(M, N, K):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(M + N + K)
    p = ns.mxfp4_quantize(torch.randn(M, K, generator=gen, device=DEV))
    q = ns.mxfp4_quantize(torch.randn(N, K, generator=gen, device=DEV))
    pv, qv = (ns.mxfp4_dequantize(*t, r, K).double() for t, r in ((p, M), (q, N)))
    want = pv @ qv.t()
    tol = (K + 4) * U32 * (pv.abs() @ qv.abs().t())
    first = ns.mxfp4_gemm(p, q, M, N, K)
    for split in (True, False):
        assert bool(((ns.mxfp4_gemm(p, q, M, N, K, split=split) - want).abs() <= tol).all()), split
    add = torch.randn(M, N, generator=gen, device=DEV)
    got = ns.mxfp4_gemm(p, q, M, N, K, beta=0.5, addend=add, out_dtype=ns.NS_BF16)
    w = want + 0.5 * add.double()
    assert bool(((got - w).abs() <= tol + 4 * U32 * (want.abs() + add.abs()) + U16 * (w.abs() + tol)).all())
    assert torch.equal(ns.mxfp4_gemm(p, q, M, N, K), first)          # the same bits every time


def test_offsets_past_32_bits():
    rows, cols = 70000, 32768                                        # 2.3e9 elements
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    for r in range(0, rows, 10000):
        x[r:r + 10000] = torch.randn(10000, cols, generator=gen, device=DEV).to(torch.bfloat16)
    along, down = ns.mxfp4_quantize_both(x)
    assert all(torch.equal(a, b) for a, b in zip(ns.mxfp4_quantize(x), along))
    tail = ns.mxfp4_quantize(x[-300:].contiguous())
    assert torch.equal(along[0][:, -300:], tail[0]) and torch.equal(along[1][:, -300:], tail[1])
    tail = ns.mxfp4_quantize(x[:, -200:].contiguous(), ns.NVFP4_COLS)
    assert torch.equal(down[0][:, -200:], tail[0]) and torch.equal(down[1][:, -200:], tail[1])
    v = ns.mxfp4_dequantize(*along, rows, cols, out_dtype=ns.NS_BF16)
    assert torch.equal(v[-300:], ns.mxfp4_dequantize(*(t[:, -300:].contiguous() for t in along), 300, cols,
                                                     out_dtype=ns.NS_BF16))
    del v, along, down
    K, N = 64, 33000
    p = ns.mxfp4_quantize(x[:, :K].contiguous())
    q = ns.mxfp4_quantize(torch.randn(N, K, generator=gen, device=DEV))
    y = ns.mxfp4_gemm(p, q, rows, N, K, out_dtype=ns.NS_BF16)        # 2.3e9 elements too
    few = ns.mxfp4_gemm(tuple(t[:, -300:].contiguous() for t in p), q, 300, N, K, out_dtype=ns.NS_BF16)
    assert torch.equal(y[-300:], few)


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own do not meet."""
    T, N, K = 1100, 1024, 9000
    x = [_x(T, K, s, "bf16")[0] for s in (1, 2)]
    w = ns.mxfp4_quantize(_x(N, K, 3, "f32")[0])
    want = [ns.mxfp4_linear(v, w, N) for v in x]
    streams = [torch.cuda.Stream() for _ in x]
    got = [torch.empty_like(v) for v in want]
    wss = [torch.empty(ns.mxfp4_linear_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV) for _ in x]
    torch.cuda.synchronize()
    for _ in range(3):
        for v, o, ws, s in zip(x, got, wss, streams):
            ns.mxfp4_linear(v, w, N, out=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tensors_that_a_call_makes_belong_to_its_stream():
    """With `stream` given and nothing else, the call's own workspace and
    outputs are not handed to the current stream's work while it runs."""
    T, N, K = 700, 640, 2048
    x = torch.randn(T, K, device=DEV)
    w = ns.mxfp4_quantize(torch.randn(N, K, device=DEV))
    dy = torch.randn(T, N, device=DEV)
    wt = ns.mxfp4_quantize(torch.randn(N, K, device=DEV), ns.NVFP4_COLS)
    G = torch.randn(300, 700, device=DEV)
    calls = [lambda s: ns.mxfp4_linear(x, w, N, keep=True, stream=s), lambda s: ns.mxfp4_quantize_both(x, stream=s),
             lambda s: ns.mxfp4_linear_backward(dy, wt, kept, K, stream=s),
             lambda s: ns.ns_orthogonalize_f16(G, [(3.4445, -4.775, 2.0315)] * 5, stream=s)]
    kept = ns.mxfp4_linear(x, w, N, keep=True)[1]
    flat = lambda v: [v] if isinstance(v, torch.Tensor) else [t for u in v for t in flat(u)]
    want = [flat(c(None)) for c in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, noise = [], []
    for _ in range(6):
        for c in calls:
            got.append(flat(c(side)))
            # the current stream's memory, in the sizes that the call has used
            noise = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in (1 << 20, 4 << 20, 1 << 22)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(calls)])), i
    assert all(bool((n == 0xFF).all()) for n in noise)


def test_binding_refuses():
    x = torch.randn(64, 96, device=DEV)
    q = ns.mxfp4_quantize(x)
    with pytest.raises(ValueError):
        ns.mxfp4_quantize(x.t())                                     # not contiguous
    with pytest.raises(ValueError):
        ns.mxfp4_quantize(x[0])                                      # not a matrix
    with pytest.raises(ValueError):
        ns.mxfp4_quantize(x, codes=q[0][:, :32].contiguous())        # too short
    with pytest.raises(TypeError):
        ns.mxfp4_quantize(x.half())
    with pytest.raises(ValueError):
        ns.mxfp4_gemm(q, q, 64, 64, 300)                             # K past the panels
    with pytest.raises(ValueError):
        ns.mxfp4_gemm(q, q, 64, 64, 96, beta=1.0, addend=torch.zeros(64, 32, device=DEV))
    with pytest.raises(ValueError):
        ns.mxfp4_linear(x, q, 65)
    with pytest.raises(ValueError):
        ns.mxfp4_linear(x, (q[0].cpu(), q[1]), 64)
    with pytest.raises(ValueError):
        ns.mxfp4_linear_backward(x, q, None, 64, need_dw=False, dx=torch.empty(64, 10, device=DEV))
    with pytest.raises(ValueError):
        ns.mxfp4_linear_backward(x, q, q, 64, beta=1.0)              # adds to nothing


def test_gemm_nan_blocks_meet_their_rows_and_columns_only():
    p, q = O.quantize(_x(70, 600, 1, "f32")[1]), O.quantize(_x(90, 600, 2, "f32")[1])
    p[1][1, 13, 2] = 255
    q[1][0, 77, 5] = 255
    got = host(ns.mxfp4_gemm(_dev(p), _dev(q), 70, 90, 600))
    nan = np.zeros((70, 90), bool)
    nan[13, :] = nan[:, 77] = True
    assert np.array_equal(np.isnan(got), nan)


def test_gemm_writes_only_its_output():
    M, N, K = 70, 67, 300
    p, q = _dev(O.quantize(_x(M, K, 1, "f32")[1])), _dev(O.quantize(_x(N, K, 2, "f32")[1]))
    for ty in (torch.float32, torch.bfloat16):
        out = torch.full((M * N + 256,), 3.0, dtype=ty, device=DEV)
        ns.mxfp4_gemm(p, q, M, N, K, out=out)
        assert (host(out)[-256:] == 3.0).all()


LINEAR = [(1, 64, 64), (1, 513, 300), (3, 100, 777), (16, 300, 1024), (17, 96, 513), (33, 1000, 256), (64, 40, 2048),
          (100, 257, 129), (700, 384, 640), (1030, 1100, 520)]


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear_and_its_gradients_match_the_formula(T, N, K, ty):
    x, xv = _x(T, K, T + N, ty)
    dy, dyv = _x(T, N, T + K, ty)
    w = 0.05 * synth.gaussian(N, K, N)
    wq, wtq = O.quantize(w), O.quantize(w.T)
    u = U16 if ty == "bf16" else U32
    y = host(ns.mxfp4_linear(x, _dev(wq), N))
    y2, kept = ns.mxfp4_linear(x, _dev(wq), N, keep=True)
    xr, xc, wv, wtv = O.held(xv), O.held(xv.T), O.dequantize(*wq, K), O.dequantize(*wtq, N)
    want, tol = xr @ wv.T, _bound(xr, wv, K)
    assert np.all(np.abs(y - want) <= tol + u * (np.abs(want) + tol))
    assert np.all(np.abs(host(y2) - want) <= tol + u * (np.abs(want) + tol))
    assert _same(kept, O.quantize(xv.T))
    dx, dw = ns.mxfp4_linear_backward(dy, _dev(wtq), kept, K)
    dr, dc = O.held(dyv), O.held(dyv.T)
    want, tol = dr @ wtv.T, _bound(dr, wtv, N)
    assert np.all(np.abs(host(dx) - want) <= tol + u * (np.abs(want) + tol))
    want, tol = dc @ xc.T, _bound(dc, xc, T)
    assert np.all(np.abs(host(dw) - want) <= tol + u * (np.abs(want) + tol))
    # one at a time, and added to an FP32 gradient
    only_dx, none = ns.mxfp4_linear_backward(dy, _dev(wtq), None, K, need_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    acc0 = synth.gaussian(N, K, 9)
    acc = torch.from_numpy(acc0).to(DEV)
    none, _ = ns.mxfp4_linear_backward(dy, None, kept, K, dw=acc, need_dx=False, beta=1.0)
    w2 = acc0 + want
    assert none is None and np.all(np.abs(host(acc) - w2) <= tol + 4 * U32 * (np.abs(acc0) + np.abs(want)))


def test_linear_gradients_match_differences():
    """On inputs that MXFP4 holds exactly, along both axes and after the
    differences' steps, the layer is linear: central differences of
    sum(y * dy) are its gradient up to the rounding of FP32."""
    g = synth.rng(3)
    T, N, K = 32, 32, 64
    x = g.choice([-2.0, -1.0, 1.0, 2.0], size=(T, K))
    w = g.choice([-2.0, -1.0, 1.0, 2.0], size=(N, K))
    dy = g.choice([-2.0, -1.0, -0.5, 0.5, 1.0, 2.0], size=(T, N))
    x[:, ::8] = w[:, ::8] = 4.0           # every block's scale stays 1 with steps of 1 below 4
    x[::8] = w[::8] = 4.0
    dy[:, ::8] = dy[::8] = 4.0
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)  # noqa: E731

    def loss(xx, ww):
        return float((host(ns.mxfp4_linear(dev(xx), ns.mxfp4_quantize(dev(ww)), N)) * dy).sum())

    _, kept = ns.mxfp4_linear(dev(x), ns.mxfp4_quantize(dev(w)), N, keep=True)
    dx, dw = ns.mxfp4_linear_backward(dev(dy), ns.mxfp4_quantize(dev(w), ns.NVFP4_COLS), kept, K)
    for i, j in [(1, 1), (5, 33), (31, 63), (2, 10)]:
        for v, grad in ((x, host(dx)), (w, host(dw))):
            hi, lo = v.copy(), v.copy()
            step = 1.0 if abs(v[i, j]) == 2.0 else 0.5
            hi[i, j] += step
            lo[i, j] -= step
            d = (loss(hi, w) - loss(lo, w) if v is x else loss(x, hi) - loss(x, lo)) / (2 * step)
            assert d == grad[i, j], (i, j, d, grad[i, j])


def test_operators_on_another_stream_and_in_a_graph():
    """Quantize, multiply and differentiate as one captured run, replayed with
    other inputs and with eager work in between."""
    T, N, K = 130, 200, 300
    w = torch.from_numpy(0.1 * synth.gaussian(N, K, 1)).to(DEV)
    x = torch.empty(T, K, device=DEV, dtype=torch.bfloat16)
    dy = torch.empty(T, N, device=DEV, dtype=torch.bfloat16)
    wq, wt = ns.mxfp4_quantize_both(w)
    y = torch.empty(T, N, device=DEV, dtype=torch.bfloat16)
    kept = (torch.empty(O.panels(T), K, 128, dtype=torch.uint8, device=DEV),
            torch.empty(O.panels(T), K, 8, dtype=torch.uint8, device=DEV))
    dx, dw = torch.empty(T, K, device=DEV), torch.empty(N, K, device=DEV)
    w1 = torch.empty(ns.mxfp4_linear_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    w2 = torch.empty(ns.mxfp4_linear_backward_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)

    def run():
        ns.mxfp4_linear(x, wq, N, out=y, kept=kept, workspace=w1)
        ns.mxfp4_linear_backward(dy, wt, kept, K, dx=dx, dw=dw, workspace=w2)

    def fill(seed):
        x.copy_(_x(T, K, seed, "bf16")[0])
        dy.copy_(_x(T, N, seed + 50, "bf16")[0])

    side = torch.cuda.Stream()
    fill(1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (2, 3, 4):
        fill(seed)
        run()
        want = [host(t).copy() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host(t), v) for t, v in zip((y, dx, dw), want)), seed
