"""The linear layer on NVFP4 weights against float64 sums of the weights'
values.  BF16 rows: every product is exact, K - 1 FP32 additions, the global
scale's product and the output's rounding; FP32 rows come in three parts, whose
products and sums are three times as many."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402
from oracle import nvfp4 as Q  # noqa: E402

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def weights(seed, N, K):
    """(operand, float64 values): codes of any N, from the oracle's quantizer of
    a padded matrix."""
    g = np.random.default_rng(seed)
    w = np.zeros((-(-N // 16) * 16, K), np.float32)
    w[:N] = g.standard_t(3, (N, K)) * 0.02
    o = Q.quantize_rows(w)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    op = dev(o.codes[:N]), dev(o.scales[:N]), torch.tensor([float(o.global_scale)], dtype=torch.float32, device=DEV)
    return op, Q.dequantize_rows(o)[:N]


def check(y, x, w, dtype):
    X, K = host(x).astype(np.float64), x.shape[1]
    want = X @ w.T
    n = K + 3 if x.dtype == torch.bfloat16 else 3 * K + 5
    bound = n * U * (np.abs(X) @ np.abs(w).T)
    half = U if dtype == torch.float32 else 2.0 ** -8
    assert y.dtype == dtype and np.all(np.abs(host(y).astype(np.float64) - want) <= bound + half * (np.abs(want) + bound))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 16, 16), (1, 1, 16), (1, 17, 48), (2, 777, 1504), (1, 1000, 4096), (5, 33, 112), (16, 64, 128),
                                   (17, 100, 144), (31, 96, 2064), (32, 4096, 272), (33, 48, 512), (100, 20, 1040), (3, 16, 11008),
                                   (16, 9000, 160)])
def test_linear(T, N, K, dtype):
    op, w = weights(N + K, N, K)
    x = torch.from_numpy(np.random.default_rng(T).standard_t(3, (T, K)).astype(np.float32)).to(TYPES[dtype]).to(DEV)
    check(ns.nvfp4_linear(x, op, N), x, w, x.dtype)
    other = torch.bfloat16 if dtype == "f32" else torch.float32
    out = torch.full((T, N), 7.0, dtype=other, device=DEV)
    assert ns.nvfp4_linear(x, op, N, out=out) is out
    check(out, x, w, other)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 21, 70016), (2, 35, 40032), (2, 18, 2080), (3, 20, 33000 // 16 * 16)])
def test_long_rows(T, N, K, dtype):
    """More of K than LDS holds at a time, steps that end inside a wave."""
    op, w = weights(N + K, N, K)
    x = torch.from_numpy(np.random.default_rng(T).standard_t(3, (T, K)).astype(np.float32)).to(TYPES[dtype]).to(DEV)
    check(ns.nvfp4_linear(x, op, N), x, w, x.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_tokens_element_by_element(dtype):
    N, K = 18, 4128
    op, w = weights(5, N, K)
    for k in list(range(0, 66)) + list(range(2040, 2060)) + list(range(4090, K)):
        x = torch.zeros(2, K, device=DEV)
        x[0, k], x[1, K - 1 - k] = 3.0, -0.25
        y = host(ns.nvfp4_linear(x.to(TYPES[dtype]), op, N, out=torch.empty(2, N, device=DEV)))
        want = host(x).astype(np.float64) @ w.T
        assert np.all(np.abs(y - want) <= 3 * U * np.abs(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(3, 4113, 160), (5, 6001, 272), (16, 8192, 144), (33, 2100, 336), (100, 2096, 128), (40, 11000, 48), (7, 4112, 1040)])
def test_pairs_of_row_groups(T, N, K, dtype):
    """More workgroups than CUs: rows of W by 16 or 32, N that ends inside either."""
    op, w = weights(N + K, N, K)
    x = torch.from_numpy(np.random.default_rng(T).standard_t(3, (T, K)).astype(np.float32)).to(TYPES[dtype]).to(DEV)
    check(ns.nvfp4_linear(x, op, N), x, w, x.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 19, 2064), (2, 5, 2064), (1, 40, 70032), (2, 33, 40016), (1, 777, 1520), (2, 16, 48), (1, 3, 4112)])
def test_rows_that_end_inside_a_lane(T, N, K, dtype):
    """K an odd multiple of 16: random rows, then the last elements one by one."""
    op, w = weights(N + K, N, K)
    x = torch.from_numpy(np.random.default_rng(T).standard_t(3, (T, K)).astype(np.float32)).to(TYPES[dtype]).to(DEV)
    check(ns.nvfp4_linear(x, op, N), x, w, x.dtype)
    for k in range(K - 48, K):
        x = torch.zeros(T, K, device=DEV)
        x[:, k] = 3.0
        y = host(ns.nvfp4_linear(x.to(TYPES[dtype]), op, N, out=torch.empty(T, N, device=DEV)))
        want = host(x).astype(np.float64) @ w.T
        assert np.all(np.abs(y - want) <= 3 * U * np.abs(want))


def test_graph_and_streams():
    op, _ = weights(7, 100, 512)
    xs = [torch.randn(T, 512, device=DEV).bfloat16() for T in (1, 2, 5, 40)]
    want = [ns.nvfp4_linear(x, op, 100) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [ns.nvfp4_linear(x, op, 100, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [ns.nvfp4_linear(x, op, 100) for x in xs]
    for _ in range(3):
        for x in xs:
            x.normal_()
        want = [ns.nvfp4_linear(x, op, 100) for x in xs]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_weights_of_the_quantizer():
    W = torch.randn(64, 320, device=DEV)
    op = ns.nvfp4_quantize(W)
    x = torch.randn(4, 320, device=DEV)
    check(ns.nvfp4_linear(x, op, 64), x, host(ns.nvfp4_dequantize(*op, 64, 320)).astype(np.float64), torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_element_meets_its_own(dtype):
    """One element of K at a time, and the far ends of the values' range."""
    N, K = 24, 304
    op, w = weights(1, N, K)
    for k0 in range(0, K, 30):
        x = torch.zeros(30, K, device=DEV)
        n = min(30, K - k0)
        x[torch.arange(n), k0 + torch.arange(n)] = 2.0 ** torch.arange(-15, -15 + n, device=DEV).float()
        y = host(ns.nvfp4_linear(x.to(TYPES[dtype]), op, N, out=torch.empty(30, N, device=DEV)))
        want = host(x).astype(np.float64) @ w.T
        assert np.all(np.abs(y - want) <= 3 * U * np.abs(want))


def test_not_finite():
    N, K = 20, 96
    op, w = weights(2, N, K)
    x = torch.ones(5, K, device=DEV)
    x[1, 3], x[2, 95], x[3, 40] = float("nan"), float("inf"), 3e38
    live = np.abs(w) > 0
    for dtype in TYPES.values():
        y = host(ns.nvfp4_linear(x.to(dtype), op, N, out=torch.empty(5, N, device=DEV)))
        assert np.isnan(y[1]).all() and np.isfinite(y[[0, 4]]).all()
        assert np.array_equal(np.isinf(y[2]), live[:, 95]) and np.array_equal(np.isnan(y[2]), ~live[:, 95])
    bad = op[0], op[1].clone(), op[2]
    bad[1][7, 2] = 0x7F                                # E4M3's NaN: what a quantizer writes for a tensor with one
    y = host(ns.nvfp4_linear(torch.ones(2, K, device=DEV), bad, N))
    assert np.isnan(y[:, 7]).all() and np.isfinite(np.delete(y, 7, 1)).all()
