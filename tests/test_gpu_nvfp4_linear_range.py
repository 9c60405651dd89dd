"""The linear layer on NVFP4 weights at the ends of FP32's range.

Bounds as in test_gpu_nvfp4_linear.py (K + 3 roundings for BF16 rows, 3 K + 5 for
FP32 rows, relative to the sum of magnitudes), and what subnormals add: every
rounding is off by at most 2^-149 besides, and of an FP32 x what lies below
2^-133 is cut off."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402
from oracle import nvfp4 as Q  # noqa: E402

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def weights(seed, N, K, sg=None):
    """(operand, float64 values), with the global scale replaced where one is given."""
    g = np.random.default_rng(seed)
    w = np.zeros((-(-N // 16) * 16, K), np.float32)
    w[:N] = g.standard_t(3, (N, K)) * 0.02
    o = Q.quantize_rows(w)
    own = np.float32(o.global_scale)
    new = own if sg is None else np.float32(sg)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    op = dev(o.codes[:N]), dev(o.scales[:N]), torch.tensor([float(new)], dtype=torch.float32, device=DEV)
    return op, Q.dequantize_rows(o)[:N] / np.float64(own) * np.float64(new)


def check(x, op, w):
    """Finite and within the bounds, in FP32 and BF16."""
    T, K = x.shape
    X, N = host(x).astype(np.float64), w.shape[0]
    n, cut = (K + 3, 0.0) if x.dtype == torch.bfloat16 else (3 * K + 5, 2.0 ** -133)
    want, size = X @ w.T, np.abs(X) @ np.abs(w).T
    assert size.max() < 2.0 ** 127
    bound = n * (U * size + 2.0 ** -149) + cut * np.sum(np.abs(w), axis=1)
    for dtype, half in ((torch.float32, U), (torch.bfloat16, 2.0 ** -8)):
        y = host(ns.nvfp4_linear(x, op, N, out=torch.empty(T, N, dtype=dtype, device=DEV))).astype(np.float64)
        tiny = 2.0 ** (-150 if dtype == torch.float32 else -134)
        assert np.all(np.abs(y - want) <= bound + half * (np.abs(want) + bound) + tiny)


SIZES = [(1, 40, 4128), (2, 33, 2064), (1, 20, 48), (5, 100, 304), (16, 17, 4096), (17, 40, 1024), (33, 20, 112), (5, 4200, 160)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_activations_up_to_the_largest(T, N, K, dtype):
    """Sums of codes times block scales would leave FP32, the results do not."""
    op, w = weights(N + K, N, K, 1.3 * 2.0 ** -20)
    g = np.random.default_rng(T)
    x = g.standard_normal((T, K)) * 1e34
    at = g.integers(0, K, (T, 2))
    x[np.arange(T), at[:, 0]], x[np.arange(T), at[:, 1]] = 3.3e38, -3e38
    check(torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype]).to(DEV), op, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_global_scales_far_from_one(T, N, K, dtype):
    x = np.random.default_rng(T).standard_t(3, (T, K))
    for e in (-149, -140, -126, -118, -115, -60, 60, 110, 112, 116):
        for sign in (1.0, -1.0):
            op, w = weights(N + K, N, K, sign * 1.0 * 2.0 ** e)
            up = min(max(-e, -90), 90)                 # of x, so that results are ordinary numbers
            check(torch.from_numpy(np.ldexp(x, up).astype(np.float32)).to(TYPES[dtype]).to(DEV), op, w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_activations_down_to_the_smallest(T, N, K, dtype):
    op, w = weights(N + K, N, K, 1.5)
    g = np.random.default_rng(T)
    x = np.ldexp(g.standard_normal((T, K)), g.integers(-148, -96, (T, K)))
    check(torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype]).to(DEV), op, w)


@pytest.mark.parametrize("T", [1, 2, 5])
def test_a_tensor_that_held_a_nan(T):
    """The quantizer's answer to one: a global scale of NaN, scales of NaN."""
    W = torch.randn(32, 64, device=DEV)
    W[3, 5] = float("nan")
    y = ns.nvfp4_linear(torch.ones(T, 64, device=DEV), ns.nvfp4_quantize(W), 32)
    assert torch.isnan(y).all()
    zero = ns.nvfp4_quantize(torch.zeros(32, 64, device=DEV))
    assert not ns.nvfp4_linear(torch.ones(T, 64, device=DEV), zero, 32).any()
