"""What 16-bit Newton–Schulz rounds and what it puts back, against float64."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host  # noqa: E402

QUINTIC = (3.4445, -4.7750, 2.0315)
U16, U32 = 2.0 ** -11, 2.0 ** -24


def _dev(a, ty=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(ty).to(DEV)


def _hadamard(n):
    h = np.ones((1, 1))
    while len(h) < n:
        h = np.block([[h, h], [h, -h]])
    return h


# ---- rows whose diagonal of B all but cancels --------------------------------

@pytest.mark.parametrize("m,n", [(2, 64), (64, 2), (62, 300), (256, 512), (512, 256), (300, 600), (600, 300), (1000, 1100)])
def test_a_vanishing_diagonal_of_b_leaves_its_row_alone(m, n):
    """Coefficients of the caller's choice may make B_ii as small as they like
    next to B's other entries, which carry the row.

    Rows of equal norm in correlated pairs, A_ii = 1 / m; with (a, b, c) =
    (1 / m + eps, -1, 0), B_ii = eps, a subnormal of f16, and B_ij = -A_ij."""
    k, kn = min(m, n), max(m, n)
    size = 1 << (kn.bit_length() - 1)
    G = np.zeros((k, kn))
    G[0::2, :size] = _hadamard(size)[0:k:2]
    G[1::2, :size] = G[0::2, :size] * np.where(np.arange(size) % 8 < 2, -1, 1)     # half of the pair's norm in common
    assert np.all((G ** 2).sum(1) == (G[0] ** 2).sum())
    X = G / np.linalg.norm(G)
    A = X @ X.T
    assert np.allclose(np.diag(A), 1 / k, rtol=1e-12)
    for eps in (1.0e-7, 1.5e-7, 2.1e-7, 3.3e-7):
        a = float(np.float32(1 / k + eps))
        B = a * np.eye(k) - A
        want = B @ X
        # X_0 holds its values exactly; A and B round once (subnormals step by
        # 2^-24), sums are FP32, A's diagonal to a few roundings of it
        dA = U16 * np.abs(A) + 2.0 ** -25
        np.fill_diagonal(dA, 8 * U32 * np.diag(A) + 2.0 ** -25)
        dB = dA + U16 * (np.abs(B) + dA) + 2.0 ** -25
        tol = dB @ np.abs(X) + (k + 16) * U32 * (np.abs(B) @ np.abs(X))
        src = G if m <= n else G.T
        got = host(ns.ns_orthogonalize_f16(_dev(src), [(a, -1.0, 0.0)]))
        got = got if m <= n else got.T
        assert np.all(np.abs(got - want) <= tol + U32 * np.abs(want)), (eps, float(np.max(np.abs(got - want) / (tol + 1e-45))))
