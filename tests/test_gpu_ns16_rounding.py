"""What 16-bit Newton–Schulz rounds and what it puts back, against float64:
the factors of B's rows, the corrected diagonals, and the error by spectrum."""
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


# ---- the corrected diagonals -----------------------------------------------------

def _orthogonal_rows(k, kn, seed):
    """k orthogonal rows of kn columns, d_i times +-1 or 0, d_i integers of seven
    bits, sixteen times as large in four rows (which then hold most of A)."""
    g = np.random.default_rng(seed)
    d = g.integers(65, 128, size=k).astype(np.float64)
    d[g.permutation(k)[:4]] *= 16
    size = min(1024, 1 << (kn.bit_length() - 1))     # sums of d_i d_j stay within 24 bits
    h = _hadamard(size)
    h = h[g.permutation(size)[:k]]
    G = np.zeros((k, kn))
    G[:, np.sort(g.permutation(kn)[:size])] = h
    return d[:, None] * G, d, size


def _rows_recursion(d, size, coeffs):
    """The scale x_i of every row of X_k = x_i times its +-1, with X rounded to
    f16 behind each step but the last as the iteration does; which rows stay
    clear of ties by more than FP32's errors; the relative error allowed."""
    x = d / (np.sqrt(size * np.sum(d ** 2)) + 1e-7)
    clear = np.ones(len(d), bool)
    plain = np.zeros(len(d))                  # what uncorrected diagonals would be off by
    for it, (a, b, c) in enumerate(coeffs):
        A = size * x * x
        B = a + b * A + c * A * A
        # A: the factors t and t^2 and the scaling (6), the sum itself exact but
        # for squares of rounded values, which may lose half a unit each; B:
        # four operations on terms of these sizes, c d^2 left out; then the row's
        # factor, the product and two scalings (6)
        sums = 6 + (size / 2 if it else 0)
        half = 2.0 ** (np.floor(np.log2(A)) - 11)
        tol = U32 * (sums * (abs(b) * A + 2 * abs(c) * A * A) + 4 * (abs(a) + abs(b) * A + abs(c) * A * A)) / np.abs(B) \
            + abs(c) * half ** 2 / np.abs(B) + 6 * U32
        Ah = A.astype(np.float16).astype(np.float64)
        Bh = (a + b * Ah + c * Ah * Ah).astype(np.float16).astype(np.float64)
        plain = np.maximum(plain, np.abs(Bh / B - 1))
        x = B * x
        if it + 1 < len(coeffs):
            v = 256 * x
            step = 2.0 ** (np.floor(np.log2(v)) - 10)
            away = np.abs(v / step - np.floor(v / step) - 0.5) * step      # from the tie
            clear &= away > 2 * tol * v
            x = v.astype(np.float16).astype(np.float64) / 256
    return x, clear, tol, plain


# B made in the product (up to 256 rows) and by itself, on every tile size; the
# factors of rows and, where m > n, of columns; batches
@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,count", [(8, 8, 1), (64, 100, 1), (100, 64, 3), (256, 512, 1), (512, 256, 1), (200, 1000, 4),
                                       (300, 1000, 1), (1000, 300, 2), (512, 600, 8), (1000, 512, 4), (1000, 4100, 1),
                                       (4100, 1000, 2), (1024, 4096, 8), (2900, 1000, 8)])
@pytest.mark.parametrize("steps", [1, 2])
def test_what_f16_takes_from_the_diagonals_is_put_back(m, n, count, steps, ty):
    """Of orthogonal rows A and B are diagonal, and a row's scale is a recursion
    of its own: it holds to FP32, though f16 holds neither A_ii nor B_ii."""
    k, kn = min(m, n), max(m, n)
    coeffs = [QUINTIC] * steps
    made = [_orthogonal_rows(k, kn, 1000 * steps + i) for i in range(count)]
    src = [_dev(G if m <= n else G.T, ty) for G, _, _ in made]
    outs = ns.ns_orthogonalize_f16_grouped(src, coeffs)
    lr, W, M = 0.5, [torch.zeros(m, n, device=DEV) for _ in made], [torch.zeros(m, n, device=DEV) for _ in made]
    scales = [1.0 + i for i in range(count)]
    ns.ns_muon_step(W, M, src, coeffs, lr=lr, momentum=0.0, nesterov=False, scales=scales)
    for o, w, sc, (G, d, size) in zip(outs, W, scales, made):
        x, clear, tol, plain = _rows_recursion(d, size, coeffs)
        assert clear.mean() > 0.9 and np.max(plain / tol) > 50          # the test can tell
        signs = np.sign(G)
        for got, f, more in ((host(o), 1.0, 0), (host(w), -lr * sc, 3 * U32)):
            got = (got if m <= n else got.T) / f
            assert np.all(got[signs == 0] == 0)
            off = np.abs(got * signs - np.abs(signs) * x[:, None]).max(1) / x
            assert np.all(off[clear] <= tol[clear] + more), float(np.max(off[clear] / tol[clear]))


# ---- the error by spectrum -------------------------------------------------------

# Rounding to f16 changes a value by up to half a step, evenly: 2^-11 / sqrt(3)
# of the binade's lower end in the root mean square; over a binade of values
# spread evenly on a logarithmic scale that is this much of the value.
RMS16 = U16 / np.sqrt(3) * np.sqrt(0.75 / (2 * np.log(2)))


def _through(s, coeffs):
    """p(s) of the steps and its derivative."""
    p, dp = s.copy(), np.ones_like(s)
    for a, b, c in coeffs:
        dp = (a + 3 * b * p ** 2 + 5 * c * p ** 4) * dp
        p = a * p + b * p ** 3 + c * p ** 5
    return p, dp


def _gains(s, coeffs):
    """What the steps make of a small change E of X = U diag(s) V^T, in that
    basis: entry by entry, of E's symmetric and antisymmetric part and (right of
    the square) of each row."""
    p, dp = _through(s, coeffs)
    with np.errstate(divide="ignore", invalid="ignore"):
        sym = np.where(np.abs(s[:, None] - s) > 1e-9 * (s[:, None] + s), (p[:, None] - p) / (s[:, None] - s),
                       (dp[:, None] + dp) / 2)
    return sym, (p[:, None] + p) / (s[:, None] + s), p / s


def _expected_error(s, n, coeffs, x0_rounded):
    """Relative error (Frobenius norm) that the f16 roundings make, to first
    order and as independent errors spread evenly over the entries: X_0 (FP32
    sources) to X_k-1, and of every step A and B outside their diagonals."""
    m, var, cur = len(s), 0.0, s / np.linalg.norm(s)
    for it, (a, b, c) in enumerate(coeffs):
        if it or x0_rounded:
            sym, anti, right = _gains(cur, coeffs[it:])
            var += np.sum(cur ** 2) / (m * n) * (np.sum(sym ** 2) / 2 + np.sum(anti ** 2) / 2 + (n - m) * np.sum(right ** 2))
        lam = cur ** 2
        bl = a + b * lam + c * lam ** 2
        after = _gains(bl * cur, coeffs[it + 1:])
        for off, gain in ((np.sum(lam ** 2) - np.sum(lam) ** 2 / m, (b + c * (lam[:, None] + lam)) * cur),
                          # B's rows are also multiplied by what its diagonals lost
                          (2 * (np.sum(bl ** 2) - np.sum(bl) ** 2 / m), np.broadcast_to(cur, (m, m)))):
            sym, anti = (gain + gain.T) / 2 * after[0], (gain - gain.T) / 2 * after[1]
            var += max(off, 0.0) / (m * m) * (np.sum(sym ** 2) + np.sum(anti ** 2))
        cur = bl * cur
    return RMS16 * np.sqrt(var) / np.linalg.norm(cur)


def _spectrum(kind, m):
    if kind == "alike":
        return np.ones(m)
    if kind.startswith("decades"):
        return np.logspace(0, -float(kind[7:]), m)
    few, floor = kind[4:].split("over")
    s = np.full(m, float(floor))
    s[:int(few)] = 1
    return s


def _with_spectrum(s, n, seed):
    g = np.random.default_rng(seed)
    u = np.linalg.qr(g.standard_normal((len(s), len(s))))[0]
    return (u * s) @ np.linalg.qr(g.standard_normal((n, len(s))))[0].T


@pytest.mark.parametrize("ty", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["alike", "decades1", "decades2", "decades3", "few 8over0.01", "few 8over0.001",
                                  "few 32over0.001"])
@pytest.mark.parametrize("m,n", [(64, 100), (256, 512), (512, 512), (300, 1000), (1000, 333), (900, 1100)])
def test_five_steps_by_spectrum(m, n, kind, ty):
    """The error is what the roundings make of this spectrum, times at most 1.5:
    1.36 if all values sat at their binades' lower ends, and the spread of a sum
    of many independent errors."""
    k, kn = min(m, n), max(m, n)
    G = _with_spectrum(_spectrum(kind, k), kn, m + n)
    src = _dev(G if m <= n else G.T, ty)
    G = src.double().cpu().numpy()
    G = G if m <= n else G.T
    u, s, vt = np.linalg.svd(G, full_matrices=False)
    p, _ = _through(s / np.linalg.norm(s), [QUINTIC] * 5)
    want = (u * p) @ vt
    got = host(ns.ns_orthogonalize_f16(src, [QUINTIC] * 5))
    err = np.linalg.norm((got if m <= n else got.T) - want) / np.linalg.norm(p)
    expected = _expected_error(s, kn, [QUINTIC] * 5, ty == torch.float32)
    print(f"[spectrum] {m}x{n} {kind} {ty}: {err:.2e}, expected {expected:.2e}", flush=True)
    assert err <= 1.5 * expected
    assert err <= 2e-3 + 0.2 / np.linalg.norm(p)                 # the documented bound


CUBIC = (1.5, -0.5, 0.0)


@pytest.mark.parametrize("name,coeffs", [("seven", [QUINTIC] * 7), ("cubic", [CUBIC] * 8), ("mixed", [QUINTIC] * 3 + [CUBIC] * 2),
                                         ("falling", [(4.0, -6.5, 3.0), (3.6, -5.4, 2.5), (3.0, -4.0, 1.8), (2.2, -2.0, 0.7)])])
@pytest.mark.parametrize("m,n", [(100, 160), (400, 700), (700, 400)])
def test_other_schedules_by_spectrum(m, n, name, coeffs):
    """Steps with coefficients of their own, more and fewer of them."""
    k, kn = min(m, n), max(m, n)
    for kind in ("decades1", "decades2"):
        G = _with_spectrum(_spectrum(kind, k), kn, m + 2 * n)
        src = _dev(G if m <= n else G.T)
        G = src.double().cpu().numpy()
        u, s, vt = np.linalg.svd(G if m <= n else G.T, full_matrices=False)
        p, _ = _through(s / np.linalg.norm(s), coeffs)
        got = host(ns.ns_orthogonalize_f16(src, coeffs))
        err = np.linalg.norm((got if m <= n else got.T) - (u * p) @ vt) / np.linalg.norm(p)
        assert err <= 1.5 * _expected_error(s, kn, coeffs, True), kind
