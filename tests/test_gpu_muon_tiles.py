"""The Muon step's last product on every tile size, whole and with tiles split
along K, rows aligned to 16 bytes and not, wide and tall, one matrix and more."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV  # noqa: E402

QUINTIC = synth.QUINTIC
U32, UBF = 2.0 ** -24, 2.0 ** -8
FIVE = 4.2e-3       # five steps of these inputs on f16 operands (derived in test_gpu_ns16)

# tile, leftover tiles split (s) or none, aligned rows (a) or not
SHAPES = {"32a": (520, 384, 1), "32": (261, 390, 1), "64a": (384, 384, 2), "64": (1170, 261, 1), "64s": (520, 1171, 3),
          "64sa": (1168, 520, 3), "128a": (1560, 648, 2), "128": (650, 1561, 2), "128s": (2340, 1041, 3),
          "128sa": (1040, 2336, 3), "256a": (2728, 904, 3), "256": (910, 2731, 3), "256s": (1950, 2731, 3),
          "256sa": (2728, 1944, 3)}


def _ns64(G):
    X = G.double().t() if G.shape[0] > G.shape[1] else G.double()
    X = X / (X.norm() + 1e-7)
    for _ in range(5):
        A = X @ X.t()
        X = QUINTIC[0] * X + (QUINTIC[1] * A + QUINTIC[2] * A @ A) @ X
    return X.t() if G.shape[0] > G.shape[1] else X


@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", SHAPES)
def test_muon_step_on_every_tile(which, wt):
    m, n, count = SHAPES[which]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(m + n)
    Gs = [synth.device_lowrank_bf16(m, n, m + i, DEV) for i in range(count)]
    Ms = [3.0 * synth.device_lowrank_bf16(m, n, n + i, DEV).float() for i in range(count)]
    # each with a margin behind it that has to stay
    bufs = [torch.full((m * n + 256,), 7.0, dtype=wt, device=DEV) for _ in range(count)]
    Ws = [b[:m * n].view(m, n) for b in bufs]
    for w in Ws:
        w.copy_(0.02 * torch.randn(m, n, generator=gen, device=DEV))
    w0, m0 = [w.double() for w in Ws], [t.double() for t in Ms]
    scales = [float(np.float32(0.2 * max(m, n) ** 0.5 * (1 + i))) for i in range(count)]
    ns.ns_muon_step(Ws, Ms, Gs, [QUINTIC] * 5, lr=0.02, momentum=0.9, weight_decay=0.1, scales=scales)
    lr, mu, wd = (float(np.float32(v)) for v in (0.02, 0.9, 0.1))
    us = []
    for M, old, g in zip(Ms, m0, Gs):
        want = mu * old + g.double()
        assert bool(((M.double() - want).abs() <= U32 * want.abs() * 1.001).all())
        us.append((g.double() + mu * M.double()).float())
    # U is the same to the bit (the product mu M is exact in 64 bits), so X_k-1, A,
    # B and the last product's sums are too: entry by entry the update is the
    # steps' own FP32 output times lr scale, up to the roundings of either's
    # factors (the scaling of X, lr, scale, t and the row's: 5) and products (2)
    outs = ns.ns_orthogonalize_f16_grouped(us, [QUINTIC] * 5)
    uw = UBF if wt == torch.bfloat16 else U32
    for w, old, o, u, sc, b in zip(Ws, w0, outs, us, scales, bufs):
        want = (1 - lr * wd) * old - lr * sc * o.double()
        # decay is a rounded factor, and the sum is rounded once (to BF16 from FP32)
        tol = 14 * U32 * lr * sc * o.double().abs() + U32 * old.abs() + (uw + U32) * 1.001 * want.abs()
        assert bool(((w - want).abs() <= tol).all()), float(((w - want).abs() / tol).max())
        ref = _ns64(u)
        assert float((o - ref).norm() / ref.norm()) <= FIVE
        assert bool((b[m * n:] == 7.0).all())
