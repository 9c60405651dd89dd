"""16-bit Newton–Schulz and the Muon step on the GPU against float64."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

import newton_schulz_amd as ns  # noqa: E402
from gpu_util import DEV, host, rel_fro  # noqa: E402

CUBIC, QUINTIC = (1.5, -0.5, 0.0), synth.QUINTIC
U16, U32, UBF = 2.0 ** -11, 2.0 ** -24, 2.0 ** -8
# Five steps round 14 operands to f16 (X_1 .. X_4, A and B of each step).  One
# rounding changes entries by at most 2^-11 of themselves, 2^-11 / sqrt(3) in
# the root mean square, and moves the result by at most about twice that
# relative to its norm (B's largest coefficient, 3.4, over X's growth); they
# add up as independent errors: sqrt(14) * 2 * 2^-11 / sqrt(3) = 2.1e-3.
# Twice that is allowed.
FIVE = 4.2e-3
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def ns64(G, coeffs, clip=np.inf):
    X = np.clip(np.asarray(G, np.float64), -clip, clip)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (np.linalg.norm(X) + 1e-7)
    for a, b, c in coeffs:
        A = X @ X.T
        X = a * X + (b * A + c * A @ A) @ X
    return X.T if tall else X


def _g(m, n, seed, ty="f32"):
    t = torch.from_numpy(synth.lowrank_gradient(m, n, seed, rank=min(32, m, n))).to(TYPES[ty])
    return t.to(DEV), t.double().numpy()


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (31, 33), (64, 64), (65, 63), (63, 130), (128, 200), (200, 128), (257, 255),
          (256, 512), (300, 1000), (1000, 333), (1100, 1024), (1024, 1300)]


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", SHAPES)
def test_one_step_within_the_roundings_bound(m, n, ty):
    """One step, entry by entry: X_0 (FP32 sources only), A and B rounded to
    f16, everything else FP32 sums."""
    G, Gv = _g(m, n, m + 3 * n, ty)
    a, b, c = QUINTIC
    X = Gv.T if m > n else Gv
    X = X / (np.linalg.norm(X) + 1e-7)
    A = X @ X.T
    B = a * np.eye(len(A)) + b * A + c * A @ A
    want = B @ X
    # absolute floors: f16 subnormals step by 2^-24, X is held times 256 (at least 128)
    dX = U16 * np.abs(X) + 2.0 ** -25 / 128
    k, kn = len(A), X.shape[1]
    dA = 2 * (np.abs(X) @ dX.T) + (kn + 8) * U32 * (np.abs(X) @ np.abs(X).T)
    dA = dA + dA.T + U16 * (np.abs(A) + dA) + 2.0 ** -25
    dB = abs(b) * dA + abs(c) * (2 * np.abs(A) @ dA + dA @ dA + (k + 8) * U32 * (np.abs(A) @ np.abs(A)))
    dB = dB + dB.T + U16 * (np.abs(B) + dB) + 2.0 ** -25
    tol = np.abs(B) @ dX + dB @ (np.abs(X) + dX) + (k + 8) * U32 * (np.abs(B) @ np.abs(X))
    if m > n:
        want, tol = want.T, tol.T
    for ot, u in ((ns.NS_F32, U32), (ns.NS_BF16, UBF)):
        got = host(ns.ns_orthogonalize_f16(G, [QUINTIC], out_dtype=ot))
        assert np.all(np.abs(got - want) <= tol + u * (np.abs(want) + tol)), float(np.max(np.abs(got - want) / tol))


# Up to 256 rows the product with B makes B itself, with 1, 2, 4 or 8 blocks of
# 32 columns to a workgroup (the third number), until a round of workgroups no
# longer takes it (0).
@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,blocks", [(64, 1000, 1), (130, 70, 1), (1500, 190, 2), (190, 2050, 2), (256, 1025, 2),
                                        (250, 4096, 4), (4096, 256, 4), (129, 5000, 4), (60, 16300, 4), (7000, 256, 8),
                                        (250, 6000, 8), (256, 8200, 0), (8200, 230, 0)])
def test_one_step_with_b_made_in_the_product(m, n, blocks, ty):
    test_one_step_within_the_roundings_bound(m, n, ty)


@pytest.mark.parametrize("m,n,count", [(64, 300, 20), (300, 64, 32), (128, 1000, 16), (200, 700, 5), (256, 512, 16), (256, 520, 16)])
def test_group_of_small_matrices(m, n, count):
    gs = [_g(m, n, 50 + i) for i in range(count)]
    outs = ns.ns_orthogonalize_f16_grouped([g for g, _ in gs], [QUINTIC] * 5)
    for o, (_, v) in zip(outs, gs):
        assert rel_fro(host(o), ns64(v, [QUINTIC] * 5)) <= FIVE
    again = ns.ns_orthogonalize_f16_grouped([g for g, _ in gs], [QUINTIC] * 5)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.parametrize("ty", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(48, 64), (64, 64), (130, 100), (256, 512), (512, 300), (1000, 333), (1100, 1024)])
def test_five_steps(m, n, ty):
    G, Gv = _g(m, n, 7 * m + n, ty)
    want = ns64(Gv, [QUINTIC] * 5)
    err = rel_fro(host(ns.ns_orthogonalize_f16(G, [QUINTIC] * 5)), want)
    print(f"[ns16] {m}x{n} {ty}: {err:.2e}", flush=True)
    assert err <= FIVE
    assert rel_fro(host(ns.ns_orthogonalize_f16(G, [QUINTIC] * 5, out_dtype=ns.NS_BF16)), want) <= FIVE + UBF


def _ns64_gpu(G, coeffs):
    X = G.double().t() if G.shape[0] > G.shape[1] else G.double()
    X = X / (X.norm() + 1e-7)
    for a, b, c in coeffs:
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    return X.t() if G.shape[0] > G.shape[1] else X


# every tile size of the three products, whole and split along K
@pytest.mark.parametrize("m,n", [(200, 600), (900, 1300), (2300, 900), (2000, 2800), (2050, 2050), (3100, 2700), (3100, 3000)])
def test_five_steps_large(m, n):
    G = synth.device_lowrank_bf16(m, n, m + n, DEV)
    want = _ns64_gpu(G, [QUINTIC] * 5)
    got = ns.ns_orthogonalize_f16(G, [QUINTIC] * 5)
    err = float((got - want).norm() / want.norm())
    print(f"[ns16] {m}x{n}: {err:.2e}", flush=True)
    assert err <= FIVE
    assert torch.equal(ns.ns_orthogonalize_f16(G, [QUINTIC] * 5), got)       # the same bits every time
    pair = ns.ns_orthogonalize_f16_grouped([G, G], [QUINTIC] * 5)
    assert torch.equal(pair[0], pair[1]) and float((pair[0] - want).norm() / want.norm()) <= FIVE


def test_clip_and_cubic():
    G, Gv = _g(200, 333, 4)
    clip = 0.02
    coeffs = [CUBIC] * 3
    assert rel_fro(host(ns.ns_orthogonalize_f16(G, coeffs, clip=clip)), ns64(Gv, coeffs, clip)) <= FIVE


def test_vectors_become_unit_vectors():
    """One row or column has one singular value, 1: three cubic steps keep it."""
    for shape in ((1, 1000), (1000, 1)):
        G, Gv = _g(*shape, 5)
        got = host(ns.ns_orthogonalize_f16(G, [CUBIC] * 3))
        assert rel_fro(got, Gv / np.linalg.norm(Gv)) <= FIVE


def test_scale_of_the_source_does_not_matter():
    G, _ = _g(100, 200, 6)
    want = ns.ns_orthogonalize_f16(G, [QUINTIC] * 5)
    # exact powers of two, eps of 1e-7 far below the norm: the same bits
    for e in (20, 100):
        assert torch.equal(ns.ns_orthogonalize_f16(G * 2.0 ** e, [QUINTIC] * 5),
                           ns.ns_orthogonalize_f16(G * 2.0 ** (e + 3), [QUINTIC] * 5))
    assert rel_fro(host(ns.ns_orthogonalize_f16(G * 2.0 ** 100, [QUINTIC] * 5)), host(want)) <= FIVE


def test_zero_and_non_finite():
    z = torch.zeros(70, 90, device=DEV)
    assert (host(ns.ns_orthogonalize_f16(z, [QUINTIC] * 5)) == 0).all()
    for bad in (float("nan"), float("inf")):
        G, _ = _g(70, 90, 1)
        G[3, 4] = bad
        assert np.isnan(host(ns.ns_orthogonalize_f16(G, [QUINTIC] * 2))).all()
    G, Gv = _g(70, 90, 1)
    G[3, 4] = float("inf")                      # an infinity is clipped like any outlier
    Gv[3, 4] = np.inf
    assert rel_fro(host(ns.ns_orthogonalize_f16(G, [QUINTIC] * 5, clip=0.05)), ns64(Gv, [QUINTIC] * 5, 0.05)) <= FIVE


def test_group_of_mixed_shapes():
    shapes = [(64, 100), (200, 64), (64, 100), (33, 500), (200, 64), (64, 100)]
    gs = [_g(*s, 10 + i) for i, s in enumerate(shapes)]
    outs = ns.ns_orthogonalize_f16_grouped([g for g, _ in gs], [QUINTIC] * 5, clips=[0.05] * 6)
    for o, (_, v) in zip(outs, gs):
        assert rel_fro(host(o), ns64(v, [QUINTIC] * 5, 0.05)) <= FIVE
    many = [_g(40, 50, 100 + i) for i in range(35)]            # more than one batch
    outs = ns.ns_orthogonalize_f16_grouped([g for g, _ in many], [QUINTIC] * 5, out_dtype=ns.NS_BF16)
    for o, (_, v) in zip(outs, many):
        assert rel_fro(host(o), ns64(v, [QUINTIC] * 5)) <= FIVE + UBF
    same = ns.ns_orthogonalize_f16_grouped([gs[0][0], gs[0][0]], [QUINTIC] * 5)    # one source twice
    assert torch.equal(same[0], same[1])


def test_nothing_is_written_behind_the_output():
    for m, n in ((33, 70), (70, 33)):
        G, _ = _g(m, n, 2)
        for ty in (torch.float32, torch.bfloat16):
            buf = torch.full((m * n + 128,), 9.0, dtype=ty, device=DEV)
            ns.ns_orthogonalize_f16(G, [QUINTIC] * 2, out=buf[:m * n].view(m, n))
            assert (host(buf)[-128:] == 9.0).all()


OPT = dict(lr=0.02, momentum=0.9, weight_decay=0.1)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("types", [("f32", "f32", "f32"), ("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"),
                                   ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("shapes", [[(100, 70)], [(64, 130), (33, 257), (64, 130)], [(300, 1000)]])
def test_muon_step(shapes, types, nesterov):
    wt, mt, gt = (TYPES[t] for t in types)
    Ws, Ms, Gs = [], [], []
    for i, s in enumerate(shapes):
        Ws.append(torch.from_numpy(0.02 * synth.gaussian(*s, 20 + i)).to(wt).to(DEV))
        Ms.append(torch.from_numpy(3.0 * synth.lowrank_gradient(*s, 30 + i)).to(mt).to(DEV))
        Gs.append(torch.from_numpy(synth.lowrank_gradient(*s, 40 + i)).to(gt).to(DEV))
    scales = [0.2 * max(s) ** 0.5 for s in shapes]
    f = {k: float(np.float32(v)) for k, v in OPT.items()}
    for step in range(2):
        w0, m0, g0 = [[host(t).astype(np.float64) for t in ts] for ts in (Ws, Ms, Gs)]
        ns.ns_muon_step(Ws, Ms, Gs, [QUINTIC] * 5, scales=scales, nesterov=nesterov, **OPT)
        for i in range(len(shapes)):
            um = UBF if types[1] == "bf16" else U32
            uw = UBF if types[0] == "bf16" else U32
            want = f["momentum"] * m0[i] + g0[i]
            got = host(Ms[i]).astype(np.float64)
            assert np.all(np.abs(got - want) <= um * np.abs(want) * (1 + um) + 1e-45)      # one fused rounding
            U = g0[i] + f["momentum"] * got if nesterov else got
            upd = f["lr"] * scales[i] * ns64(U, [QUINTIC] * 5)
            want = (1 - f["lr"] * f["weight_decay"]) * w0[i] - upd
            off = np.linalg.norm(host(Ws[i]) - want)
            assert off <= FIVE * np.linalg.norm(upd) + (uw + 2 * U32) * np.linalg.norm(want)
            assert np.array_equal(host(Gs[i]), g0[i])


def test_muon_of_one_step_and_without_scales():
    W = torch.from_numpy(0.02 * synth.gaussian(70, 200, 1)).to(DEV)
    M = torch.zeros(70, 200, device=DEV)
    G, Gv = _g(70, 200, 2)
    w0 = host(W).astype(np.float64)
    ns.ns_muon_step([W], [M], [G], [CUBIC], lr=0.5, momentum=0.0, nesterov=False)
    upd = 0.5 * ns64(Gv, [CUBIC])
    assert np.array_equal(host(M), host(G))
    assert np.linalg.norm(host(W) - (w0 - upd)) <= FIVE * np.linalg.norm(upd) + 2 * U32 * np.linalg.norm(w0)


def test_muon_non_finite_and_zero_gradients():
    W = torch.ones(40, 50, device=DEV, dtype=torch.bfloat16)
    M = torch.zeros(40, 50, device=DEV)
    ns.ns_muon_step([W], [M], [torch.zeros(40, 50, device=DEV)], [QUINTIC] * 5, lr=0.5, weight_decay=0.5)
    assert (host(W) == 0.75).all() and (host(M) == 0).all()          # decay alone
    G = torch.ones(40, 50, device=DEV)
    G[1, 2] = float("nan")
    ns.ns_muon_step([W], [M], [G], [QUINTIC] * 5, lr=0.5)
    assert np.isnan(host(W)).all() and np.isnan(host(M)).sum() == 1


def test_muon_writes_only_its_arrays():
    for m, n in ((33, 70), (70, 33)):
        buf = [torch.full((m * n + 128,), 2.0, dtype=t, device=DEV) for t in (torch.bfloat16, torch.float32)]
        W, M = (b[:m * n].view(m, n) for b in buf)
        G, _ = _g(m, n, 3, "bf16")
        g0 = G.clone()
        ns.ns_muon_step([W], [M], [G], [QUINTIC] * 2, lr=0.1)
        assert all((host(b)[-128:] == 2.0).all() for b in buf) and torch.equal(G, g0)


def test_binding_refuses():
    G, _ = _g(33, 70, 1)
    with pytest.raises(ValueError):
        ns.ns_orthogonalize_f16(G.t(), [QUINTIC])                    # not contiguous
    with pytest.raises(ValueError):
        ns.ns_orthogonalize_f16(G, [QUINTIC], out=torch.empty(70, 33, device=DEV))
    with pytest.raises(ns.NSError):
        ns.ns_orthogonalize_f16(G, [QUINTIC], out=G)
    with pytest.raises(ns.NSError):
        ns.ns_orthogonalize_f16(G, [QUINTIC], clip=0.0)
    with pytest.raises(ns.NSError):
        ns.ns_orthogonalize_f16(G, [])
    with pytest.raises(ValueError):
        ns.ns_orthogonalize_f16_grouped([G, G], [QUINTIC], clips=[1.0])
    W, M = torch.zeros_like(G), torch.zeros_like(G)
    with pytest.raises(ValueError):
        ns.ns_muon_step([W], [M], [], [QUINTIC], lr=0.1)
    with pytest.raises(ValueError):
        ns.ns_muon_step([W], [M[:, :35].contiguous()], [G], [QUINTIC], lr=0.1)
    with pytest.raises(TypeError):
        ns.ns_muon_step([W, W.bfloat16()], [M, M], [G, G], [QUINTIC], lr=0.1)
    with pytest.raises(ns.NSError):
        ns.ns_muon_step([W], [W], [G], [QUINTIC], lr=0.1)
    with pytest.raises(ns.NSError):
        ns.ns_muon_step([W], [M], [G], [QUINTIC], lr=float("nan"))


def test_muon_in_a_graph_with_the_layer_it_trains():
    """A training step as it is used -- forward, gradients, Muon, the new
    weights quantized -- captured and replayed against the eager run."""
    T, N, K = 96, 128, 160
    x = torch.from_numpy(synth.gaussian(T, K, 1)).to(DEV).to(torch.bfloat16)
    dy = torch.from_numpy(1e-2 * synth.gaussian(T, N, 2)).to(DEV).to(torch.bfloat16)
    w0 = torch.from_numpy(0.05 * synth.gaussian(N, K, 3)).to(DEV)
    W, M, dw = w0.clone(), torch.zeros(N, K, device=DEV), torch.empty(N, K, device=DEV)
    y, dx = torch.empty(T, N, device=DEV), torch.empty(T, K, device=DEV)
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    along, down = (u8(1, N, 128), u8(1, N, 8)), (u8(1, K, 128), u8(1, K, 8))
    kept = (u8(1, K, 128), u8(1, K, 8))
    ws = [u8(ns.mxfp4_linear_workspace_bytes(T, N, K)), u8(ns.mxfp4_linear_backward_workspace_bytes(T, N, K)),
          u8(ns.ns_f16_workspace_bytes([(N, K)]))]

    def step():
        ns.mxfp4_quantize_both(W, along=along, down=down)
        ns.mxfp4_linear(x, along, N, out=y, kept=kept, workspace=ws[0])
        ns.mxfp4_linear_backward(dy, down, kept, K, dx=dx, dw=dw, workspace=ws[1])
        ns.ns_muon_step([W], [M], [dw], [QUINTIC] * 5, lr=0.01, workspace=ws[2])

    def reset():
        W.copy_(w0)
        M.zero_()

    eager = []
    reset()
    for _ in range(3):
        step()
        eager.append([host(t).copy() for t in (W, M, y, dx)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    reset()
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host(t), v) for t, v in zip((W, M, y, dx), want))
        ns.ns_orthogonalize_f16(x, [QUINTIC] * 2)               # eager work between the replays
