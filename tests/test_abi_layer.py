"""The entry points between 4-bit layers refuse bad arguments before anything
is enqueued (CPU only: the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

ns = pytest.importorskip("newton_schulz_amd")
lib = ns._lib
ARG, SHAPE, WS = ns.NS_ERR_ARG, ns.NS_ERR_SHAPE, ns.NS_ERR_WORKSPACE
BIG = 1 << 24


def at(i, off=0):
    """Distinct fake device addresses, 1 TiB apart."""
    return (i + 1) * (1 << 40) + off


def test_sizes():
    assert lib.mxfp8_codes_bytes(33, 70) == 33 * 256 and lib.mxfp8_scales_bytes(33, 70) == 33 * 8
    assert lib.mxfp8_codes_bytes(2, 257) == 2 * 2 * 256
    for bad in ((0, 5), (5, -1), (BIG + 1, 5), (BIG, BIG)):
        assert lib.mxfp8_codes_bytes(*bad) == 0 and lib.mxfp8_scales_bytes(*bad) == 0
    w = lib.mx_rms_norm_backward_workspace_bytes
    assert w(1, 64) >= 64 * 4 and w(0, 64) == 0 and w(5, 32769) == 0
    assert lib.mxfp8_gemm_workspace_bytes(0, 5, 5) == 0


def test_dropout():
    d = lib.mx_dropout

    def call(x=at(0), t=0, rows=4, cols=8, p=0.5, rng=at(1), out=at(2)):
        return d(x, t, rows, cols, p, rng, out, None)
    assert call(x=None) == ARG and call(out=None) == ARG and call(rng=None) == ARG and call(t=2) == ARG
    for p in (-0.1, 1.0, 0.999999, float("nan"), float("inf")):
        assert call(p=p) == ARG
    assert call(rows=0) == SHAPE and call(cols=BIG + 1) == SHAPE and call(rows=BIG, cols=BIG) == SHAPE
    assert call(x=at(0, 4)) == ARG and call(out=at(2, 8)) == ARG and call(rng=at(1, 4)) == ARG
    assert call(out=at(0, 64)) == ARG                    # shifted over x
    assert call(rng=at(2, 16)) == ARG                    # the generator's words inside the output


def norm(**k):
    a = ns.MxNormArgs()
    d = dict(x=at(0), weight=at(1), T=8, C=64, eps=1e-6, drop=0.0, xt=0, ht=0, wt=0, yt=0, y=at(2))
    d.update(k)
    for n, v in d.items():
        setattr(a, n, v)
    return lib.mx_rms_norm(ctypes.byref(a), None)


def test_norm():
    assert lib.mx_rms_norm(None, None) == ARG
    assert norm(x=None) == ARG and norm(weight=None) == ARG
    assert norm(y=None) == ARG                           # nothing to write
    for t in ("xt", "ht", "wt", "yt"):
        assert norm(**{t: 2}) == ARG
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == ARG
    assert norm(T=0) == SHAPE and norm(C=0) == SHAPE and norm(C=32769) == SHAPE and norm(T=BIG + 1) == SHAPE
    assert norm(residual=at(3)) == ARG                   # no h
    assert norm(h=at(3)) == ARG                          # h is x here
    assert norm(ht=1) == ARG                             # of another type
    assert norm(drop=0.5, rng=at(4)) == ARG              # no h
    assert norm(drop=0.5, h=at(3)) == ARG                # no generator
    assert norm(drop=1.0, h=at(3), rng=at(4)) == ARG and norm(drop=-0.5, h=at(3), rng=at(4)) == ARG
    assert norm(codes8=at(5)) == ARG and norm(scales4=at(5)) == ARG and norm(kept_codes=at(5), rstd=at(7)) == ARG
    assert norm(kept_codes=at(5), kept_scales=at(6)) == ARG          # needs rstd
    for n in ("x", "weight", "y", "rstd"):
        assert norm(**{n: at(8, 8)}) == ARG
    assert norm(codes8=at(5, 8), scales8=at(6)) == ARG
    assert norm(y=at(0)) == ARG and norm(y=at(0, 1024)) == ARG and norm(rstd=at(2, 16)) == ARG
    assert norm(residual=at(3), h=at(0)) == ARG                      # over x
    assert norm(residual=at(3), h=at(3, 64)) == ARG                  # beside the residual's own place
    assert norm(codes4=at(5), scales4=at(5, 64)) == ARG
    assert norm(codes8=at(5), scales8=at(6), kept_codes=at(5, 128), kept_scales=at(7), rstd=at(8)) == ARG
    assert norm(drop=0.5, residual=at(3), h=at(4), rng=at(4, 32)) == ARG


def back(ws=at(20), wb=1 << 30, **k):
    a = ns.MxNormBackwardArgs()
    d = dict(dy=at(0), h=at(1), rstd=at(2), weight=at(3), dh=at(4), dweight=at(5), T=8, C=64, drop=0.0, beta=0.0,
             dyt=0, ht=0, wt=0, xt=0)
    d.update(k)
    for n, v in d.items():
        setattr(a, n, v)
    return lib.mx_rms_norm_backward(ctypes.byref(a), ws, wb, None)


def test_norm_backward():
    assert lib.mx_rms_norm_backward(None, None, 0, None) == ARG
    for n in ("dy", "h", "rstd", "weight", "dh"):
        assert back(**{n: None}) == ARG
        assert back(**{n: at(9, 8)}) == ARG
    for t in ("dyt", "ht", "wt", "xt"):
        assert back(**{t: -1}) == ARG
    assert back(T=0) == SHAPE and back(C=40000) == SHAPE
    need = lib.mx_rms_norm_backward_workspace_bytes(8, 64)
    assert back(wb=need - 1) == WS and back(ws=None, wb=0) == WS
    assert back(beta=float("nan")) == ARG and back(drop=0.5) == ARG and back(drop=float("nan")) == ARG
    assert back(dh=at(0)) == ARG and back(dx=at(4, 64)) == ARG and back(dweight=at(4)) == ARG
    assert back(dh_in=at(4, 64)) == ARG                  # beside its own place
    assert back(ws=at(1, 256)) == ARG and back(ws=at(20, 8)) == ARG
    assert back(drop=0.5, rng=at(4, 16)) == ARG


def test_mxfp8():
    q = lib.mxfp8_quantize
    x, c, s = at(0), at(1), at(2)
    assert q(None, 0, 4, 4, c, s, None) == ARG and q(x, 3, 4, 4, c, s, None) == ARG and q(x, 0, 4, 0, c, s, None) == SHAPE
    assert q(at(0, 4), 0, 4, 4, c, s, None) == ARG and q(x, 0, 64, 64, at(0, 1024), s, None) == ARG
    assert q(x, 0, 64, 64, c, at(1, 64), None) == ARG
    d = lib.mxfp8_dequantize
    assert d(c, s, 4, 4, None, 0, None) == ARG and d(c, s, 4, 4, c, 0, None) == ARG and d(c, s, 0, 4, x, 0, None) == SHAPE
    g = lib.mxfp8_gemm

    def call(M=64, N=64, K=64, alpha=1.0, beta=0.0, addend=None, out=at(4), ot=0, ws=None, wb=0, p=at(0)):
        return g(p, at(1), at(2), at(3), M, N, K, alpha, beta, addend, out, ot, ws, wb, None)
    assert call(p=None) == ARG and call(M=0) == SHAPE and call(N=BIG, K=BIG) == SHAPE
    assert call(beta=1.0) == ARG and call(alpha=float("nan")) == ARG and call(beta=float("inf"), addend=at(5)) == ARG
    assert call(ot=2) == ARG and call(out=at(0, 4096)) == ARG and call(out=at(4, 4)) == ARG
    assert call(beta=1.0, addend=at(4, 256)) == ARG and call(beta=1.0, addend=at(4), ot=1) == ARG
    assert call(ws=at(2, 1024), wb=1 << 20) == ARG


def test_nvfp4_linear():
    f = lib.nvfp4_linear

    def call(x=at(0), xt=0, T=2, K=64, c=at(1), s=at(2), g=at(3), N=5, y=at(4), yt=0):
        return f(x, xt, T, K, c, s, g, N, y, yt, None)
    for n in ("x", "c", "s", "g", "y"):
        assert call(**{n: None}) == ARG
    assert call(xt=2) == ARG and call(yt=-1) == ARG
    assert call(K=72) == SHAPE and call(T=0) == SHAPE and call(N=0) == SHAPE and call(K=BIG + 16) == SHAPE
    assert call(x=at(0, 8)) == ARG and call(g=at(3, 2)) == ARG and call(y=at(0, 32)) == ARG and call(y=at(1)) == ARG


def test_binding():
    """What only the binding can see: shapes, types and generators."""
    with pytest.raises(ValueError):
        ns._need_rng(None, torch.device("cuda", 0))
    with pytest.raises(ValueError):
        ns._need_rng(torch.zeros(2), torch.device("cuda", 0))
    with pytest.raises(ValueError):
        ns._need_rng(torch.zeros(3, dtype=torch.int64), torch.device("cuda", 0))
    ok = torch.zeros(2, 7, 256, dtype=torch.uint8), torch.zeros(2, 7, 8, dtype=torch.uint8)
    ns._need_blocks(ok, "p", 7, 300, 256)
    for rows, cols, width in ((6, 300, 256), (8, 300, 256), (7, 200, 256), (7, 600, 256), (7, 300, 128)):
        with pytest.raises(ValueError):
            ns._need_blocks(ok, "p", rows, cols, width)
    with pytest.raises(TypeError):
        ns._need_blocks((ok[0].to(torch.int32).view(-1), ok[1]), "p", 7, 300, 256)
    x = torch.zeros(3, 4)
    with pytest.raises(ValueError):
        ns.mx_rms_norm(x, torch.ones(4))                 # not on a device
    with pytest.raises(ValueError):
        ns.mx_rms_norm(torch.zeros(4), torch.ones(4))    # not a matrix
    with pytest.raises(ValueError):
        ns.mx_dropout(x, 0.5, None)
    with pytest.raises(ValueError):
        ns.mx_rms_norm_backward(x, x, torch.zeros(3), torch.ones(4), beta=1.0)


def test_more_threads_than_a_launch_takes():
    """A row a workgroup, or 256 results one, beyond 2^32 threads."""
    assert norm(T=1 << 22, C=1025) == SHAPE and norm(T=1 << 24, C=1025) == SHAPE
    assert norm(T=1 << 22, C=16384) == SHAPE

    def linear(T, N, K=16):
        return lib.nvfp4_linear(at(0), 0, T, K, at(1), at(2), at(3), N, at(4), 0, None)
    assert linear(1 << 20, 1025) == SHAPE
    assert linear(BIG, 65) == SHAPE
