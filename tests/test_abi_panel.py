"""The MXFP4 and 16-bit Newton–Schulz entry points refuse bad arguments before
anything is enqueued (CPU only: the addresses are never dereferenced)."""
import ctypes

import pytest

ns = pytest.importorskip("newton_schulz_amd")
lib = ns._lib
ARG, SHAPE, WS = ns.NS_ERR_ARG, ns.NS_ERR_SHAPE, ns.NS_ERR_WORKSPACE
BIG = 1 << 24


def _addr(i, off=0):
    """Distinct fake device addresses, 1 TiB apart."""
    return ctypes.c_void_p((i + 1) * (1 << 40) + off)


def test_sizes():
    assert lib.mxfp4_codes_bytes(33, 70, 0) == 33 * 128 and lib.mxfp4_scales_bytes(33, 70, 0) == 33 * 8
    assert lib.mxfp4_codes_bytes(33, 70, 1) == 70 * 128
    assert lib.mxfp4_codes_bytes(2, 257, 0) == 2 * 2 * 128
    for bad in ((0, 5, 0), (5, 0, 0), (5, 5, 2), (BIG + 1, 5, 0), (BIG, BIG, 0)):
        assert lib.mxfp4_codes_bytes(*bad) == 0 and lib.mxfp4_scales_bytes(*bad) == 0
    assert lib.mxfp4_linear_workspace_bytes(1, 64, 64) == 0       # quantized in registers
    assert lib.mxfp4_linear_workspace_bytes(100, 64, 64) >= 100 * (128 + 8)
    assert lib.mxfp4_linear_workspace_bytes(0, 64, 64) == 0
    one = lambda v: (ctypes.c_int64 * 1)(v)  # noqa: E731
    assert lib.ns_f16_workspace_bytes(1, one(0), one(5)) == 0
    assert lib.ns_f16_workspace_bytes(1, one(1 << 20), one(1 << 12)) == 0      # 2^32 elements
    a = lib.ns_f16_workspace_bytes(1, one(64), one(100))
    assert a >= 3 * 64 * 128 * 2 + 2 * 64 * 64 * 2 and a == lib.ns_f16_workspace_bytes(1, one(100), one(64))


def test_quantizers():
    x, c, s, d, t = (_addr(i) for i in range(5))
    q = lib.mxfp4_quantize
    assert q(None, 0, 4, 4, 0, c, s, None) == ARG
    assert q(x, 2, 4, 4, 0, c, s, None) == ARG                    # dtype
    assert q(x, 0, 4, 4, 2, c, s, None) == ARG                    # axis
    assert q(x, 0, 0, 4, 0, c, s, None) == SHAPE
    assert q(x, 0, 4, -1, 0, c, s, None) == SHAPE
    assert q(x, 0, BIG + 1, 1, 0, c, s, None) == SHAPE
    assert q(x, 0, BIG, BIG, 0, c, s, None) == SHAPE              # too many elements
    assert q(_addr(0, 4), 0, 4, 4, 0, c, s, None) == ARG          # alignment
    assert q(x, 0, 4, 4, 0, _addr(1, 8), s, None) == ARG
    assert q(x, 0, 64, 64, 0, _addr(0, 1024), s, None) == ARG     # codes inside x
    assert q(x, 0, 64, 64, 0, c, _addr(1, 64), None) == ARG       # scales inside the codes
    both = lib.mxfp4_quantize_both
    assert both(x, 0, 64, 64, c, s, c, t, None) == ARG
    assert both(x, 0, 64, 64, c, s, d, s, None) == ARG
    assert both(x, 0, 64, 64, c, s, d, None, None) == ARG
    de = lib.mxfp4_dequantize
    assert de(c, s, 64, 64, 0, c, 0, None) == ARG
    assert de(c, s, 64, 64, 0, _addr(3, 8), 0, None) == ARG
    assert de(c, s, 64, 0, 0, x, 0, None) == SHAPE
    assert de(c, s, 64, 64, 0, x, 5, None) == ARG


def test_product():
    p, ps, q, qs, o, a, w = (_addr(i) for i in range(7))
    g = lib.mxfp4_gemm

    def call(M=64, N=64, K=64, alpha=1.0, beta=0.0, addend=None, out=o, ot=0, ws=None, wb=0, pc=p):
        return g(pc, ps, q, qs, M, N, K, alpha, beta, addend, out, ot, ws, wb, None)
    assert call(pc=None) == ARG
    assert call(M=0) == SHAPE and call(K=-3) == SHAPE and call(N=BIG + 1) == SHAPE
    assert call(M=BIG, N=BIG) == SHAPE
    assert call(beta=1.0) == ARG                                  # no addend
    assert call(alpha=float("nan")) == ARG and call(beta=float("inf"), addend=a) == ARG
    assert call(ot=3) == ARG
    assert call(out=_addr(0, 4096)) == ARG                        # over an operand
    assert call(beta=1.0, addend=_addr(4, 256)) == ARG            # shifted over the output
    assert call(beta=1.0, addend=o, ot=1) == ARG                  # in place needs FP32
    assert call(out=_addr(4, 4)) == ARG
    big = dict(M=1024, N=1024, K=16384)
    need = lib.mxfp4_gemm_workspace_bytes(1024, 1024, 16384)
    assert need > 0
    assert call(**big, ws=w, wb=need - 1) == WS
    assert call(**big, ws=_addr(6, 8), wb=need) == ARG
    assert call(**big, ws=_addr(2, 4096), wb=need) == ARG         # workspace over an operand


def test_linear():
    x, wc, ws_, y, kc, ks, z = (_addr(i) for i in range(7))
    T, N, K = 100, 64, 96
    need = lib.mxfp4_linear_workspace_bytes(T, N, K)

    def call(T=T, N=N, K=K, x=x, y=y, kc=None, ks=None, ws=z, wb=need, yt=1):
        return lib.mxfp4_linear(x, 1, T, K, wc, ws_, N, y, yt, kc, ks, ws, wb, None)
    assert call(x=None) == ARG and call(yt=4) == ARG
    assert call(T=0) == SHAPE and call(N=0) == SHAPE
    assert call(kc=kc) == ARG                                     # codes without scales
    assert call(ws=None, wb=0) == WS and call(wb=need - 1) == WS
    assert call(y=x) == ARG and call(y=_addr(3, 2)) == ARG
    assert call(kc=y, ks=ks) == ARG                               # kept over the output
    assert call(ws=x) == ARG
    need = lib.mxfp4_linear_backward_workspace_bytes(T, N, K)
    dx, dw = _addr(8), _addr(9)

    def back(dy=x, wt=wc, wts=ws_, k=kc, kss=ks, dx=dx, dw=dw, dwt=0, beta=0.0, ws=z, wb=need, T=T):
        return lib.mxfp4_linear_backward(dy, 1, T, N, K, wt, wts, k, kss, dx, 0, dw, dwt, beta, ws, wb, None)
    assert back(dy=None) == ARG and back(dx=None, dw=None) == ARG
    assert back(wt=None) == ARG and back(kss=None) == ARG
    assert back(beta=1.0, dwt=1) == ARG and back(beta=1.0, dw=None) == ARG and back(beta=float("nan")) == ARG
    assert back(T=0) == SHAPE
    assert back(ws=None) == WS and back(wb=need - 1) == WS
    assert back(dx=dw) == ARG and back(dw=x) == ARG and back(ws=kc) == ARG


def _arr(t, *v):
    return (t * len(v))(*v)


def test_orthogonalize():
    G, o, w = (_addr(i) for i in range(3))
    co = _arr(ctypes.c_float, 1.5, -0.5, 0.0)
    need = lib.ns_f16_workspace_bytes(1, _arr(ctypes.c_int64, 33), _arr(ctypes.c_int64, 70))

    def call(G=G, m=33, n=70, coeffs=co, k=1, clip=1.0, out=o, ot=0, ws=w, wb=need):
        return lib.ns_orthogonalize_f16(G, 0, m, n, coeffs, k, clip, out, ot, ws, wb, None)
    assert call(G=None) == ARG and call(out=None) == ARG and call(coeffs=None) == ARG
    assert call(k=0) == ARG and call(ot=2) == ARG
    assert call(coeffs=_arr(ctypes.c_float, 1.5, float("inf"), 0.0)) == ARG
    for clip in (0.0, -1.0, float("nan")):
        assert call(clip=clip) == ARG
    assert call(m=0) == SHAPE and call(n=BIG + 1) == SHAPE and call(m=1 << 16, n=1 << 15) == SHAPE
    assert call(ws=None) == WS and call(wb=need - 1) == WS
    assert call(out=_addr(0, 64)) == ARG and call(G=_addr(0, 2)) == ARG and call(ws=_addr(1, 16)) == ARG
    assert lib.ns_orthogonalize_f16_grouped(0, _arr(ctypes.c_void_p, G), None, None, 0, co, 1, None, None, 0, w, need,
                                            None) == ARG


@pytest.mark.parametrize("count", [2, 40])       # the ranges' table on the stack and on the heap
def test_groups_and_muon(count):
    ms, ns_ = _arr(ctypes.c_int64, *[33] * count), _arr(ctypes.c_int64, *[70] * count)
    co = _arr(ctypes.c_float, 1.5, -0.5, 0.0)
    need = lib.ns_f16_workspace_bytes(count, ms, ns_)
    V = lambda base: [(base << 44) + (i << 20) for i in range(1, count + 1)]  # noqa: E731
    P = lambda v: _arr(ctypes.c_void_p, *v)  # noqa: E731
    ws = ctypes.c_void_p(9 << 44)

    def group(G, out):
        return lib.ns_orthogonalize_f16_grouped(count, P(G), ms, ns_, 0, co, 1, None, P(out), 0, ws, need, None)
    one = V(2)
    assert group(V(1), one[:-1] + [one[0]]) == ARG                # an output twice
    assert group(V(1), one[:-1] + [V(1)[0] + 64]) == ARG          # an output in another's input
    assert group(V(1), one[:-1] + [(9 << 44) + 256]) == ARG       # in the workspace
    opt = ns.NsMuonOptions(0.1, 0.9, 0.0, 1)

    def muon(W=V(1), M=V(2), G=V(3), opt=opt, scale=None, wb=need, k=1):
        return lib.ns_muon_step(count, P(W), 0, P(M), 0, P(G), 1, ms, ns_, co, k, ctypes.byref(opt), scale, ws, wb, None)
    assert muon(W=[None] + V(1)[1:]) == ARG
    assert muon(M=V(1)) == ARG and muon(G=V(2)) == ARG
    assert muon(W=V(1)[:-1] + [V(1)[0] + 128]) == ARG
    assert muon(opt=ns.NsMuonOptions(float("nan"), 0.9, 0.0, 1)) == ARG
    assert muon(scale=_arr(ctypes.c_float, *[float("inf")] * count)) == ARG
    assert muon(wb=need - 1) == WS and muon(k=0) == ARG
    assert muon(G=V(3)[:-1] + [V(3)[0] + 2]) == ARG               # alignment
