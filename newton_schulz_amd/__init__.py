"""Python binding of the NVFP4 Newton–Schulz library (libnvfp4ns.so).

Argument marshalling only: every step runs in the HIP kernels behind the C
ABI declared in ``include/nvfp4ns.h``.  torch supplies device memory and the
current stream.  There is no fallback: if the library is missing this
module raises ImportError.

Functions carry the C names:
    nvfp4_quantize, nvfp4_quantize_noalloc, nvfp4_quantize_rht, nvfp4_dequantize,
    nvfp4_gemm_workspace_bytes, nvfp4_gemm, ns_workspace_bytes, ns_workspace_layout,
    ns_orthogonalize, ns_orthogonalize_rht, ns_orthogonalize_ex,
    ns_abs_quantile_workspace_bytes, ns_abs_quantile,
    ns_grouped_workspace_bytes, ns_orthogonalize_grouped, ns_orthogonalize_grouped_ex,
    ns_orthogonalize_grouped_on,
    mxfp4_quantize, mxfp4_quantize_both, mxfp4_dequantize, mxfp4_gemm_workspace_bytes, mxfp4_gemm,
    mxfp4_linear, mxfp4_linear_backward,
    ns_f16_workspace_bytes, ns_orthogonalize_f16, ns_orthogonalize_f16_grouped, ns_muon_step,
    mx_dropout, mx_rms_norm, mx_rms_norm_backward, mxfp8_quantize, mxfp8_dequantize,
    mxfp8_gemm_workspace_bytes, mxfp8_gemm, nvfp4_linear
"""
import collections
import contextlib
import ctypes
import os

# torch first: the library must bind to the HIP runtime torch has loaded (the
# one that owns the devices, streams and memory it is handed), not bring in
# a second copy ahead of it.
import torch  # noqa: F401

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnvfp4ns.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python newton_schulz_amd/build.py` "
        "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)

NS_OK, NS_ERR_ARG, NS_ERR_SHAPE, NS_ERR_WORKSPACE, NS_ERR_HIP = 0, -1, -2, -3, -4
NS_F32, NS_BF16 = 0, 1
NVFP4_ROWS, NVFP4_COLS = 0, 1
STATUS_NAMES = {0: "NS_OK", -1: "NS_ERR_ARG", -2: "NS_ERR_SHAPE",
                -3: "NS_ERR_WORKSPACE", -4: "NS_ERR_HIP"}

_i64, _sz, _vp, _f, _i = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float, ctypes.c_int
_u16 = ctypes.c_uint16
_d = ctypes.c_double


class NsOptions(ctypes.Structure):
    """ns_options of the C ABI."""
    _fields_ = [("clip", ctypes.c_float), ("clip_quantile", ctypes.c_double),
                ("rht_masks", ctypes.POINTER(ctypes.c_uint16)), ("adaptive46", ctypes.c_int)]

class NsMuonOptions(ctypes.Structure):
    """ns_muon_options of the C ABI."""
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("nesterov", ctypes.c_int)]


class MxNormArgs(ctypes.Structure):
    """mx_norm_args of the C ABI."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "residual", "weight", "rng", "h", "rstd", "y", "codes8",
                                                "scales8", "codes4", "scales4", "kept_codes", "kept_scales")]
                + [("T", ctypes.c_int64), ("C", ctypes.c_int64), ("eps", ctypes.c_double),
                   ("drop", ctypes.c_double)] + [(n, ctypes.c_int) for n in ("xt", "ht", "wt", "yt")])


class MxNormBackwardArgs(ctypes.Structure):
    """mx_norm_backward_args of the C ABI."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("dy", "h", "rstd", "weight", "dh_in", "rng", "dh", "dx", "dweight")]
                + [("T", ctypes.c_int64), ("C", ctypes.c_int64), ("drop", ctypes.c_double),
                   ("beta", ctypes.c_float)] + [(n, ctypes.c_int) for n in ("dyt", "ht", "wt", "xt")])


class NsWorkspaceMap(ctypes.Structure):
    """ns_workspace_map of the C ABI (byte offsets into an NS workspace)."""
    _fields_ = [("xm", ctypes.c_int64), ("xn", ctypes.c_int64),
                ("x", ctypes.c_size_t), ("a", ctypes.c_size_t), ("b", ctypes.c_size_t),
                ("qx_codes", ctypes.c_size_t), ("qx_scales", ctypes.c_size_t),
                ("qt_codes", ctypes.c_size_t), ("qt_scales", ctypes.c_size_t),
                ("qa_codes", ctypes.c_size_t), ("qa_scales", ctypes.c_size_t),
                ("qb_codes", ctypes.c_size_t), ("qb_scales", ctypes.c_size_t),
                ("global_scales", ctypes.c_size_t), ("total", ctypes.c_size_t)]


_SIGS = {
    "nvfp4_quantize_workspace_bytes": (_sz, [_i64, _i64]),
    "nvfp4_quantize": (_i, [_vp, _i, _i64, _i64, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nvfp4_quantize_noalloc": (_i, [_vp, _i, _i64, _i64, _i, _vp, _vp, _vp, _vp]),
    "nvfp4_quantize_rht": (_i, [_vp, _i, _i64, _i64, _i, _u16, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nvfp4_quantize_46": (_i, [_vp, _i, _i64, _i64, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "nvfp4_dequantize": (_i, [_vp, _vp, _vp, _i64, _i64, _i, _vp, _i, _vp]),
    "nvfp4_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64, _i]),
    "nvfp4_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i, _f, _f, _vp, _vp, _vp,
                        _vp, _sz, _vp]),
    "ns_workspace_bytes": (_sz, [_i64, _i64]),
    "ns_workspace_layout": (_i, [_i64, _i64, _vp]),
    "ns_orthogonalize": (_i, [_vp, _i, _i64, _i64, _vp, _i, _f, _vp, _i, _vp, _sz, _vp]),
    "ns_orthogonalize_rht": (_i, [_vp, _i, _i64, _i64, _vp, _i, _f, _vp, _vp, _i, _vp, _sz, _vp]),
    "ns_orthogonalize_ex": (_i, [_vp, _i, _i64, _i64, _vp, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "ns_abs_quantile_workspace_bytes": (_sz, []),
    "ns_abs_quantile": (_i, [_vp, _i, _i64, _d, _vp, _vp, _sz, _vp]),
    "ns_grouped_workspace_bytes": (_sz, [_i, _vp, _vp]),
    "ns_orthogonalize_grouped": (_i, [_i, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "ns_orthogonalize_grouped_ex": (_i, [_i, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _sz,
                                         _vp]),
    "ns_orthogonalize_grouped_on": (_i, [_i, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _sz,
                                         _vp, _i, _vp]),
    "mxfp4_codes_bytes": (_sz, [_i64, _i64, _i]),
    "mxfp4_scales_bytes": (_sz, [_i64, _i64, _i]),
    "mxfp4_quantize": (_i, [_vp, _i, _i64, _i64, _i, _vp, _vp, _vp]),
    "mxfp4_quantize_both": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "mxfp4_dequantize": (_i, [_vp, _vp, _i64, _i64, _i, _vp, _i, _vp]),
    "mxfp4_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxfp4_gemm": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _f, _f, _vp, _vp, _i, _vp, _sz, _vp]),
    "mxfp4_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxfp4_linear": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _i64, _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "mxfp4_linear_backward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxfp4_linear_backward": (_i, [_vp, _i, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i,
                                   _f, _vp, _sz, _vp]),
    "ns_f16_workspace_bytes": (_sz, [_i, _vp, _vp]),
    "ns_orthogonalize_f16": (_i, [_vp, _i, _i64, _i64, _vp, _i, _f, _vp, _i, _vp, _sz, _vp]),
    "ns_orthogonalize_f16_grouped": (_i, [_i, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _vp, _sz,
                                          _vp]),
    "ns_muon_step": (_i, [_i, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _sz,
                          _vp]),
    "mx_dropout": (_i, [_vp, _i, _i64, _i64, _d, _vp, _vp, _vp]),
    "mx_rms_norm": (_i, [_vp, _vp]),
    "mx_rms_norm_backward_workspace_bytes": (_sz, [_i64, _i64]),
    "mx_rms_norm_backward": (_i, [_vp, _vp, _sz, _vp]),
    "mxfp8_codes_bytes": (_sz, [_i64, _i64]),
    "mxfp8_scales_bytes": (_sz, [_i64, _i64]),
    "mxfp8_quantize": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp]),
    "mxfp8_dequantize": (_i, [_vp, _vp, _i64, _i64, _vp, _i, _vp]),
    "mxfp8_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mxfp8_gemm": (_i, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _f, _f, _vp, _vp, _i, _vp, _sz, _vp]),
    "nvfp4_linear": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class NSError(RuntimeError):
    def __init__(self, status, where):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


def _check(status, where):
    if status != NS_OK:
        raise NSError(status, where)


def _torch():
    import torch
    return torch


def _stream(stream, device=None):
    """The stream to enqueue on: `stream`, else the current stream of the
    tensors' device."""
    if stream is not None:
        if device is not None and getattr(stream, "device", device) != device:
            raise ValueError(f"a stream of {stream.device} for tensors on {device}")
        return ctypes.c_void_p(stream.cuda_stream)
    torch = _torch()
    if device is None or device.index is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    # the handle itself: building a Stream object costs 2 us a call
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))


_HERE = contextlib.nullcontext()


def _on(device):
    """Makes `device` the current one (nothing to do where it is already)."""
    torch = _torch()
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _dt(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return NS_F32
    if t.dtype == torch.bfloat16:
        return NS_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _out_dtype(code):
    torch = _torch()
    return torch.float32 if code == NS_F32 else torch.bfloat16


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need_cuda(*ts):
    ts = [t for t in ts if t is not None]
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous device tensors")
    if any(t.device != ts[0].device for t in ts):
        raise ValueError("tensors must be on one device")


def _need(t, name, dtypes, numel):
    """A caller-supplied tensor: one of `dtypes` and at least `numel`
    elements, so that no kernel reads or writes past its end."""
    if t is None:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {numel} needed")


def _need_shape(t, name, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _floats():
    torch = _torch()
    return (torch.float32, torch.bfloat16)


# ------------------------------------------------------------- quantizer --

def nvfp4_quantize(x, axis=NVFP4_ROWS, codes=None, scales=None, global_scale=None,
                   workspace=None, stream=None, adaptive46=False):
    """NVFP4 quantization of a 2-D float32/bfloat16 device tensor.

    Returns (codes uint8 [r][c/2], scales uint8 [r][c/16], s_g float32 [1]),
    in the layout of x (NVFP4_ROWS) or of x^T (NVFP4_COLS).  adaptive46=True
    calls nvfp4_quantize_46 (adaptive 4/6 block scaling).
    """
    torch = _torch()
    _need_cuda(x)
    rows, cols = x.shape
    r, c = (rows, cols) if axis == NVFP4_ROWS else (cols, rows)
    dev = x.device
    if codes is None:
        codes = torch.empty((r, c // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((r, c // 16), dtype=torch.uint8, device=dev)
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=dev)
    wsb = _lib.nvfp4_quantize_workspace_bytes(rows, cols)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    _need_quant_outputs(x, rows, cols, codes, scales, global_scale, workspace)
    fn, name = ((_lib.nvfp4_quantize_46, "nvfp4_quantize_46") if adaptive46
                else (_lib.nvfp4_quantize, "nvfp4_quantize"))
    with torch.cuda.device(dev):
        _check(fn(_ptr(x), _dt(x), rows, cols, axis, _ptr(codes), _ptr(scales), _ptr(global_scale),
                  _ptr(workspace), workspace.numel(), _stream(stream, dev)), name)
    return codes, scales, global_scale


def nvfp4_quantize_noalloc(x, axis=NVFP4_ROWS, codes=None, scales=None, global_scale=None,
                           stream=None):
    """nvfp4_quantize through the allocation-free entry point (its scratch is
    the library's static device array); outputs as nvfp4_quantize."""
    torch = _torch()
    _need_cuda(x)
    rows, cols = x.shape
    r, c = (rows, cols) if axis == NVFP4_ROWS else (cols, rows)
    dev = x.device
    if codes is None:
        codes = torch.empty((r, c // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((r, c // 16), dtype=torch.uint8, device=dev)
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=dev)
    _need_quant_outputs(x, rows, cols, codes, scales, global_scale, None)
    with torch.cuda.device(dev):
        _check(_lib.nvfp4_quantize_noalloc(_ptr(x), _dt(x), rows, cols, axis, _ptr(codes),
                                           _ptr(scales), _ptr(global_scale),
                                           _stream(stream, dev)), "nvfp4_quantize_noalloc")
    return codes, scales, global_scale


def _need_quant_outputs(x, rows, cols, codes, scales, global_scale, workspace):
    torch = _torch()
    _need_cuda(x, codes, scales, global_scale, workspace)
    _need(codes, "codes", (torch.uint8,), rows * cols // 2)
    _need(scales, "scales", (torch.uint8,), rows * cols // 16)
    _need(global_scale, "global_scale", (torch.float32,), 1)
    _need(workspace, "workspace", (torch.uint8,), 0)


def nvfp4_quantize_rht(x, mask, axis=NVFP4_ROWS, codes=None, scales=None, global_scale=None,
                       workspace=None, stream=None):
    """Q_1x16(x H) (NVFP4_ROWS) or Q_16x1(H^T x) (NVFP4_COLS) with the random
    Hadamard transform H_16^r of the 16-bit sign mask; outputs as
    nvfp4_quantize."""
    torch = _torch()
    _need_cuda(x)
    rows, cols = x.shape
    r, c = (rows, cols) if axis == NVFP4_ROWS else (cols, rows)
    dev = x.device
    if codes is None:
        codes = torch.empty((r, c // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((r, c // 16), dtype=torch.uint8, device=dev)
    if global_scale is None:
        global_scale = torch.empty(1, dtype=torch.float32, device=dev)
    wsb = _lib.nvfp4_quantize_workspace_bytes(rows, cols)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    _need_quant_outputs(x, rows, cols, codes, scales, global_scale, workspace)
    with torch.cuda.device(dev):
        _check(_lib.nvfp4_quantize_rht(_ptr(x), _dt(x), rows, cols, axis, int(mask) & 0xFFFF,
                                       _ptr(codes), _ptr(scales), _ptr(global_scale),
                                       _ptr(workspace), workspace.numel(), _stream(stream, dev)),
               "nvfp4_quantize_rht")
    return codes, scales, global_scale


def nvfp4_dequantize(codes, scales, global_scale, rows, cols, axis=NVFP4_ROWS,
                     out_dtype=NS_F32, out=None, stream=None):
    """x_hat = x_E2M1 * s * s_g, in the original rows x cols orientation."""
    torch = _torch()
    _need_cuda(codes, scales, global_scale, out)
    if out is None:
        out = torch.empty((rows, cols), dtype=_out_dtype(out_dtype), device=codes.device)
    _need(codes, "codes", (torch.uint8,), rows * cols // 2)
    _need(scales, "scales", (torch.uint8,), rows * cols // 16)
    _need(global_scale, "global_scale", (torch.float32,), 1)
    _need(out, "out", (_out_dtype(out_dtype),), rows * cols)
    with torch.cuda.device(codes.device):
        _check(_lib.nvfp4_dequantize(_ptr(codes), _ptr(scales), _ptr(global_scale), rows, cols,
                                     axis, _ptr(out), out_dtype, _stream(stream, codes.device)),
               "nvfp4_dequantize")
    return out


def nvfp4_quantize_workspace_bytes(rows, cols):
    return int(_lib.nvfp4_quantize_workspace_bytes(rows, cols))


def nvfp4_gemm_workspace_bytes(M, N, K, symmetric=False):
    return int(_lib.nvfp4_gemm_workspace_bytes(M, N, K, 1 if symmetric else 0))


def nvfp4_gemm(p, q, M, N, K, symmetric=False, alpha=1.0, beta=0.0, addend=None, out=None,
               amax_out=None, workspace=None, split=True, stream=None):
    """out = beta*addend + alpha*s_gP*s_gQ*(P Q^T); p, q = (codes, scales, s_g).

    With split=True (default) a workspace of nvfp4_gemm_workspace_bytes() is
    allocated when none is given, so the product runs with the same launch
    schedule as inside ns_orthogonalize.
    """
    torch = _torch()
    (pc, ps, pg), (qc, qs, qg) = p, q
    _need_cuda(pc, ps, pg, qc, qs, qg, addend, out, amax_out)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=pc.device)
    if workspace is None and split:
        nb = nvfp4_gemm_workspace_bytes(M, N, K, symmetric)
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=pc.device)
    _need_cuda(pc, workspace)
    u8 = (torch.uint8,)
    _need(pc, "p codes", u8, M * K // 2)
    _need(ps, "p scales", u8, M * K // 16)
    _need(qc, "q codes", u8, N * K // 2)
    _need(qs, "q scales", u8, N * K // 16)
    _need(pg, "p s_g", (torch.float32,), 1)
    _need(qg, "q s_g", (torch.float32,), 1)
    _need(out, "out", (torch.float32,), M * N)
    if float(beta) != 0.0:
        _need(addend, "addend", (torch.float32,), M * N)
    _need(amax_out, "amax_out", (torch.int32, torch.uint32), 1)
    _need(workspace, "workspace", u8, 0)
    wsp, wsn = (_ptr(workspace), workspace.numel()) if workspace is not None else (_ptr(None), 0)
    with torch.cuda.device(pc.device):
        _check(_lib.nvfp4_gemm(_ptr(pc), _ptr(ps), _ptr(pg), _ptr(qc), _ptr(qs), _ptr(qg),
                               M, N, K, 1 if symmetric else 0, float(alpha), float(beta),
                               _ptr(addend), _ptr(out), _ptr(amax_out), wsp, wsn,
                               _stream(stream, pc.device)),
               "nvfp4_gemm")
    return out


# ---------------------------------------------------------- Newton–Schulz --

def ns_workspace_bytes(m, n):
    return int(_lib.ns_workspace_bytes(m, n))


def ns_workspace_layout(m, n):
    """ns_workspace_layout: dict of the byte offsets (and xm, xn, total) of
    the iteration's operands inside an ns_orthogonalize workspace."""
    mp = NsWorkspaceMap()
    _check(_lib.ns_workspace_layout(m, n, ctypes.byref(mp)), "ns_workspace_layout")
    return {name: int(getattr(mp, name)) for name, _ in NsWorkspaceMap._fields_}


def ns_workspace_views(ws, m, n):
    """Views of the operands inside an NS workspace (uint8 device tensor):
    X, A, B as float32 matrices, the four NVFP4 operands as (codes, scales)
    uint8 matrices, and the four tensor scales as float32[4]."""
    torch = _torch()
    L = ns_workspace_layout(m, n)
    xm, xn = L["xm"], L["xn"]

    def f32(off, r, c):
        return ws[off:off + 4 * r * c].view(torch.float32).view(r, c)

    def u8(off, r, c):
        return ws[off:off + r * c].view(r, c)

    return {"X": f32(L["x"], xm, xn), "A": f32(L["a"], xm, xm), "B": f32(L["b"], xm, xm),
            "qX": (u8(L["qx_codes"], xm, xn // 2), u8(L["qx_scales"], xm, xn // 16)),
            "qX16": (u8(L["qt_codes"], xn, xm // 2), u8(L["qt_scales"], xn, xm // 16)),
            "qA": (u8(L["qa_codes"], xm, xm // 2), u8(L["qa_scales"], xm, xm // 16)),
            "qB": (u8(L["qb_codes"], xm, xm // 2), u8(L["qb_scales"], xm, xm // 16)),
            "sg": ws[L["global_scales"]:L["global_scales"] + 16].view(torch.float32)}


def _need_ns(G, out, workspace):
    torch = _torch()
    _need_cuda(G, out, workspace)
    _need_shape(out, "out", G.shape)
    _need(out, "out", _floats(), G.numel())
    _need(workspace, "workspace", (torch.uint8,), 0)


def _coeff_array(coeffs):
    flat = [float(v) for abc in coeffs for v in abc]
    return (ctypes.c_float * len(flat))(*flat), len(flat) // 3


def ns_orthogonalize(G, coeffs, clip=float("inf"), out_dtype=NS_F32, out=None, workspace=None,
                     stream=None):
    """k NVFP4 Newton–Schulz steps on one m x n float32/bfloat16 matrix."""
    torch = _torch()
    _need_cuda(G, out)
    m, n = G.shape
    if out is None:
        out = torch.empty((m, n), dtype=_out_dtype(out_dtype), device=G.device)
    if workspace is None:
        workspace = torch.empty(ns_workspace_bytes(m, n), dtype=torch.uint8, device=G.device)
    _need_ns(G, out, workspace)
    carr, k = _coeff_array(coeffs)
    with torch.cuda.device(G.device):
        _check(_lib.ns_orthogonalize(_ptr(G), _dt(G), m, n, carr, k, float(clip), _ptr(out),
                                     _dt(out), _ptr(workspace), workspace.numel(),
                                     _stream(stream, G.device)), "ns_orthogonalize")
    return out


def ns_orthogonalize_rht(G, coeffs, masks, clip=float("inf"), out_dtype=NS_F32, out=None,
                         workspace=None, stream=None):
    """ns_orthogonalize with the random Hadamard transform of each step
    (one 16-bit sign mask per coefficient triple)."""
    torch = _torch()
    _need_cuda(G, out)
    m, n = G.shape
    if out is None:
        out = torch.empty((m, n), dtype=_out_dtype(out_dtype), device=G.device)
    if workspace is None:
        workspace = torch.empty(ns_workspace_bytes(m, n), dtype=torch.uint8, device=G.device)
    _need_ns(G, out, workspace)
    carr, k = _coeff_array(coeffs)
    if len(masks) != k:
        raise ValueError("one Hadamard mask per step")
    marr = (ctypes.c_uint16 * k)(*[int(v) & 0xFFFF for v in masks])
    with torch.cuda.device(G.device):
        _check(_lib.ns_orthogonalize_rht(_ptr(G), _dt(G), m, n, carr, k, float(clip), marr,
                                         _ptr(out), _dt(out), _ptr(workspace), workspace.numel(),
                                         _stream(stream, G.device)), "ns_orthogonalize_rht")
    return out


def ns_orthogonalize_ex(G, coeffs, clip=float("inf"), clip_quantile=0.0, rht_masks=None,
                        out_dtype=NS_F32, out=None, workspace=None, stream=None, adaptive46=False):
    """ns_orthogonalize with an on-device quantile clip (clip_quantile in
    (0, 1]; 0 uses `clip`), the random Hadamard transform (one 16-bit mask
    per step) and/or adaptive 4/6 block scaling on every quantization."""
    torch = _torch()
    _need_cuda(G, out)
    m, n = G.shape
    if out is None:
        out = torch.empty((m, n), dtype=_out_dtype(out_dtype), device=G.device)
    if workspace is None:
        workspace = torch.empty(ns_workspace_bytes(m, n), dtype=torch.uint8, device=G.device)
    _need_ns(G, out, workspace)
    carr, k = _coeff_array(coeffs)
    opt = NsOptions(float(clip), float(clip_quantile), None, 1 if adaptive46 else 0)
    marr = None
    if rht_masks is not None:
        if len(rht_masks) != k:
            raise ValueError("one Hadamard mask per step")
        marr = (ctypes.c_uint16 * k)(*[int(v) & 0xFFFF for v in rht_masks])
        opt.rht_masks = ctypes.cast(marr, ctypes.POINTER(ctypes.c_uint16))
    with torch.cuda.device(G.device):
        _check(_lib.ns_orthogonalize_ex(_ptr(G), _dt(G), m, n, carr, k, ctypes.byref(opt),
                                        _ptr(out), _dt(out), _ptr(workspace), workspace.numel(),
                                        _stream(stream, G.device)), "ns_orthogonalize_ex")
    return out


def ns_abs_quantile_workspace_bytes():
    return int(_lib.ns_abs_quantile_workspace_bytes())


def ns_abs_quantile(x, q, out=None, workspace=None, stream=None):
    """The q-quantile of |x| (k-th smallest magnitude, k = ceil(q N)) as a
    one-element float32 device tensor."""
    torch = _torch()
    _need_cuda(x)
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(ns_abs_quantile_workspace_bytes(), dtype=torch.uint8, device=x.device)
    _need_cuda(x, out, workspace)
    _need(out, "out", (torch.float32,), 1)
    _need(workspace, "workspace", (torch.uint8,), 0)
    with torch.cuda.device(x.device):
        _check(_lib.ns_abs_quantile(_ptr(x), _dt(x), x.numel(), float(q), _ptr(out),
                                    _ptr(workspace), workspace.numel(), _stream(stream, x.device)),
               "ns_abs_quantile")
    return out


def ns_grouped_workspace_bytes(shapes):
    cnt = len(shapes)
    ms = (ctypes.c_int64 * cnt)(*[s[0] for s in shapes])
    ns = (ctypes.c_int64 * cnt)(*[s[1] for s in shapes])
    return int(_lib.ns_grouped_workspace_bytes(cnt, ms, ns))


def ns_orthogonalize_grouped(Gs, coeffs, clips, out_dtype=NS_F32, outs=None, workspace=None,
                             stream=None):
    """ns_orthogonalize over a list of matrices with one schedule."""
    torch = _torch()
    cnt = len(Gs)
    _need_cuda(*Gs)
    dt = _dt(Gs[0])
    if any(_dt(g) != dt for g in Gs):
        raise TypeError("all inputs must share one dtype")
    shapes = [tuple(g.shape) for g in Gs]
    if outs is None:
        outs = [torch.empty(s, dtype=_out_dtype(out_dtype), device=Gs[0].device) for s in shapes]
    if workspace is None:
        workspace = torch.empty(ns_grouped_workspace_bytes(shapes), dtype=torch.uint8,
                                device=Gs[0].device)
    _need_group(Gs, outs, workspace)
    if len(clips) != cnt:
        raise ValueError("one clip per matrix")
    gp = (ctypes.c_void_p * cnt)(*[g.data_ptr() for g in Gs])
    op = (ctypes.c_void_p * cnt)(*[o.data_ptr() for o in outs])
    ms = (ctypes.c_int64 * cnt)(*[s[0] for s in shapes])
    ns = (ctypes.c_int64 * cnt)(*[s[1] for s in shapes])
    cl = (ctypes.c_float * cnt)(*[float(c) for c in clips])
    carr, k = _coeff_array(coeffs)
    dev = Gs[0].device
    with torch.cuda.device(dev):
        _check(_lib.ns_orthogonalize_grouped(cnt, gp, ms, ns, dt, carr, k, cl, op, _dt(outs[0]),
                                             _ptr(workspace), workspace.numel(),
                                             _stream(stream, dev)), "ns_orthogonalize_grouped")
    return outs


def _need_group(Gs, outs, workspace):
    torch = _torch()
    if len(Gs) == 0 or len(outs) != len(Gs):
        raise ValueError("one output per matrix, at least one matrix")
    _need_cuda(*Gs, *outs, workspace)
    for i, (g, o) in enumerate(zip(Gs, outs)):
        _need_shape(o, f"outs[{i}]", g.shape)
        _need(o, f"outs[{i}]", (outs[0].dtype,), g.numel())
    _need(outs[0], "outs[0]", _floats(), 0)
    _need(workspace, "workspace", (torch.uint8,), 0)


def ns_orthogonalize_grouped_ex(Gs, coeffs, clips=None, clip_quantile=0.0, rht_masks=None,
                                out_dtype=NS_F32, outs=None, workspace=None, stream=None,
                                adaptive46=False):
    """ns_orthogonalize_grouped with a per-matrix quantile clip, the random
    Hadamard transform and/or adaptive 4/6 scaling (options shared by every
    matrix)."""
    torch = _torch()
    cnt = len(Gs)
    _need_cuda(*Gs)
    dt = _dt(Gs[0])
    if any(_dt(g) != dt for g in Gs):
        raise TypeError("all inputs must share one dtype")
    shapes = [tuple(g.shape) for g in Gs]
    if outs is None:
        outs = [torch.empty(s, dtype=_out_dtype(out_dtype), device=Gs[0].device) for s in shapes]
    if workspace is None:
        workspace = torch.empty(ns_grouped_workspace_bytes(shapes), dtype=torch.uint8,
                                device=Gs[0].device)
    _need_group(Gs, outs, workspace)
    if clips is not None and len(clips) != cnt:
        raise ValueError("one clip per matrix")
    gp = (ctypes.c_void_p * cnt)(*[g.data_ptr() for g in Gs])
    op = (ctypes.c_void_p * cnt)(*[o.data_ptr() for o in outs])
    ms = (ctypes.c_int64 * cnt)(*[s[0] for s in shapes])
    ns_ = (ctypes.c_int64 * cnt)(*[s[1] for s in shapes])
    cl = (ctypes.c_float * cnt)(*[float(c) for c in clips]) if clips is not None else None
    carr, k = _coeff_array(coeffs)
    opt = NsOptions(float("inf"), float(clip_quantile), None, 1 if adaptive46 else 0)
    marr = None
    if rht_masks is not None:
        if len(rht_masks) != k:
            raise ValueError("one Hadamard mask per step")
        marr = (ctypes.c_uint16 * k)(*[int(v) & 0xFFFF for v in rht_masks])
        opt.rht_masks = ctypes.cast(marr, ctypes.POINTER(ctypes.c_uint16))
    dev = Gs[0].device
    with torch.cuda.device(dev):
        _check(_lib.ns_orthogonalize_grouped_ex(cnt, gp, ms, ns_, dt, carr, k, cl,
                                                ctypes.byref(opt), op, _dt(outs[0]),
                                                _ptr(workspace), workspace.numel(),
                                                _stream(stream, dev)),
               "ns_orthogonalize_grouped_ex")
    return outs


def ns_orthogonalize_grouped_on(Gs, coeffs, streams, clips=None, clip_quantile=0.0,
                                rht_masks=None, adaptive46=False, out_dtype=NS_F32, outs=None,
                                workspace=None, stream=None):
    """ns_orthogonalize_grouped_ex on the caller's streams (a list of
    torch.cuda.Stream, 1 to 16): the library keeps nothing between calls."""
    torch = _torch()
    cnt = len(Gs)
    _need_cuda(*Gs)
    dt = _dt(Gs[0])
    if any(_dt(g) != dt for g in Gs):
        raise TypeError("all inputs must share one dtype")
    shapes = [tuple(g.shape) for g in Gs]
    if outs is None:
        outs = [torch.empty(s, dtype=_out_dtype(out_dtype), device=Gs[0].device) for s in shapes]
    if workspace is None:
        workspace = torch.empty(ns_grouped_workspace_bytes(shapes), dtype=torch.uint8,
                                device=Gs[0].device)
    _need_group(Gs, outs, workspace)
    if clips is not None and len(clips) != cnt:
        raise ValueError("one clip per matrix")
    gp = (ctypes.c_void_p * cnt)(*[g.data_ptr() for g in Gs])
    op = (ctypes.c_void_p * cnt)(*[o.data_ptr() for o in outs])
    ms = (ctypes.c_int64 * cnt)(*[s[0] for s in shapes])
    ns_ = (ctypes.c_int64 * cnt)(*[s[1] for s in shapes])
    cl = (ctypes.c_float * cnt)(*[float(c) for c in clips]) if clips is not None else None
    carr, k = _coeff_array(coeffs)
    opt = NsOptions(float("inf"), float(clip_quantile), None, 1 if adaptive46 else 0)
    marr = None
    if rht_masks is not None:
        if len(rht_masks) != k:
            raise ValueError("one Hadamard mask per step")
        marr = (ctypes.c_uint16 * k)(*[int(v) & 0xFFFF for v in rht_masks])
        opt.rht_masks = ctypes.cast(marr, ctypes.POINTER(ctypes.c_uint16))
    sarr = (ctypes.c_void_p * max(len(streams), 1))(*[s.cuda_stream for s in streams])
    dev = Gs[0].device
    with torch.cuda.device(dev):
        _check(_lib.ns_orthogonalize_grouped_on(cnt, gp, ms, ns_, dt, carr, k, cl,
                                                ctypes.byref(opt), op, _dt(outs[0]),
                                                _ptr(workspace), workspace.numel(), sarr,
                                                len(streams), _stream(stream, dev)),
               "ns_orthogonalize_grouped_on")
    return outs


# ----------------------------------------------------------------- MXFP4 --

def _empty(shape, dtype, dev, stream):
    """A new tensor, of the stream that the call enqueues on: the allocator may
    give its memory away again as soon as that stream's work is in order."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if stream.device != dev:
        raise ValueError(f"a stream of {stream.device} for tensors on {dev}")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _wrote(given):
    """Tells autograd of the caller's tensors that a call has written (None:
    not given), so that one saved for a backward pass is reported."""
    for t in given:
        if t is not None:
            _torch().autograd.graph.increment_version(t)


def _mx_panels(n):
    return -(-n // 256)


def _mx_buffers(rows, cols, codes, scales, dev, stream):
    """Codes and scales of an operand of `rows` rows blocked along `cols`."""
    torch = _torch()
    p = _mx_panels(cols)
    if codes is None:
        codes = _empty((p, rows, 128), torch.uint8, dev, stream)
    if scales is None:
        scales = _empty((p, rows, 8), torch.uint8, dev, stream)
    return codes, scales


def _need_mx(codes, scales, name, rows, cols):
    """The row count is the pitch from panel to panel, so a larger operand's
    panels would be read in the wrong places: the shape has to be the call's.
    Other views need its size, flat buffers at least that."""
    torch = _torch()
    p = _mx_panels(cols)
    for t, what, n in ((codes, "codes", 128), (scales, "scales", 8)):
        if t is None or t.dtype == torch.uint8 and t.shape == (p, rows, n):
            continue
        what = f"{name} {what}"
        _need(t, what, (torch.uint8,), p * rows * n)
        if t.dim() == 3:
            _need_shape(t, what, (p, rows, n))
        elif t.dim() != 1 and t.numel() != p * rows * n:
            raise ValueError(f"{what}: {t.numel()} elements, {p * rows * n} needed")


def _need_2d(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: a matrix is needed, got shape {tuple(t.shape)}")


def mxfp4_quantize(x, axis=NVFP4_ROWS, codes=None, scales=None, stream=None):
    """MXFP4 quantization of a 2-D float32/bfloat16 device tensor in one pass.

    Returns (codes uint8 [panels][r][128], scales uint8 [panels][r][8]) of x
    (NVFP4_ROWS, r = rows) or of x^T (NVFP4_COLS, r = columns), panels of 256
    elements along the blocked axis.
    """
    _need_2d(x, "x")
    given = codes, scales
    rows, cols = x.shape
    r, c = (rows, cols) if axis == NVFP4_ROWS else (cols, rows)
    codes, scales = _mx_buffers(r, c, codes, scales, x.device, stream)
    _need_cuda(x, codes, scales)
    _need_mx(codes, scales, "out", r, c)
    with _on(x.device):
        _check(_lib.mxfp4_quantize(_ptr(x), _dt(x), rows, cols, axis, _ptr(codes), _ptr(scales),
                                   _stream(stream, x.device)), "mxfp4_quantize")
    _wrote(given)
    return codes, scales


def mxfp4_quantize_both(x, along=None, down=None, stream=None):
    """Both quantizations of x in one pass: ((codes, scales) of NVFP4_ROWS,
    (codes, scales) of NVFP4_COLS)."""
    _need_2d(x, "x")
    rows, cols = x.shape
    rc, rs = _mx_buffers(rows, cols, *(along or (None, None)), x.device, stream)
    cc, cs = _mx_buffers(cols, rows, *(down or (None, None)), x.device, stream)
    _need_cuda(x, rc, rs, cc, cs)
    _need_mx(rc, rs, "along", rows, cols)
    _need_mx(cc, cs, "down", cols, rows)
    with _on(x.device):
        _check(_lib.mxfp4_quantize_both(_ptr(x), _dt(x), rows, cols, _ptr(rc), _ptr(rs), _ptr(cc),
                                        _ptr(cs), _stream(stream, x.device)), "mxfp4_quantize_both")
    _wrote((*(along or ()), *(down or ())))
    return (rc, rs), (cc, cs)


def mxfp4_dequantize(codes, scales, rows, cols, axis=NVFP4_ROWS, out_dtype=NS_F32, out=None,
                     stream=None):
    """The values of an MXFP4 tensor, in the original rows x cols orientation."""
    _need_cuda(codes, scales, out)
    given = out
    if out is None:
        out = _empty((rows, cols), _out_dtype(out_dtype), codes.device, stream)
    r, c = (rows, cols) if axis == NVFP4_ROWS else (cols, rows)
    _need_mx(codes, scales, "in", r, c)
    _need(out, "out", _floats(), rows * cols)
    with _on(codes.device):
        _check(_lib.mxfp4_dequantize(_ptr(codes), _ptr(scales), rows, cols, axis, _ptr(out), _dt(out),
                                     _stream(stream, codes.device)), "mxfp4_dequantize")
    _wrote((given,))
    return out


def mxfp4_gemm_workspace_bytes(M, N, K):
    return int(_lib.mxfp4_gemm_workspace_bytes(M, N, K))


def _mx_workspace(need, workspace, dev, stream):
    """The given workspace, or a new one where the call needs any."""
    torch = _torch()
    if workspace is None:
        return _empty(need, torch.uint8, dev, stream) if need else None
    _need(workspace, "workspace", (torch.uint8,), 0)
    return workspace


def _ws_args(workspace):
    return (_ptr(None), 0) if workspace is None else (_ptr(workspace), workspace.numel())


def mxfp4_gemm(p, q, M, N, K, alpha=1.0, beta=0.0, addend=None, out_dtype=NS_F32, out=None,
               workspace=None, split=True, stream=None):
    """out = beta*addend + alpha*(P Q^T); p, q = (codes, scales) along K.

    With split=True (default) a workspace of mxfp4_gemm_workspace_bytes() is
    allocated when none is given."""
    torch = _torch()
    (pc, ps), (qc, qs) = p, q
    dev = pc.device
    given = out
    if out is None:
        out = _empty((M, N), _out_dtype(out_dtype), dev, stream)
    if workspace is not None or split:
        workspace = _mx_workspace(mxfp4_gemm_workspace_bytes(M, N, K), workspace, dev, stream)
    _need_cuda(pc, ps, qc, qs, addend, out, workspace)
    _need_mx(pc, ps, "p", M, K)
    _need_mx(qc, qs, "q", N, K)
    _need(out, "out", _floats(), M * N)
    if float(beta) != 0.0:
        _need(addend, "addend", (torch.float32,), M * N)
    with _on(dev):
        _check(_lib.mxfp4_gemm(_ptr(pc), _ptr(ps), _ptr(qc), _ptr(qs), M, N, K, float(alpha),
                               float(beta), _ptr(addend), _ptr(out), _dt(out),
                               *_ws_args(workspace), _stream(stream, dev)), "mxfp4_gemm")
    _wrote((given,))
    return out


def mxfp4_linear_workspace_bytes(T, N, K):
    return int(_lib.mxfp4_linear_workspace_bytes(T, N, K))


def mxfp4_linear_backward_workspace_bytes(T, N, K):
    return int(_lib.mxfp4_linear_backward_workspace_bytes(T, N, K))


def mxfp4_linear(x, w, N, out=None, keep=False, kept=None, workspace=None, stream=None):
    """y = Q(x) w^T for x [T][K] (float32/bfloat16) and MXFP4 weights w =
    (codes, scales) of [N][K] along K; y takes x's dtype unless `out` is given.

    keep=True (or a `kept` pair of buffers) also quantizes x along the tokens
    and returns (y, kept), kept = (codes, scales) for mxfp4_linear_backward."""
    wc, ws_ = w
    _need_2d(x, "x")
    T, K = x.shape
    dev = x.device
    given = (out, *(kept or ()))
    if out is None:
        out = _empty((T, N), x.dtype, dev, stream)
    kc, ks = _mx_buffers(K, T, *(kept or (None, None)), dev, stream) if keep or kept else (None, None)
    workspace = _mx_workspace(mxfp4_linear_workspace_bytes(T, N, K), workspace, dev, stream)
    _need_cuda(x, wc, ws_, out, kc, ks, workspace)
    _need_mx(wc, ws_, "w", N, K)
    _need(out, "out", _floats(), T * N)
    if kc is not None:
        _need_mx(kc, ks, "kept", K, T)
    with _on(dev):
        _check(_lib.mxfp4_linear(_ptr(x), _dt(x), T, K, _ptr(wc), _ptr(ws_), N, _ptr(out), _dt(out),
                                 _ptr(kc), _ptr(ks), *_ws_args(workspace),
                                 _stream(stream, dev)), "mxfp4_linear")
    _wrote(given)
    return (out, (kc, ks)) if kc is not None else out


def mxfp4_linear_backward(dy, wt, kept, K, dx=None, dw=None, need_dx=True, need_dw=True, beta=0.0,
                          workspace=None, stream=None):
    """Gradients of mxfp4_linear for dy [T][N]: (dx [T][K], dw [N][K]).

    wt = (codes, scales) of the weights along N (NVFP4_COLS of [N][K]), kept as
    returned by mxfp4_linear.  need_dx / need_dw False leaves one out (None is
    returned in its place).  dw = beta * dw + gradient (beta != 0 needs a
    float32 `dw`); new tensors take dy's dtype."""
    _need_2d(dy, "dy")
    T, N = dy.shape
    dev = dy.device
    given = dx if need_dx else None, dw if need_dw else None
    if need_dx and dx is None:
        dx = _empty((T, K), dy.dtype, dev, stream)
    if need_dw and dw is None:
        if float(beta) != 0.0:
            raise ValueError("beta != 0 adds to a dw that is given")
        dw = _empty((N, K), dy.dtype, dev, stream)
    dx, dw = dx if need_dx else None, dw if need_dw else None
    (wc, ws_), (kc, ks) = wt if need_dx else (None, None), kept if need_dw else (None, None)
    workspace = _mx_workspace(mxfp4_linear_backward_workspace_bytes(T, N, K), workspace, dev, stream)
    _need_cuda(dy, dx, dw, wc, ws_, kc, ks, workspace)
    if need_dx:
        _need_mx(wc, ws_, "wt", K, N)
        _need(dx, "dx", _floats(), T * K)
    if need_dw:
        _need_mx(kc, ks, "kept", K, T)
        _need(dw, "dw", _floats(), N * K)
    with _on(dev):
        _check(_lib.mxfp4_linear_backward(_ptr(dy), _dt(dy), T, N, K, _ptr(wc), _ptr(ws_), _ptr(kc),
                                          _ptr(ks), _ptr(dx), _dt(dx) if need_dx else NS_F32, _ptr(dw),
                                          _dt(dw) if need_dw else NS_F32, float(beta),
                                          *_ws_args(workspace), _stream(stream, dev)),
               "mxfp4_linear_backward")
    _wrote(given)
    return dx, dw


# ---------------------------------------------- 16-bit Newton–Schulz, Muon --

def _shape_arrays(shapes):
    cnt = len(shapes)
    return ((ctypes.c_int64 * cnt)(*[s[0] for s in shapes]),
            (ctypes.c_int64 * cnt)(*[s[1] for s in shapes]))


def ns_f16_workspace_bytes(shapes):
    """Workspace of the 16-bit calls for a list of (m, n)."""
    ms, ns_ = _shape_arrays(shapes)
    return int(_lib.ns_f16_workspace_bytes(len(shapes), ms, ns_))


def _pointers(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def ns_orthogonalize_f16(G, coeffs, clip=float("inf"), out_dtype=NS_F32, out=None, workspace=None,
                         stream=None):
    """k Newton–Schulz steps with f16 operands on one m x n float32/bfloat16
    matrix of any shape.

    Five quintic steps are off by 0.4e-3 to 2e-3 (relative Frobenius norm) for
    singular values alike or within a decade, 4e-3 within two, up to 1.5e-2
    within three, and at most 2e-3 + 0.2 / ||result||_F."""
    _need_cuda(G, out)
    _need_2d(G, "G")
    m, n = G.shape
    given = out
    if out is None:
        out = _empty((m, n), _out_dtype(out_dtype), G.device, stream)
    workspace = _mx_workspace(ns_f16_workspace_bytes([(m, n)]), workspace, G.device, stream)
    _need_ns(G, out, workspace)
    carr, k = _coeff_array(coeffs)
    with _on(G.device):
        _check(_lib.ns_orthogonalize_f16(_ptr(G), _dt(G), m, n, carr, k, float(clip), _ptr(out),
                                         _dt(out), *_ws_args(workspace),
                                         _stream(stream, G.device)), "ns_orthogonalize_f16")
    _wrote((given,))
    return out


def ns_orthogonalize_f16_grouped(Gs, coeffs, clips=None, out_dtype=NS_F32, outs=None,
                                 workspace=None, stream=None):
    """ns_orthogonalize_f16 over a list of matrices; those of one shape run as
    one batch."""
    cnt = len(Gs)
    _need_cuda(*Gs)
    dt = _dt(Gs[0])
    if any(_dt(g) != dt for g in Gs):
        raise TypeError("all inputs must share one dtype")
    for i, g in enumerate(Gs):
        _need_2d(g, f"Gs[{i}]")
    shapes = [tuple(g.shape) for g in Gs]
    dev = Gs[0].device
    given = outs or ()
    if outs is None:
        outs = [_empty(s, _out_dtype(out_dtype), dev, stream) for s in shapes]
    workspace = _mx_workspace(ns_f16_workspace_bytes(shapes), workspace, dev, stream)
    _need_group(Gs, outs, workspace)
    if clips is not None and len(clips) != cnt:
        raise ValueError("one clip per matrix")
    ms, ns_ = _shape_arrays(shapes)
    cl = (ctypes.c_float * cnt)(*[float(c) for c in clips]) if clips is not None else None
    carr, k = _coeff_array(coeffs)
    with _on(dev):
        _check(_lib.ns_orthogonalize_f16_grouped(cnt, _pointers(Gs), ms, ns_, dt, carr, k, cl,
                                                 _pointers(outs), _dt(outs[0]),
                                                 *_ws_args(workspace), _stream(stream, dev)),
               "ns_orthogonalize_f16_grouped")
    _wrote(given)
    return outs


def ns_muon_step(Ws, Ms, Gs, coeffs, lr, momentum=0.95, weight_decay=0.0, nesterov=True, scales=None,
                 workspace=None, stream=None):
    """One Muon step, in place on the weights Ws and momenta Ms (lists of
    matrices, each list of one dtype): M <- momentum M + G; U = G + momentum M
    (nesterov) or M; W <- (1 - lr weight_decay) W - lr scale NS(U).

    NS runs on f16 operands, whatever the arrays' types, and is off by as much
    as ns_orthogonalize_f16.  To autograd it is an update in place (without
    no_grad), so a weight that a pending backward pass has saved is reported."""
    cnt = len(Ws)
    if cnt == 0 or len(Ms) != cnt or len(Gs) != cnt:
        raise ValueError("one momentum and one gradient per weight matrix, at least one")
    _need_cuda(*Ws, *Ms, *Gs)
    shapes = []
    for i, (w, m, g) in enumerate(zip(Ws, Ms, Gs)):
        _need_2d(w, f"Ws[{i}]")
        shapes.append(tuple(w.shape))
        for t, first, name in ((w, Ws[0], "Ws"), (m, Ms[0], "Ms"), (g, Gs[0], "Gs")):
            _need_shape(t, f"{name}[{i}]", w.shape)
            if t.dtype != first.dtype:
                raise TypeError(f"{name}: one dtype for all matrices")
    if scales is not None and len(scales) != cnt:
        raise ValueError("one scale per matrix")
    dev = Ws[0].device
    workspace = _mx_workspace(ns_f16_workspace_bytes(shapes), workspace, dev, stream)
    _need_cuda(Ws[0], workspace)
    ms, ns_ = _shape_arrays(shapes)
    sc = (ctypes.c_float * cnt)(*[float(c) for c in scales]) if scales is not None else None
    carr, k = _coeff_array(coeffs)
    opt = NsMuonOptions(float(lr), float(momentum), float(weight_decay), 1 if nesterov else 0)
    with _on(dev):
        _check(_lib.ns_muon_step(cnt, _pointers(Ws), _dt(Ws[0]), _pointers(Ms), _dt(Ms[0]),
                                 _pointers(Gs), _dt(Gs[0]), ms, ns_, carr, k, ctypes.byref(opt), sc,
                                 *_ws_args(workspace), _stream(stream, dev)),
               "ns_muon_step")
    _wrote((*Ws, *Ms))
    return Ws


# ------------------------------------------- between 4-bit linear layers --
# Calls of a few microseconds on the GPU: a tensor made here is not checked
# again, and a stream or device object is not made where a number serves.

def _new(shape, strides, dtype, dev, stream):
    """As _empty; with its strides given, a tensor takes half the time."""
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=dev)
    if stream.device != dev:
        raise ValueError(f"a stream of {stream.device} for tensors on {dev}")
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=dev)


def _launch(fn, name, dev, stream, *args):
    """fn(*args, stream) with the tensors' device the current one."""
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev.index)
    elif getattr(stream, "device", dev) != dev:
        raise ValueError(f"a stream of {stream.device} for tensors on {dev}")
    else:
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status != NS_OK:
        raise NSError(status, name)


def _need_on(dev, *ts):
    """Contiguous tensors (or None) of one device, a GPU."""
    if dev.type != "cuda":
        raise ValueError("tensors must be contiguous device tensors")
    for t in ts:
        if t is not None and not (t.is_contiguous() and t.device == dev):
            raise ValueError("tensors must be contiguous device tensors, on one device")


def _scratch(need, workspace, dev, stream):
    """The given workspace, or a new one where the call needs any."""
    if workspace is None:
        return _new((need,), (1,), torch.uint8, dev, stream) if need else None
    _need(workspace, "workspace", (torch.uint8,), 0)
    _need_on(dev, workspace)
    return workspace


_TYPES = {torch.float32: NS_F32, torch.bfloat16: NS_BF16}
_KINDS = tuple(_TYPES)


def _type_of(t):
    d = _TYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return d


def _need_rng(rng, dev):
    """Seed and offset: two 64-bit words on the device."""
    if rng is None:
        raise ValueError("dropout needs rng: seed and offset as an int64 device tensor")
    if rng.dtype not in (torch.int64, torch.uint64) or rng.numel() != 2:
        raise ValueError("rng: two 64-bit integers, seed and offset")
    _need_on(dev, rng)


def _need_like(t, name, shape, dtypes):
    """A caller's tensor of a shape and one of some types."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")


def _need_blocks(pair, name, rows, cols, width):
    """As _need_mx, for codes of `width` bytes a panel's row."""
    p = _mx_panels(cols)
    for t, what, n in ((pair[0], "codes", width), (pair[1], "scales", 8)):
        if t.dtype == torch.uint8 and t.shape == (p, rows, n):
            continue
        what = f"{name} {what}"
        _need(t, what, (torch.uint8,), p * rows * n)
        if t.dim() == 3:
            _need_shape(t, what, (p, rows, n))
        elif t.dim() != 1 and t.numel() != p * rows * n:
            raise ValueError(f"{what}: {t.numel()} elements, {p * rows * n} needed")


def _blocks(wanted, name, rows, cols, width, dev, stream, written):
    """(codes, scales) of an output operand: new ones (True), the caller's pair,
    noted in `written`, or None."""
    if wanted is None or wanted is False:
        return None
    if wanted is True:
        p = _mx_panels(cols)
        return (_new((p, rows, width), (rows * width, width, 1), torch.uint8, dev, stream),
                _new((p, rows, 8), (rows * 8, 8, 1), torch.uint8, dev, stream))
    _need_on(dev, *wanted)
    _need_blocks(wanted, name, rows, cols, width)
    written += wanted
    return wanted


def mx_dropout(x, drop, rng, out=None, stream=None):
    """k x / (1 - drop) for a float32/bfloat16 matrix, k drawn from the seed and
    offset in `rng` (two 64-bit integers on the device); of a gradient, with the
    same drop and rng, its own backward pass.  `out` may be x."""
    _need_2d(x, "x")
    rows, cols = x.shape
    dev, t = x.device, _type_of(x)
    _need_on(dev, x)
    _need_rng(rng, dev)
    given = out
    if out is None:
        out = _new((rows, cols), (cols, 1), x.dtype, dev, stream)
    else:
        _need_on(dev, out)
        _need_like(out, "out", x.shape, (x.dtype,))
    _launch(_lib.mx_dropout, "mx_dropout", dev, stream, x.data_ptr(), t, rows, cols, drop, rng.data_ptr(),
            out.data_ptr())
    if given is not None:
        _wrote((given,))
    return out


NormOut = collections.namedtuple("NormOut", "h rstd y mxfp8 mxfp4 kept")
NormOut.__doc__ = """What mx_rms_norm returns: the residual stream, the rows' 1 / rms, and y in the
wanted forms (None for the others); operands are (codes, scales)."""
NormGrads = collections.namedtuple("NormGrads", "dh dx dw")


def mx_rms_norm(x, weight, eps=1e-6, residual=None, drop=0.0, rng=None, y=None, mxfp8=None, mxfp4=None,
                kept=None, rstd=None, h=None, stream=None):
    """h = residual + dropout(x) and y = h / sqrt(mean(h^2) + eps) * weight, row by row.

    x [T][C] and residual (or None) are float32/bfloat16, weight [C] too; h has
    the residual's type (x's without one; it is x itself without residual and
    dropout) and may be given, also as the residual itself.  y (x's type unless
    given), mxfp8 (operand of mxfp8_gemm), mxfp4 (operand of mxfp4_gemm), kept
    (MXFP4 along the tokens, for mxfp4_linear_backward) and rstd (for
    mx_rms_norm_backward) are outputs: True for a new one, or the caller's
    tensor or (codes, scales); y where none of the four is asked for."""
    _need_2d(x, "x")
    T, C = shape = x.shape
    dev = x.device
    _need_on(dev, x, weight)
    if weight.shape != (C,):
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected {(C,)}")
    a = MxNormArgs()
    a.x, a.weight, a.T, a.C, a.eps, a.drop = x.data_ptr(), weight.data_ptr(), T, C, eps, drop
    a.xt = a.ht = _type_of(x)
    a.wt = _type_of(weight)
    written = []
    if residual is not None:
        _need_on(dev, residual)
        _need_like(residual, "residual", shape, _KINDS)
        a.residual = residual.data_ptr()
    if drop:
        _need_rng(rng, dev)
        a.rng = rng.data_ptr()
    if residual is not None or drop:
        kind = x.dtype if residual is None else residual.dtype
        if h is None:
            h = _new(shape, (C, 1), kind, dev, stream)
        else:
            _need_on(dev, h)
            _need_like(h, "h", shape, (kind,))
            written.append(h)
        a.h, a.ht = h.data_ptr(), _TYPES[kind]
    elif h is not None:
        raise ValueError("h is x itself without residual and dropout")
    p8 = _blocks(mxfp8, "mxfp8", T, C, 256, dev, stream, written)
    p4 = _blocks(mxfp4, "mxfp4", T, C, 128, dev, stream, written)
    pk = _blocks(kept, "kept", C, T, 128, dev, stream, written)
    if p8 is not None:
        a.codes8, a.scales8 = p8[0].data_ptr(), p8[1].data_ptr()
    if p4 is not None:
        a.codes4, a.scales4 = p4[0].data_ptr(), p4[1].data_ptr()
    if pk is not None:
        a.kept_codes, a.kept_scales = pk[0].data_ptr(), pk[1].data_ptr()
    if y is None and p8 is None and p4 is None and pk is None or y is True:
        y = _new(shape, (C, 1), x.dtype, dev, stream)
    elif y is False:
        y = None
    elif y is not None:
        _need_on(dev, y)
        _need_like(y, "y", shape, _KINDS)
        written.append(y)
    if y is not None:
        a.y, a.yt = y.data_ptr(), _TYPES[y.dtype]
    if rstd is None or rstd is False:
        rstd = None if pk is None else _new((T,), (1,), torch.float32, dev, stream)
    elif rstd is True:
        rstd = _new((T,), (1,), torch.float32, dev, stream)
    else:
        _need_on(dev, rstd)
        _need_like(rstd, "rstd", (T,), (torch.float32,))
        written.append(rstd)
    if rstd is not None:
        a.rstd = rstd.data_ptr()
    _launch(_lib.mx_rms_norm, "mx_rms_norm", dev, stream, ctypes.byref(a))
    if written:
        _wrote(written)
    return NormOut(x if h is None else h, rstd, y, p8, p4, pk)


def mx_rms_norm_backward_workspace_bytes(T, C):
    return int(_lib.mx_rms_norm_backward_workspace_bytes(T, C))


def mx_rms_norm_backward(dy, h, rstd, weight, dh=None, drop=0.0, rng=None, out=None, dx=None, dw=None,
                         need_dw=True, beta=0.0, x_dtype=None, workspace=None, stream=None):
    """Gradients of mx_rms_norm for dy [T][C], the gradient of y: (dh, dx, dw).

    h and rstd are the forward call's, dh what reaches h by other ways (the
    residual stream's gradient, or None); `out` takes the sum (may be dh
    itself).  dx is the gradient of x, through the same dropout, in x_dtype
    (dy's unless given); where it equals the gradient of h (no dropout, one
    type) it is that tensor.  dw = beta * dw + gradient is float32."""
    _need_2d(dy, "dy")
    T, C = shape = dy.shape
    dev = dy.device
    if dw is None and need_dw and float(beta) != 0.0:
        raise ValueError("beta != 0 adds to a dw that is given")
    _need_on(dev, dy, h, rstd, weight)
    _need_like(h, "h", shape, _KINDS)
    _need_like(rstd, "rstd", (T,), (torch.float32,))
    _need_like(weight, "weight", (C,), _KINDS)
    a = MxNormBackwardArgs()
    a.T, a.C, a.drop, a.beta = T, C, drop, beta
    a.dy, a.h, a.rstd, a.weight = dy.data_ptr(), h.data_ptr(), rstd.data_ptr(), weight.data_ptr()
    a.dyt, a.ht, a.wt = _type_of(dy), _TYPES[h.dtype], _TYPES[weight.dtype]
    written = []
    if dh is not None:
        _need_on(dev, dh)
        _need_like(dh, "dh", shape, (h.dtype,))
        a.dh_in = dh.data_ptr()
    if drop:
        _need_rng(rng, dev)
        a.rng = rng.data_ptr()
    if out is None:
        out = _new(shape, (C, 1), h.dtype, dev, stream)
    else:
        _need_on(dev, out)
        _need_like(out, "out", shape, (h.dtype,))
        written.append(out)
    a.dh = out.data_ptr()
    if x_dtype is None:
        x_dtype = dy.dtype if dx is None else dx.dtype
    if dx is not None:
        _need_on(dev, dx)
        _need_like(dx, "dx", shape, (x_dtype,))
        written.append(dx)
    elif drop or x_dtype != h.dtype:
        dx = _new(shape, (C, 1), x_dtype, dev, stream)
    if dx is not None:
        a.dx, a.xt = dx.data_ptr(), _type_of(dx)
    if not need_dw:
        dw = workspace = None
    else:
        if dw is None:
            dw = _new((C,), (1,), torch.float32, dev, stream)
        else:
            _need_on(dev, dw)
            _need_like(dw, "dw", (C,), (torch.float32,))
            written.append(dw)
        a.dweight = dw.data_ptr()
        workspace = _scratch(_lib.mx_rms_norm_backward_workspace_bytes(T, C), workspace, dev, stream)
    _launch(_lib.mx_rms_norm_backward, "mx_rms_norm_backward", dev, stream, ctypes.byref(a),
            *_ws_args(workspace))
    if written:
        _wrote(written)
    return NormGrads(out, out if dx is None else dx, dw)


def mxfp8_quantize(x, codes=None, scales=None, stream=None):
    """MXFP8 quantization of a 2-D float32/bfloat16 device tensor along its rows:
    (codes uint8 [panels][rows][256], scales uint8 [panels][rows][8])."""
    _need_2d(x, "x")
    rows, cols = x.shape
    dev, t = x.device, _type_of(x)
    p = _mx_panels(cols)
    given = codes, scales
    if codes is None:
        codes = _new((p, rows, 256), (rows * 256, 256, 1), torch.uint8, dev, stream)
    if scales is None:
        scales = _new((p, rows, 8), (rows * 8, 8, 1), torch.uint8, dev, stream)
    _need_on(dev, x, codes, scales)
    _need_blocks((codes, scales), "out", rows, cols, 256)
    _launch(_lib.mxfp8_quantize, "mxfp8_quantize", dev, stream, x.data_ptr(), t, rows, cols, codes.data_ptr(),
            scales.data_ptr())
    _wrote(given)
    return codes, scales


def mxfp8_dequantize(codes, scales, rows, cols, out_dtype=NS_F32, out=None, stream=None):
    """The values of an MXFP8 tensor, rows x cols."""
    dev = codes.device
    _need_on(dev, codes, scales, out)
    _need_blocks((codes, scales), "in", rows, cols, 256)
    given = out
    if out is None:
        out = _new((rows, cols), (cols, 1), _out_dtype(out_dtype), dev, stream)
    else:
        _need(out, "out", _KINDS, rows * cols)
    _launch(_lib.mxfp8_dequantize, "mxfp8_dequantize", dev, stream, codes.data_ptr(), scales.data_ptr(), rows, cols,
            out.data_ptr(), _TYPES[out.dtype])
    if given is not None:
        _wrote((given,))
    return out


def mxfp8_gemm_workspace_bytes(M, N, K):
    return int(_lib.mxfp8_gemm_workspace_bytes(M, N, K))


def mxfp8_gemm(p, q, M, N, K, alpha=1.0, beta=0.0, addend=None, out_dtype=NS_F32, out=None, workspace=None,
               split=True, stream=None):
    """out = beta*addend + alpha*(P Q^T) for p = (codes, scales) in MXFP8 and q in
    MXFP4, both along K: 8-bit activations by 4-bit weights.  float32 results
    keep every bit up to their FP32 sum; in bfloat16 ones a product loses up to
    2^-13 of the largest among its eight neighbours along K.

    With split=True (default) a workspace of mxfp8_gemm_workspace_bytes() is
    allocated when none is given."""
    (pc, ps), (qc, qs) = p, q
    dev = pc.device
    _need_on(dev, pc, ps, qc, qs, addend, out)
    _need_blocks(p, "p", M, K, 256)
    _need_mx(qc, qs, "q", N, K)
    given = out
    if out is None:
        out = _new((M, N), (N, 1), _out_dtype(out_dtype), dev, stream)
    else:
        _need(out, "out", _KINDS, M * N)
    add = None
    if beta:
        _need(addend, "addend", (torch.float32,), M * N)
        add = None if addend is None else addend.data_ptr()
    if workspace is not None or split:
        workspace = _scratch(_lib.mxfp8_gemm_workspace_bytes(M, N, K), workspace, dev, stream)
    _launch(_lib.mxfp8_gemm, "mxfp8_gemm", dev, stream, pc.data_ptr(), ps.data_ptr(), qc.data_ptr(), qs.data_ptr(),
            M, N, K, alpha, beta, add, out.data_ptr(), _TYPES[out.dtype], *_ws_args(workspace))
    if given is not None:
        _wrote((given,))
    return out


def _need_nv_rows(codes, scales, N, K):
    """NVFP4 weights of N rows: matrices have to be the call's, since a transposed
    operand (quantized along the other axis) has as many elements; other views
    need its size."""
    for t, what, n in ((codes, "codes", K // 2), (scales, "scales", K // 16)):
        if t.dtype != torch.uint8:
            raise TypeError("w: codes and scales are uint8")
        if t.dim() == 2:
            _need_shape(t, f"w {what}", (N, n))
        elif t.numel() != N * n:
            raise ValueError(f"w {what}: {t.numel()} elements, {N * n} needed")


def nvfp4_linear(x, w, N, out=None, stream=None):
    """y = x W^T for x [T][K] (float32/bfloat16, not quantized) and NVFP4 weights
    w = (codes, scales, global_scale) of [N][K] as nvfp4_quantize returns them;
    y takes x's dtype unless `out` is given.  Built for few tokens."""
    codes, scales, sg = w
    _need_2d(x, "x")
    T, K = x.shape
    dev, t = x.device, _type_of(x)
    _need_on(dev, x, codes, scales, sg, out)
    _need_nv_rows(codes, scales, N, K)
    _need(sg, "global_scale", (torch.float32,), 1)
    given = out
    if out is None:
        out = _new((T, N), (N, 1), x.dtype, dev, stream)
    else:
        _need(out, "out", _KINDS, T * N)
    _launch(_lib.nvfp4_linear, "nvfp4_linear", dev, stream, x.data_ptr(), t, T, K, codes.data_ptr(),
            scales.data_ptr(), sg.data_ptr(), N, out.data_ptr(), _TYPES[out.dtype])
    if given is not None:
        _wrote((given,))
    return out
