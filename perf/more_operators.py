"""Cases that measure the operators between two 4-bit linear layers: the
root-mean-square norm with the residual's addition, dropout and outputs in 8 or
4 bits, its backward pass, dropout by itself, products of 8-bit activations
with 4-bit weights, and products with NVFP4 weights.

Each case is a plain dict; `prepare` draws its inputs on the GPU from a seed,
`run` makes one pass through the operator, in plain torch operations where
`own` is false and through the framework where it is true, and `exact` gives
the definition's values in 64 bits.

Storage that inputs come in: MXFP4 and MXFP8 matrices are cut along the blocked
axis into panels of 256 elements, codes [panels][rows][128 or 256] bytes,
scales [panels][rows][8] E8M0 bytes, one per block of 32; what lies behind a
row's end is zero.  NVFP4 weights are [rows][cols / 2] code bytes (element 2i
in the low nibble), [rows][cols / 16] E4M3 scale bytes and one FP32 scale.

Dropout: element (t, c) takes half c % 2 of word c / 2 % 4 of Philox4x32-10
with counter (c / 8, t, offset low, offset high) and key (seed low, seed high);
it is kept where those 16 bits are at least round(65536 p).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
PANEL, BLOCK = 256, 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token in front of a layer: launches count
        {"name": "norm 1 token", "op": "norm", "T": 1, "C": 4096, "type": "bf16", "res": "bf16", "out": "mxfp8", "drop": 0.0, "train": False},
        # a prompt, the residual stream in FP32
        {"name": "norm 8192 tokens", "op": "norm", "T": 8192, "C": 4096, "type": "bf16", "res": "f32", "out": "mxfp8", "drop": 0.0, "train": False},
        # a training step with dropout on the branch: MXFP4 along features and tokens, then the gradients
        {"name": "norm step 8192 tokens", "op": "norm", "T": 8192, "C": 4096, "type": "bf16", "res": "bf16", "out": "mxfp4", "drop": 0.1, "train": True},
        # a ragged batch without a residual, everything in FP32, with its gradients
        {"name": "norm step 333x1111", "op": "norm", "T": 333, "C": 1111, "type": "f32", "res": "", "out": "y", "drop": 0.0, "train": True},
        # dropout behind the MLP's activation and its gradient
        {"name": "dropout 8192x11008", "op": "dropout", "T": 8192, "C": 11008, "type": "bf16", "drop": 0.1},
        # a small ragged one
        {"name": "dropout 777x1501", "op": "dropout", "T": 777, "C": 1501, "type": "f32", "drop": 0.5},
        # a prompt through the gated MLP's up projection, 8-bit activations
        {"name": "product8 8192x11008x4096", "op": "product8", "M": 8192, "N": 11008, "K": 4096, "out": "bf16", "beta": 0.0},
        # a ragged one added to what is there, in FP32
        {"name": "product8 1000x777x1501 add", "op": "product8", "M": 1000, "N": 777, "K": 1501, "out": "f32", "beta": 1.0},
        # one token: the weights' bytes count
        {"name": "product8 1 token", "op": "product8", "M": 1, "N": 11008, "K": 4096, "out": "bf16", "beta": 0.0},
        # one token through NVFP4 weights
        {"name": "nvfp4 linear 1 token", "op": "nvfp4", "T": 1, "N": 11008, "K": 4096, "type": "bf16"},
        # a small batch of requests through the down projection
        {"name": "nvfp4 linear 16 tokens", "op": "nvfp4", "T": 16, "N": 4096, "K": 11008, "type": "bf16"},
        # a few FP32 rows, a ragged number of outputs
        {"name": "nvfp4 linear 5x777x1504", "op": "nvfp4", "T": 5, "N": 777, "K": 1504, "type": "f32"},
    ]


def _size(rng, lo, hi):
    """A size spread over the range's logarithm, as often odd as it falls."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dropout", "product8", "nvfp4"])
    if op == "norm":
        train = rng.random() < 0.5
        c = {"op": op, "T": _size(rng, 1, 8192), "C": _size(rng, 16, 4096), "type": rng.choice(["f32", "bf16"]),
             "out": rng.choice(["y", "mxfp8", "mxfp4"]), "drop": rng.choice([0.0, 0.1, 0.25]), "train": train}
        c["res"] = rng.choice([c["type"], "f32"]) if c["drop"] else rng.choice(["", c["type"], "f32"])
        return c
    if op == "dropout":
        return {"op": op, "T": _size(rng, 1, 8192), "C": _size(rng, 1, 8192), "type": rng.choice(["f32", "bf16"]),
                "drop": rng.choice([0.05, 0.1, 0.5])}
    if op == "product8":
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 16, 11008), "K": _size(rng, 16, 4096),
                "out": rng.choice(["f32", "bf16"]), "beta": rng.choice([0.0, 1.0, 0.5])}
    return {"op": op, "T": _size(rng, 1, 32), "N": _size(rng, 16, 11008), "K": 16 * _size(rng, 1, 688),
            "type": rng.choice(["f32", "bf16"])}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _heavy(g, rows, cols, scale):
    """Student-t(3) * scale with 0.1% of the entries 50 times larger: the heavy
    tails of activations and gradients."""
    x = torch.randn((rows, cols), generator=g, device=DEV)
    chi = torch.zeros((rows, cols), device=DEV)
    for _ in range(3):
        chi += torch.randn((rows, cols), generator=g, device=DEV).square_()
    x = x.div_(chi.div_(3.0).sqrt_()).mul_(scale)
    far = torch.rand((rows, cols), generator=g, device=DEV) < 0.001
    return torch.where(far, x * 50.0, x)


def _rng(seed):
    """Seed and offset of the dropout's generator, as a device tensor."""
    return torch.tensor([(int(seed) * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), int(seed) * 7 + (5 << 32)], dtype=torch.int64, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "norm":
        T, C, ty = case["T"], case["C"], TYPES[case["type"]]
        rt = TYPES[case["res"] or case["type"]]
        s = {"case": case, "x": _heavy(g, T, C, 0.3).to(ty), "w": (1.0 + 0.2 * torch.randn(C, generator=g, device=DEV)).to(ty),
             "r": _heavy(g, T, C, 1.0).to(rt) if case["res"] else None, "rng": _rng(seed) if case["drop"] else None}
        if case["train"]:
            s["dy"] = _heavy(g, T, C, 1e-3).to(ty)
            s["dh"] = (1e-3 * torch.randn((T, C), generator=g, device=DEV)).to(rt) if case["res"] else None
        return s
    if op == "dropout":
        T, C, ty = case["T"], case["C"], TYPES[case["type"]]
        return {"case": case, "x": _heavy(g, T, C, 1.0).to(ty), "dy": _heavy(g, T, C, 1e-3).to(ty), "rng": _rng(seed)}
    if op == "product8":
        M, N, K = case["M"], case["N"], case["K"]
        s = {"case": case, "p": _pack8(_heavy(g, M, K, 1.0)), "q": _pack4(0.02 * torch.randn((N, K), generator=g, device=DEV))}
        if case["beta"]:
            s["addend"] = torch.randn((M, N), generator=g, device=DEV)
        return s
    T, N, K = case["T"], case["N"], case["K"]
    return {"case": case, "x": _heavy(g, T, K, 1.0).to(TYPES[case["type"]]), "w": _pack_nv(0.02 * torch.randn((N, K), generator=g, device=DEV))}


# ------------------------------------------------------------- plain form --

def _blocks(x):
    """[rows][blocks of 32] of x in FP32, zeros behind a row's end up to a whole panel."""
    rows, cols = x.shape
    v = torch.zeros((rows, -(-cols // PANEL) * PANEL), dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    return v.view(rows, -1, BLOCK)


def _scale_exponent(v, emax):
    """floor(log2 max) - emax of each block, E8M0's range; -127 for zeros."""
    top = v.abs().amax(-1)
    e = (torch.frexp(top)[1] - 1 - emax).clamp_(-127, 127)
    return torch.where(top > 0, e, torch.full_like(e, -127))


def _e2m1(a):
    """E2M1 codes of a: the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    neg = torch.signbit(a)
    a = a.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += neg.to(torch.uint8) * 8
    return code


def _e2m1_values(code):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=code.device)
    return table[code.int()]


def _encode4(x):
    v = _blocks(x)
    e = _scale_exponent(v, 2)
    return _e2m1(torch.ldexp(v, -e[..., None])), e


def _encode8(x):
    v = _blocks(x)
    e = _scale_exponent(v, 8)
    return torch.ldexp(v, -e[..., None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), e


def _in_panels(a, width):
    return a.reshape(a.shape[0], -1, width).transpose(0, 1).contiguous()


def _pack4(x):
    code, e = _encode4(x)
    code = code.view(code.shape[0], -1)
    return _in_panels(code[:, 0::2] | (code[:, 1::2] << 4), 128), _in_panels((e + 127).to(torch.uint8), 8)


def _pack8(x):
    code, e = _encode8(x)
    return _in_panels(code.view(torch.uint8), 256), _in_panels((e + 127).to(torch.uint8), 8)


def _scaled(v, e, cols):
    return torch.ldexp(v, e[..., None]).view(v.shape[0], -1)[:, :cols]


def _held4(x):
    """What x becomes when it is held in MXFP4 along its rows, in FP32."""
    code, e = _encode4(x)
    return _scaled(_e2m1_values(code), e, x.shape[1])


def _held8(x):
    code, e = _encode8(x)
    return _scaled(code.float(), e, x.shape[1])


def _rows_of(a):
    return a.transpose(0, 1).reshape(a.shape[1], -1)


def _unpack4(q, cols):
    pair, byte = _rows_of(q[0]), _rows_of(q[1])
    code = torch.stack((pair & 15, pair >> 4), -1).view(pair.shape[0], -1, BLOCK)
    return _scaled(_e2m1_values(code), byte.int() - 127, cols)


def _unpack8(p, cols):
    code, byte = _rows_of(p[0]), _rows_of(p[1])
    return _scaled(code.view(torch.float8_e4m3fn).float().view(code.shape[0], -1, BLOCK), byte.int() - 127, cols)


def _pack_nv(w):
    """NVFP4 weights: blocks of 16 along the rows."""
    rows, cols = w.shape
    v = w.view(rows, -1, 16)
    sg = v.abs().amax() / 2688.0
    scale = (v.abs().amax(-1) / (6.0 * sg)).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = (scale.float() * sg)[..., None]
    code = _e2m1(torch.where(unit > 0, v / unit, torch.zeros_like(v))).view(rows, -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale.view(torch.uint8), sg.reshape(1)


def _unpack_nv(w):
    pair, scale, sg = w
    code = torch.stack((pair & 15, pair >> 4), -1).view(pair.shape[0], -1, 16)
    return (_e2m1_values(code) * scale.view(torch.float8_e4m3fn).float()[..., None]).view(pair.shape[0], -1) * sg


def _mul32(a, b):
    """High and low words of a * b, a a 32-bit number, b 32-bit values in 64."""
    t, u = a * (b & 0xFFFF), a * (b >> 16)
    return (u + (t >> 16)) >> 16, (t + ((u & 0xFFFF) << 16)) & 0xFFFFFFFF


def _keep(case, rng):
    """The elements that dropout keeps, and what it multiplies them by."""
    T, C = case["T"], case["C"]
    cut = int(math.floor(case["drop"] * 65536.0 + 0.5))
    seed, off = rng[0], rng[1]
    c0 = torch.arange(-(-C // 8), device=DEV).expand(T, -1)
    c1 = torch.arange(T, device=DEV)[:, None].expand_as(c0)
    c2, c3 = (off & 0xFFFFFFFF).expand_as(c0), ((off >> 32) & 0xFFFFFFFF).expand_as(c0)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul32(0xD2511F53, c0)
        h1, l1 = _mul32(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack((c0, c1, c2, c3), -1)
    half = torch.stack((words & 0xFFFF, words >> 16), -1).reshape(T, -1)[:, :C]
    return half >= cut, 65536.0 / (65536 - cut)


def _dropped(x, keep, scale):
    return torch.where(keep, x * torch.tensor(scale, dtype=torch.float32).to(x.dtype), torch.zeros((), dtype=x.dtype, device=x.device))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x, w, r, ty = s["x"], s["w"].float(), s["r"], s["x"].dtype
        out = {}
        h = x
        if case["drop"]:
            keep, scale = _keep(case, s["rng"])
        if r is not None:       # one rounding of the sum: product and sum in 64 bits
            branch = _dropped(x.double(), keep, scale) if case["drop"] else x.double()
            h = out["h"] = (r.double() + branch).float().to(r.dtype)
        # the sum in 64 bits: codes of values next to a border hang on it
        rstd = (1.0 / (h.double().square().mean(1) + EPS).sqrt()).float()
        xhat = h.float() * rstd[:, None]
        y = xhat * w
        if case["out"] == "y":
            out["y"] = y.to(ty)
        elif case["out"] == "mxfp8":
            out["y8"] = _held8(y).to(torch.bfloat16)
        else:
            out["y4"] = _held4(y).to(torch.bfloat16)
            if case["train"]:
                out["kept"] = _held4(y.t()).t().contiguous().to(torch.bfloat16)
        if case["train"]:
            dy = s["dy"].float()
            g = dy * w
            dh = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
            if s["dh"] is not None:
                dh = dh + s["dh"].float()
            out["dh"] = dh.to(h.dtype)
            if case["drop"]:
                out["dx"] = _dropped(dh, keep, scale).to(ty)
            out["dw"] = (dy * xhat).double().sum(0).float()
        return out
    if op == "dropout":
        keep, scale = _keep(case, s["rng"])
        return [_dropped(v.float(), keep, scale).to(v.dtype) for v in (s["x"], s["dy"])]
    if op == "product8":
        y = _unpack8(s["p"], case["K"]) @ _unpack4(s["q"], case["K"]).t()
        if case["beta"]:
            y = y + case["beta"] * s["addend"]
        return y.to(TYPES[case["out"]])
    return (s["x"].float() @ _unpack_nv(s["w"]).t()).to(s["x"].dtype)


# ---------------------------------------------------------------- the calls --

def _run_own(s):
    import newton_schulz_amd as ns
    case = s["case"]
    op = case["op"]
    if op == "norm":
        T, C, train = case["T"], case["C"], case["train"]
        n = ns.mx_rms_norm(s["x"], s["w"], EPS, residual=s["r"], drop=case["drop"], rng=s["rng"], y=case["out"] == "y",
                           mxfp8=case["out"] == "mxfp8", mxfp4=case["out"] == "mxfp4", kept=case["out"] == "mxfp4" and train, rstd=train)
        out = {}
        if s["r"] is not None:
            out["h"] = n.h
        if n.y is not None:
            out["y"] = n.y
        if n.mxfp8 is not None:
            out["y8"] = ns.mxfp8_dequantize(*n.mxfp8, T, C, ns.NS_BF16)
        if n.mxfp4 is not None:
            out["y4"] = ns.mxfp4_dequantize(*n.mxfp4, T, C, ns.NVFP4_ROWS, ns.NS_BF16)
        if n.kept is not None:
            out["kept"] = ns.mxfp4_dequantize(*n.kept, T, C, ns.NVFP4_COLS, ns.NS_BF16)
        if train:
            g = ns.mx_rms_norm_backward(s["dy"], n.h, n.rstd, s["w"], dh=s["dh"], drop=case["drop"], rng=s["rng"])
            out["dh"], out["dw"] = g.dh, g.dw
            if case["drop"]:
                out["dx"] = g.dx
        return out
    if op == "dropout":
        return [ns.mx_dropout(v, case["drop"], s["rng"]) for v in (s["x"], s["dy"])]
    if op == "product8":
        return ns.mxfp8_gemm(s["p"], s["q"], case["M"], case["N"], case["K"], beta=case["beta"], addend=s.get("addend"),
                             out_dtype=ns.NS_F32 if case["out"] == "f32" else ns.NS_BF16)
    return ns.nvfp4_linear(s["x"], s["w"], case["N"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work --

def _bytes(t):
    return 4 if t == "f32" else 2


def work(case):
    op = case["op"]
    if op == "norm":
        n, size = case["T"] * case["C"], _bytes(case["type"])
        res = _bytes(case["res"] or case["type"])
        b = n * size + case["C"] * size + (2 * n * res if case["res"] else 0)       # x, the weight, the residual read and written
        if case["out"] == "y":
            b += n * size
        elif case["out"] == "mxfp8":
            b += n * (2 * (1 + 1 / BLOCK) + 2)                                     # written, read back, the values
        else:
            b += (2 if case["train"] else 1) * n * (2 * (0.5 + 1 / BLOCK) + 2)
        if case["train"]:
            b += n * (size + 2 * res) + (n * res if case["res"] else 0) + (n * size if case["drop"] else 0) + 4 * case["C"]
        return {"bytes": b, "flops": (20.0 if case["train"] else 6.0) * n}
    if op == "dropout":
        n = case["T"] * case["C"]
        return {"bytes": 4 * n * _bytes(case["type"]), "flops": 4.0 * n}
    if op == "product8":
        M, N, K = case["M"], case["N"], case["K"]
        out = M * N * (_bytes(case["out"]) + (4 if case["beta"] else 0))
        return {"bytes": M * K * (1 + 1 / BLOCK) + N * K * (0.5 + 1 / BLOCK) + out, "flops": 2.0 * M * N * K}
    T, N, K, size = case["T"], case["N"], case["K"], _bytes(case["type"])
    return {"bytes": N * K * (0.5 + 1 / 16) + size * T * (K + N), "flops": 2.0 * T * N * K}


# ------------------------------------------------------------------ exact --

def _held64(x, emax, mant, low, top):
    """x in blocks of 32 along its rows from the definition, in FP64: `mant`
    bits behind the leading one, quanta of 2^low at least, values up to `top`,
    in units of 2^(floor(log2 max) - emax)."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % BLOCK)).unflatten(1, (-1, BLOCK))
    m = v.abs().amax(-1, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(m.clamp(min=2.0 ** -149))) - emax).clamp(-127, 127))
    r = v / unit
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -40))).sub(mant).clamp(min=low))
    return ((r / step).round() * step).clamp(-top, top).mul(unit).flatten(1)[:, :cols]


def _mx4(x):
    return _held64(x, 2, 1, -1, 6.0)


def _mx8(x):
    return _held64(x, 8, 3, -9, 448.0)


def _decode_e2m1(nib):
    sign, mag = torch.where(nib >= 8, -1.0, 1.0).double(), nib % 8
    # code 2e + m is (1 + m / 2) 2^(e - 1), and m / 2 where e is 0
    e, m = torch.div(mag, 2, rounding_mode="floor"), mag % 2
    return sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)


def _decode_e4m3(byte):
    b = byte.to(torch.float64)
    sign, b = torch.where(b >= 128, -1.0, 1.0).double(), b % 128
    e, m = torch.div(b, 8, rounding_mode="floor"), b % 8
    return sign * torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)


def _nibbles(code):
    return torch.cat(((code & 15)[..., None], (code >> 4)[..., None]), -1).flatten(-2).to(torch.float64)


def _operand64(q, cols, decode):
    code, byte = (t.permute(1, 0, 2) for t in q)
    val = decode(code).unflatten(2, (8, 32)) * torch.exp2(byte.double() - 127)[..., None]
    return val.flatten(1)[:, :cols]


def _factors64(case, rng):
    """What dropout multiplies every element by, from numpy's 64-bit words."""
    T, C = case["T"], case["C"]
    seed, off = (int(v) for v in rng.cpu())
    cut = int(math.floor(case["drop"] * 65536.0 + 0.5))
    low = np.uint64(0xFFFFFFFF)
    n = -(-C // 8)
    a = np.tile(np.arange(n, dtype=np.uint64), T)
    b = np.repeat(np.arange(T, dtype=np.uint64), n)
    c = np.full(T * n, off & 0xFFFFFFFF, np.uint64)
    d = np.full(T * n, (off >> 32) & 0xFFFFFFFF, np.uint64)
    for i in range(10):
        ka = np.uint64(((seed & 0xFFFFFFFF) + i * 0x9E3779B9) & 0xFFFFFFFF)
        kb = np.uint64((((seed >> 32) & 0xFFFFFFFF) + i * 0xBB67AE85) & 0xFFFFFFFF)
        p, q = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (q >> np.uint64(32)) ^ b ^ ka, q & low, (p >> np.uint64(32)) ^ d ^ kb, p & low
    bits = np.stack((a, b, c, d), -1).astype("<u4").view("<u2").reshape(T, n * 8)[:, :C]
    return torch.from_numpy((bits >= cut) * (65536.0 / (65536 - cut))).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        w, out = s["w"].double(), {}
        f = _factors64(case, s["rng"]) if case["drop"] else 1.0
        h = s["x"].double()
        if case["res"]:
            h = s["r"].double() + f * h
            out["h"] = h
            # the norm is of the residual stream as it is held
            h = h.to(s["r"].dtype).double()
        u = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["C"] + EPS)
        y = u * w
        if case["out"] == "y":
            out["y"] = y
        elif case["out"] == "mxfp8":
            out["y8"] = _mx8(y)
        else:
            out["y4"] = _mx4(y)
            if case["train"]:
                out["kept"] = _mx4(y.t()).t().contiguous()
        if case["train"]:
            dy = s["dy"].double()
            inv = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / case["C"] + EPS)
            dh = inv * (dy * w - u * ((dy * w * u).sum(1, keepdim=True) / case["C"]))
            if case["res"]:
                dh = dh + s["dh"].double()
            out["dh"] = dh
            if case["drop"]:
                out["dx"] = dh * f
            out["dw"] = (dy * u).sum(0)
        return out
    if op == "dropout":
        f = _factors64(case, s["rng"])
        return [s["x"].double() * f, s["dy"].double() * f]
    if op == "product8":
        y = _operand64(s["p"], case["K"], _decode_e4m3) @ _operand64(s["q"], case["K"], lambda c: _decode_e2m1(_nibbles(c))).mT
        return y + case["beta"] * s["addend"].double() if case["beta"] else y
    code, scale, sg = s["w"]
    w = _decode_e2m1(_nibbles(code)).unflatten(1, (-1, 16)) * _decode_e4m3(scale)[..., None]
    return (s["x"].double() @ w.flatten(1).mT) * sg.double()
