"""Cases that measure the MXFP4 operators (quantizer, product, linear layer)
and the 16-bit Newton-Schulz operators (orthogonalization, Muon step).

Each case is a plain dict; `prepare` draws its inputs on the GPU from a seed,
`run` makes one pass through the operator, in plain torch operations where
`own` is false and through the framework where it is true, and `exact` gives
the definition's values in 64 bits.

MXFP4 storage (both forms take operands in it): a matrix is cut along the
blocked axis into panels of 256 elements; codes are [panels][rows][128] bytes
(element 2i in the low nibble), scales [panels][rows][8] E8M0 bytes, one per
32-element block, and what lies behind a row's end is an all-zero block.
"""
import math

import torch

own = False

DEV = "cuda"
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
PANEL, BLOCK = 256, 32
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the standalone quantizer's workload: a 2^28-element BF16 tensor there and back
        {"name": "quantize 16384x16384 bf16", "op": "quantize", "rows": 16384, "cols": 16384, "axis": "rows", "type": "bf16"},
        # a small ragged FP32 tensor blocked down its columns: launches count
        {"name": "quantize 333x1111 f32 down", "op": "quantize", "rows": 333, "cols": 1111, "axis": "cols", "type": "f32"},
        # activations of one layer, wanted along the features (forward) and along the tokens (weight gradient)
        {"name": "quantize both 8192x4096", "op": "quantize", "rows": 8192, "cols": 4096, "axis": "both", "type": "bf16"},
        # the gated MLP's up projection on 8192 tokens, both operands held in 4 bits
        {"name": "product 8192x11008x4096", "op": "product", "M": 8192, "N": 11008, "K": 4096, "out": "bf16", "beta": 0.0},
        # a ragged product added to what is there, in FP32
        {"name": "product 1000x777x1501 add", "op": "product", "M": 1000, "N": 777, "K": 1501, "out": "f32", "beta": 1.0},
        # one token through the MLP's up projection: the weights' bytes count
        {"name": "linear 1 token", "op": "linear", "T": 1, "N": 11008, "K": 4096, "type": "bf16", "train": False},
        # a training step of the layer: forward, then the gradients of input and weights
        {"name": "linear step 8192 tokens", "op": "linear", "T": 8192, "N": 4096, "K": 4096, "type": "bf16", "train": True},
        # the smallest Newton-Schulz workload: launches count
        {"name": "orthogonalize 256x512", "op": "orthogonalize", "m": 256, "n": 512, "count": 1, "type": "f32"},
        # the MLP's up projection, its gradient taller than wide
        {"name": "orthogonalize 11008x4096", "op": "orthogonalize", "m": 11008, "n": 4096, "count": 1, "type": "bf16"},
        # the square 2048 gradients of four layers in one call
        {"name": "orthogonalize 4x 2048x2048", "op": "orthogonalize", "m": 2048, "n": 2048, "count": 4, "type": "bf16"},
        # the key and value projections' weights of four blocks: one optimizer step
        {"name": "muon 8x 1024x4096", "op": "muon", "m": 1024, "n": 4096, "count": 8, "type": "bf16", "nesterov": True},
        # one ragged weight matrix
        {"name": "muon 1000x333", "op": "muon", "m": 1000, "n": 333, "count": 1, "type": "f32", "nesterov": False},
    ]


def _size(rng, lo, hi):
    """A size spread over the range's logarithm, as often odd as it falls."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "linear", "orthogonalize", "muon"])
    if op == "quantize":
        rows, cols = _size(rng, 1, 16384), _size(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": cols, "axis": rng.choice(["rows", "cols", "both"]), "type": rng.choice(["f32", "bf16"])}
    if op == "product":
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 16, 11008), "K": _size(rng, 16, 4096),
                "out": rng.choice(["f32", "bf16"]), "beta": rng.choice([0.0, 1.0, 0.5])}
    if op == "linear":
        train = rng.random() < 0.5
        return {"op": op, "T": _size(rng, 1, 8192), "N": _size(rng, 64, 4096 if train else 11008), "K": _size(rng, 64, 4096),
                "type": rng.choice(["f32", "bf16"]), "train": train}
    m, n = _size(rng, 48, 4096), _size(rng, 48, 4096)
    c = {"op": op, "m": m, "n": n, "count": rng.choice([1, 1, 2, 3]), "type": rng.choice(["f32", "bf16"])}
    if op == "muon":
        c["nesterov"] = rng.random() < 0.5
    return c


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


def _gradient(g, rows, cols):
    """A rank-32 signal of norm 1 with N(0, 0.01^2) noise and 0.1% of the
    entries 50 times larger: a weight matrix's gradient."""
    r = min(32, rows, cols)
    s = torch.randn((rows, r), generator=g, device=DEV) @ torch.randn((r, cols), generator=g, device=DEV)
    x = s / s.norm() + 0.01 * torch.randn((rows, cols), generator=g, device=DEV)
    far = torch.rand((rows, cols), generator=g, device=DEV) < 0.001
    return torch.where(far, x * 50.0, x)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        return {"case": case, "x": _heavy(g, case["rows"], case["cols"], 0.02).to(TYPES[case["type"]])}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s = {"case": case, "p": _pack(_heavy(g, M, K, 1.0)), "q": _pack(0.02 * torch.randn((N, K), generator=g, device=DEV))}
        if case["beta"]:
            s["addend"] = torch.randn((M, N), generator=g, device=DEV)
        return s
    if op == "linear":
        T, N, K, ty = case["T"], case["N"], case["K"], TYPES[case["type"]]
        w = 0.02 * torch.randn((N, K), generator=g, device=DEV)
        s = {"case": case, "x": _heavy(g, T, K, 1.0).to(ty), "w": _pack(w)}
        if case["train"]:  # a trained layer's weights are held along both axes
            s["wt"] = _pack(w.t())
            s["dy"] = _heavy(g, T, N, 1e-3).to(ty)
        return s
    m, n, ty = case["m"], case["n"], TYPES[case["type"]]
    s = {"case": case, "g": [_gradient(g, m, n).to(ty) for _ in range(case["count"])]}
    if op == "muon":
        s["w"] = [(0.02 * torch.randn((m, n), generator=g, device=DEV)).to(torch.bfloat16) for _ in range(case["count"])]
        s["mom"] = [5.0 * _gradient(g, m, n) for _ in range(case["count"])]
    return s


MUON = {"lr": 2e-3, "momentum": 0.95, "weight_decay": 0.1}


def _muon_scale(m, n):
    return 0.2 * math.sqrt(max(m, n))


# ------------------------------------------------------------- plain form --

def _panels(n):
    return -(-n // PANEL)


def _encode(x):
    """E2M1 codes [rows][panels * 256] and E8M0 bytes [rows][panels * 8] of
    blocks along the rows of x: the scale is the power of two at the block's
    largest magnitude over 4, a magnitude rounds to the nearest of
    0, .5, 1, 1.5, 2, 3, 4, 6 with ties to the even code."""
    rows, cols = x.shape
    v = torch.zeros((rows, _panels(cols) * PANEL), dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, -1, BLOCK)
    top = v.abs().amax(-1)
    e = (torch.frexp(top)[1] - 3).clamp_(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    a = torch.ldexp(v, -e[..., None])
    neg = torch.signbit(a)
    a.abs_()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += neg.to(torch.uint8) * 8
    return code.view(rows, -1), (e + 127).to(torch.uint8)


def _values(code, byte, cols):
    """The FP32 values that codes and scale bytes stand for, the first `cols` of each row."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=code.device)
    rows = code.shape[0]
    v = table[code.view(rows, -1, BLOCK).int()] * torch.ldexp(torch.ones((), device=code.device), byte.int() - 127)[..., None]
    return v.view(rows, -1)[:, :cols]


def _pack(x):
    """x quantized along its rows, in the storage form."""
    code, byte = _encode(x)
    rows = code.shape[0]
    pair = code[:, 0::2] | (code[:, 1::2] << 4)
    return (pair.view(rows, -1, 128).transpose(0, 1).contiguous(), byte.view(rows, -1, 8).transpose(0, 1).contiguous())


def _unpack(q, cols):
    pair, byte = (t.transpose(0, 1).reshape(t.shape[1], -1) for t in q)
    return _values(torch.stack((pair & 15, pair >> 4), -1).view(pair.shape[0], -1), byte, cols)


def _held(x):
    """What x becomes when it is held in MXFP4 along its rows, in FP32."""
    return _values(*_encode(x), x.shape[1])


def _orthogonalize(u):
    """STEPS Newton-Schulz steps on u in FP32, on the side where rows <= columns."""
    tall = u.shape[0] > u.shape[1]
    x = u.t() if tall else u
    x = x / (x.square().sum().sqrt() + 1e-7)
    a, b, c = QUINTIC
    for _ in range(STEPS):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if tall else x


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        x, ty = s["x"], TYPES[case["type"]]
        along = [_held(x).to(ty)] if case["axis"] != "cols" else []
        down = [_held(x.t()).t().contiguous().to(ty)] if case["axis"] != "rows" else []
        return along + down
    if op == "product":
        y = _unpack(s["p"], case["K"]) @ _unpack(s["q"], case["K"]).t()
        if case["beta"]:
            y = y + case["beta"] * s["addend"]
        return y.to(TYPES[case["out"]])
    if op == "linear":
        x, ty = s["x"], TYPES[case["type"]]
        y = (_held(x) @ _unpack(s["w"], case["K"]).t()).to(ty)
        if not case["train"]:
            return y
        dy = s["dy"]
        dx = _held(dy) @ _unpack(s["wt"], case["N"]).t()
        dw = _held(dy.t()) @ _held(x.t()).t()
        return {"y": y, "dx": dx.to(ty), "dw": dw.to(ty)}
    if op == "orthogonalize":
        return [_orthogonalize(g.float()).to(torch.bfloat16) for g in s["g"]]
    mu, lr, wd = MUON["momentum"], MUON["lr"], MUON["weight_decay"]
    for g, mom, w in zip(s["g"], s["mom"], s["w"]):
        mom.mul_(mu).add_(g.float())
        u = g.float() + mu * mom if case["nesterov"] else mom
        w.copy_((1.0 - lr * wd) * w.float() - lr * _muon_scale(*w.shape) * _orthogonalize(u))
    return {"w": s["w"], "mom": s["mom"]}


# ---------------------------------------------------------------- the calls --

def _run_own(s):
    import newton_schulz_amd as ns
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        x, R, C = s["x"], case["rows"], case["cols"]
        ty = ns.NS_F32 if case["type"] == "f32" else ns.NS_BF16
        if case["axis"] == "both":
            along, down = ns.mxfp4_quantize_both(x)
            return [ns.mxfp4_dequantize(*along, R, C, ns.NVFP4_ROWS, ty), ns.mxfp4_dequantize(*down, R, C, ns.NVFP4_COLS, ty)]
        axis = ns.NVFP4_ROWS if case["axis"] == "rows" else ns.NVFP4_COLS
        return [ns.mxfp4_dequantize(*ns.mxfp4_quantize(x, axis), R, C, axis, ty)]
    if op == "product":
        return ns.mxfp4_gemm(s["p"], s["q"], case["M"], case["N"], case["K"], beta=case["beta"], addend=s.get("addend"),
                             out_dtype=ns.NS_F32 if case["out"] == "f32" else ns.NS_BF16)
    if op == "linear":
        if not case["train"]:
            return ns.mxfp4_linear(s["x"], s["w"], case["N"])
        y, kept = ns.mxfp4_linear(s["x"], s["w"], case["N"], keep=True)
        dx, dw = ns.mxfp4_linear_backward(s["dy"], s["wt"], kept, case["K"])
        return {"y": y, "dx": dx, "dw": dw}
    if op == "orthogonalize":
        return ns.ns_orthogonalize_f16_grouped(s["g"], [QUINTIC] * STEPS, out_dtype=ns.NS_BF16)
    ns.ns_muon_step(s["w"], s["mom"], s["g"], [QUINTIC] * STEPS, scales=[_muon_scale(*w.shape) for w in s["w"]],
                    nesterov=case["nesterov"], **MUON)
    return {"w": s["w"], "mom": s["mom"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work --

def _held_bytes(rows, cols):
    return rows * cols * (0.5 + 1.0 / BLOCK)


def _steps_flops(m, n):
    """Products of the steps, the symmetric ones' upper halves alone."""
    m, n = min(m, n), max(m, n)
    return STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2.0 * m * m * n)


def work(case):
    op = case["op"]
    if op == "quantize":
        n, size = case["rows"] * case["cols"], 4 if case["type"] == "f32" else 2
        ways = 2 if case["axis"] == "both" else 1
        # x once, each form written and read back, the values written
        return {"bytes": n * size + ways * (2 * _held_bytes(case["rows"], case["cols"]) + n * size), "flops": 4.0 * n * ways}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        out = M * N * ((4 if case["out"] == "f32" else 2) + (4 if case["beta"] else 0))
        return {"bytes": _held_bytes(M, K) + _held_bytes(N, K) + out, "flops": 2.0 * M * N * K}
    if op == "linear":
        T, N, K, size = case["T"], case["N"], case["K"], 4 if case["type"] == "f32" else 2
        w = _held_bytes(N, K)
        if not case["train"]:
            return {"bytes": w + size * (T * K + T * N), "flops": 2.0 * T * N * K}
        return {"bytes": 2 * w + size * (2 * T * K + 2 * T * N + N * K) + 2 * _held_bytes(T, K), "flops": 6.0 * T * N * K}
    m, n, size = case["m"], case["n"], 4 if case["type"] == "f32" else 2
    one = m * n * (size + 2)                      # the gradient, and the result or the weights
    if op == "muon":
        one += m * n * (2 + 8)                    # the weights read, the momentum read and written
    return {"bytes": case["count"] * one, "flops": case["count"] * _steps_flops(m, n)}


# ------------------------------------------------------------------ exact --

def _held64(x):
    """MXFP4 along the rows of x from its definition, in FP64: quanta of half a
    step below 2, one below 4 and two above, in units of the block's scale."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % BLOCK)).unflatten(1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -149))) - 2).clamp(-127, 127))
    r = v / unit
    step = torch.where(r.abs() >= 4, 2.0, torch.where(r.abs() >= 2, 1.0, 0.5)).double()
    return ((r / step).round() * step).clamp(-6, 6).mul(unit).flatten(1)[:, :cols]


def _decode64(q, cols):
    code, byte = (t.permute(1, 0, 2) for t in q)
    nib = torch.cat(((code & 15)[..., None], (code >> 4)[..., None]), -1).flatten(2).to(torch.float64)
    sign, mag = torch.where(nib >= 8, -1.0, 1.0).double(), nib % 8
    # code 2e + m is (1 + m / 2) 2^(e - 1), and m / 2 where e is 0
    e, m = torch.div(mag, 2, rounding_mode="floor"), mag % 2
    val = sign * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    val = val.unflatten(2, (8, 32)) * torch.exp2(byte.double() - 127)[..., None]
    return val.flatten(1)[:, :cols]


def _polar64(u):
    flip = u.shape[0] > u.shape[1]
    x = u.double().t() if flip else u.double()
    x = x / (torch.linalg.matrix_norm(x) + 1e-7)
    a, b, c = QUINTIC
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        s = x @ x.mT
        x = (a * eye + s @ (b * eye + c * s)) @ x
    return x.mT if flip else x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        if case["rows"] * case["cols"] > 1 << 28:
            return None
        both = case["axis"] == "both"
        along = _held64(s["x"]) if both or case["axis"] == "rows" else None
        down = _held64(s["x"].t()).t() if both or case["axis"] == "cols" else None
        return [v for v in (along, down) if v is not None]
    if op == "product":
        y = _decode64(s["p"], case["K"]) @ _decode64(s["q"], case["K"]).mT
        return y + case["beta"] * s["addend"].double() if case["beta"] else y
    if op == "linear":
        y = _held64(s["x"]) @ _decode64(s["w"], case["K"]).mT
        if not case["train"]:
            return y
        return {"y": y, "dx": _held64(s["dy"]) @ _decode64(s["wt"], case["N"]).mT,
                "dw": _held64(s["dy"].t()) @ _held64(s["x"].t()).mT}
    if op == "orthogonalize":
        return [_polar64(g) for g in s["g"]]
    mu, lr, wd = (float(torch.tensor(MUON[k], dtype=torch.float32)) for k in ("momentum", "lr", "weight_decay"))
    ws, moms = [], []
    for g, mom, w in zip(s["g"], s["mom"], s["w"]):
        new = mu * mom.double() + g.double()
        u = g.double() + mu * new if case["nesterov"] else new
        ws.append((1 - lr * wd) * w.double() - lr * _muon_scale(*w.shape) * _polar64(u))
        moms.append(new)
    return {"w": ws, "mom": moms}
