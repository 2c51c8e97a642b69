"""Timed cases of a pre-norm feed-forward block over the NF4 base whose saved activations are 8 bits wide.

Operators (the entry points of bit_quantized_lora_blockwise_amd they stand for):

  pack         mx8_quantize + mx8_dequantize: an activation matrix to E4M3 codes with one
               power-of-two scale for each 32 values of a row, and the values that they stand for.
  norm         rms_norm_fwd: S = X + R, Y = S / sqrt(mean(S^2) + eps) * w, and with `save` Y in 8 bits.
  norm_back    rms_norm_bwd: dX = (w dY - n mean(n w dY)) / rms + dS with n = S / rms, dw = sum over rows of n dY.
  swiglu       qlora_swiglu_fwd: [G | U] = X W'^T + s T L2 with T = X L1 for both halves of a stacked gate|up
               projection, H = silu(G) U, and with `save` T and G and U in 8 bits.
  swiglu_back  qlora_swiglu_bwd: from dH, the packed X, G and U and from T the gradients dX, dL1 and dL2.
  linear_back  qlora_linear_bwd_mx8: the gradients of a linear of the same base from its packed input.

Packed layout: codes uint8 [rows, Kp], scales uint8 [rows, Kp / 32], Kp = the row length rounded up to
32, padded with zeros.  Scale byte e stands for 2^(e - 127): the least power of two, 2^-117 at least,
that the block's largest value is at most 448 times of.  G and U are one packed matrix of 2 M rows.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # a few rows of fp32 activations that end inside a block: pure latency
        {"name": "pack ragged fp32", "op": "pack", "rows": 7, "cols": 777, "dtype": "fp32"},
        # the input of the LLaMA-7B down projection, 4096 tokens, kept for the backward
        {"name": "pack 7B down input", "op": "pack", "rows": 4096, "cols": 11008, "dtype": "bf16"},
        # one token between two LLaMA-7B blocks: pure latency
        {"name": "norm one token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True, "save": False},
        # training on LLaMA-65B: the residual's sum, the layers' input and its 8-bit copy
        {"name": "norm 65B, saved", "op": "norm", "rows": 2048, "cols": 8192, "dtype": "bf16", "residual": True, "save": True},
        # a small fp32 model with no round size
        {"name": "norm back ragged fp32", "op": "norm_back", "rows": 333, "cols": 1000, "dtype": "fp32", "residual": False},
        # training on LLaMA-7B
        {"name": "norm back 7B", "op": "norm_back", "rows": 4096, "cols": 4096, "dtype": "bf16", "residual": True},
        # one token through the LLaMA-7B gate and up projections
        {"name": "swiglu 7B, one token", "op": "swiglu", "M": 1, "K": 4096, "F": 11008, "r": 64, "save": False},
        # training through the LLaMA-65B gate and up projections
        {"name": "swiglu 65B, saved", "op": "swiglu", "M": 2048, "K": 8192, "F": 22016, "r": 64, "save": True},
        # a small block with no round size
        {"name": "swiglu back ragged", "op": "swiglu_back", "M": 130, "K": 576, "F": 777, "r": 12},
        # training through the LLaMA-7B gate and up projections
        {"name": "swiglu back 7B", "op": "swiglu_back", "M": 4096, "K": 4096, "F": 11008, "r": 64},
        # a small linear's gradients
        {"name": "linear back ragged", "op": "linear_back", "M": 77, "K": 1088, "N": 333, "r": 5},
        # training through the LLaMA-7B down projection
        {"name": "linear back 7B down", "op": "linear_back", "M": 4096, "K": 11008, "N": 4096, "r": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pack", "norm", "norm_back", "swiglu", "swiglu", "swiglu_back", "linear_back"])
    if op in ("pack", "norm", "norm_back"):
        rows, cols = _log(rng, 1, 16384), _log(rng, 16, 22016)
        while rows * cols > 11008 * 8192:
            rows = max(1, rows // 2)
        case = {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
        if op != "pack":
            case["residual"] = rng.random() < 0.7
        if op == "norm":
            case["save"] = rng.random() < 0.6
        return case
    M, K, r = _log(rng, 1, 4096), 64 * _log(rng, 1, 172), rng.randint(1, 64)
    n = _log(rng, 16, 22016)
    if rng.random() < 0.6:
        n = max(16, n // 16 * 16)
    while M * K * n > 2048 * 8192 * 11008:
        M = max(1, M // 2)
    if op == "linear_back":
        return {"op": op, "M": M, "K": K, "N": n, "r": r}
    case = {"op": op, "M": M, "K": K, "F": n, "r": r}
    if op == "swiglu":
        case["save"] = rng.random() < (0.8 if M > 16 else 0.3)
    return case


# ---- inputs ----------------------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=g.device) * std).to(dtype)


def _activations(g, M, K, dtype=torch.bfloat16):
    """N(0, 1) with a few channels ten times as large, as a residual stream has them, and (among
    many) rows of zeros, as padding has them."""
    x = _normal(g, (M, K), 1.0)
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device=g.device)] *= 10.0
    if M >= 16:
        x[torch.randint(0, M, (max(1, M // 64),), generator=g, device=g.device)] = 0.0
    return x.to(dtype)


def _mx8_pack(x):
    """Codes and scales of the rows of x in the packed layout."""
    value, e = _mx8_round(_blocks(x.float()))
    codes = value.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape[0], -1)
    return codes, (e + 127).to(torch.uint8)


def _nf4_levels():
    """16 levels: equal shares of a normal distribution on each side of an exact zero."""
    d = 1 - (1 / 32 + 1 / 30) / 2
    z = lambda n: torch.special.ndtri(torch.linspace(0.5, d, n, dtype=torch.float64))[1:]  # noqa: E731
    pos, neg = z(9), z(8)
    return (torch.cat([-neg.flip(0), torch.zeros(1, dtype=torch.float64), pos]) / pos[-1]).float()


def _nf4_pack(w):
    """Codes, second-level scale bytes and group scales of the NF4 base."""
    flat = w.float().reshape(-1, 64)
    a = flat.abs().amax(1)
    q = _nf4_levels().to(w.device)
    code = torch.bucketize(flat / a.clamp_min(1e-30)[:, None], (q[1:] + q[:-1]) / 2).to(torch.uint8)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).reshape(w.shape[0], -1)
    nb = a.numel()
    pad = torch.nn.functional.pad(a, (0, -nb % 256)).view(-1, 256)
    c1 = pad.amax(1)
    c2 = (pad / c1[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)[:nb].contiguous()
    return codes, c2, c1


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case)
    dtype = torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16
    if case["op"] in ("pack", "norm", "norm_back"):
        rows, cols = case["rows"], case["cols"]
        s["X"] = _activations(g, rows, cols, dtype)
        if case["op"] == "norm":
            s["w"] = _normal(g, (cols,), 0.2).add_(1.0).to(dtype)
            if case["residual"]:
                s["R"] = _normal(g, (rows, cols), 0.3, dtype)
        if case["op"] == "norm_back":
            s["w"] = _normal(g, (cols,), 0.2).add_(1.0).to(dtype)
            live = (s["X"] != 0).any(1, keepdim=True)                  # padding has no gradient
            s["dY"] = torch.where(live, _normal(g, (rows, cols), 0.01), 0.0).to(torch.bfloat16)
            if case["residual"]:
                s["dS"] = _normal(g, (rows, cols), 0.01, dtype)
        return s
    M, K, r = case["M"], case["K"], case["r"]
    n, halves = (case["N"], 1) if case["op"] == "linear_back" else (case["F"], 2)
    s["codes"], s["c2"], s["c1"] = _nf4_pack(_normal(g, (halves * n, K), 0.02, torch.bfloat16))
    s["levels"] = _nf4_levels().to(dev)
    s["scale"] = 2.0
    s["L1"] = _normal(g, (halves, K, r), K ** -0.5, torch.bfloat16)
    s["L2"] = _normal(g, (halves, r, n), 0.01, torch.bfloat16)
    X = _activations(g, M, K)
    if case["op"] == "swiglu":
        s["X"] = X
        return s
    s["x8"] = _mx8_pack(X)
    # what the forward left for the backward
    s["T"] = torch.stack([X.float() @ s["L1"][h].float() for h in range(halves)]).to(torch.bfloat16)
    if case["op"] == "swiglu_back":
        s["gu8"] = _mx8_pack(_normal(g, (2 * M, n), 1.3))
        s["dH"] = _normal(g, (M, n), 0.01, torch.bfloat16)
    else:
        s["dY"] = _normal(g, (M, n), 0.01, torch.bfloat16)
        s["L1"], s["L2"], s["T"] = s["L1"][0], s["L2"][0], s["T"][0]
    return s


# ---- the plain forms -------------------------------------------------------------------

def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 32)).view(x.shape[0], -1, 32)


def _mx8_round(blocks):
    """Blocks [..., 32] to their E4M3 values (over the block's scale) and the scale's exponent."""
    mant, exp = torch.frexp(blocks.abs().amax(-1))                     # 448 = 0.875 * 2^9
    e = torch.where(mant > 0, exp - 9 + (mant > 0.875).int(), torch.full_like(exp, -117)).clamp_min(-117)
    v = torch.ldexp(blocks, -e.unsqueeze(-1))
    step = torch.ldexp(torch.full_like(v, 0.125), (torch.frexp(v)[1] - 1).clamp_min(-6))
    return torch.round(v / step) * step, e


def _mx8_values(x):
    """The values that the rows of x stand for once packed."""
    value, e = _mx8_round(_blocks(x))
    return torch.ldexp(value, e.unsqueeze(-1)).view(x.shape[0], -1)[:, :x.shape[1]]


def _mx8_unpack(packed, cols):
    codes, scales = packed
    v = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int().unsqueeze(-1) - 127).view(codes.shape[0], -1)[:, :cols]


def _base(s):
    """fp32 values of the base's bf16 weights."""
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(-1, 64)
    sb = s["c2"].view(torch.float8_e4m3fn).float() * s["c1"].repeat_interleave(256)[:s["c2"].numel()]
    return (s["levels"][code.int()] * sb[:, None]).to(torch.bfloat16).float().view(-1, s["K"])


def _plain_rows(s):
    X = s["X"].float()
    if s["op"] == "pack":
        return _mx8_values(X).to(torch.bfloat16)
    w = s["w"].float()
    if s["op"] == "norm":
        out = {}
        if s["residual"]:
            out["S"] = (X + s["R"].float()).to(s["X"].dtype)
            X = out["S"].float()
        Y = X * torch.rsqrt((X * X).mean(1, keepdim=True) + EPS) * w
        out["Y"] = Y.to(torch.bfloat16)
        if s["save"]:
            out["Y8"] = _mx8_values(Y).to(torch.bfloat16)
        return out
    dY = s["dY"].float()
    inv = torch.rsqrt((X * X).mean(1, keepdim=True) + EPS)
    n, d = X * inv, dY * w
    dX = inv * (d - n * (n * d).mean(1, keepdim=True))
    if s["residual"]:
        dX = dX + s["dS"].float()
    return {"dX": dX.to(s["X"].dtype), "dw": (n * dY).sum(0)}


def _plain(s):
    if s["op"] in ("pack", "norm", "norm_back"):
        return _plain_rows(s)
    L1, L2, c, W = s["L1"].float(), s["L2"].float(), s["scale"], _base(s)
    if s["op"] == "swiglu":
        X = s["X"].float()
        T = X @ L1
        Z = X @ W.t() + c * (T @ L2).transpose(0, 1).reshape(s["M"], -1)
        G, U = Z[:, :s["F"]], Z[:, s["F"]:]
        H = (G / (1 + torch.exp(-G)) * U).to(torch.bfloat16)
        if not s["save"]:
            return {"H": H}
        return {"H": H, "T": T.to(torch.bfloat16), "GU": _mx8_values(torch.cat([G, U])).to(torch.bfloat16)}
    X, T = _mx8_unpack(s["x8"], s["K"]), s["T"].float()
    if s["op"] == "linear_back":
        dY = s["dY"].float()
        G = c * (dY @ L2.t())
        return {"dX": (dY @ W + G @ L1.t()).to(torch.bfloat16), "dL1": X.t() @ G, "dL2": c * (T.t() @ dY)}
    gate, up = _mx8_unpack(s["gu8"], s["F"]).view(2, s["M"], -1)
    dH = s["dH"].float()
    sig = 1 / (1 + torch.exp(-gate))
    dZ = torch.stack([dH * up * sig * (1 + gate * (1 - sig)), dH * gate * sig])
    G = c * (dZ @ L2.transpose(1, 2).contiguous())
    dX = dZ[0] @ W[:s["F"]] + dZ[1] @ W[s["F"]:] + G[0] @ L1[0].t() + G[1] @ L1[1].t()
    return {"dX": dX.to(torch.bfloat16), "dL1": X.t() @ G, "dL2": c * (T.transpose(1, 2).contiguous() @ dZ)}


# ---- one pass --------------------------------------------------------------------------

def run(s):
    if not own:
        return _plain(s)
    import bit_quantized_lora_blockwise_amd as q
    if s["op"] == "pack":
        return q.mx8_dequantize(*q.mx8_quantize(s["X"]), *s["X"].shape)
    if s["op"] == "norm":
        Y, S, y8 = q.rms_norm_fwd(s["X"], s["w"], EPS, residual=s.get("R"), mx8=s["save"])
        out = {"Y": Y}
        if s["residual"]:
            out["S"] = S
        if s["save"]:
            out["Y8"] = q.mx8_dequantize(*y8, *Y.shape)
        return out
    if s["op"] == "norm_back":
        dX, dw = q.rms_norm_bwd(s["dY"], s["X"], s["w"], EPS, dS=s.get("dS"))
        return {"dX": dX, "dw": dw}
    base = (s["codes"], s["c2"], s["c1"])
    if s["op"] == "swiglu":
        H, T, gu8 = q.qlora_swiglu_fwd(s["X"], *base, s["F"], s["L1"], s["L2"], s["scale"], T_out=s["save"],
                                       mx8=s["save"])
        if not s["save"]:
            return {"H": H}
        return {"H": H, "T": T, "GU": q.mx8_dequantize(*gu8, 2 * s["M"], s["F"])}
    if s["op"] == "swiglu_back":
        dX, dL1, dL2 = q.qlora_swiglu_bwd(s["x8"], s["dH"], *base, s["L1"], s["L2"], s["gu8"], s["T"], s["scale"])
    else:
        dX, dL1, dL2 = q.qlora_linear_bwd_mx8(s["x8"], s["dY"], *base, s["L1"], s["L2"], s["T"], s["scale"])
    return {"dX": dX, "dL1": dL1, "dL2": dL2}


def work(case):
    op = case["op"]
    if op in ("pack", "norm", "norm_back"):
        n, b = case["rows"] * case["cols"], 4 if case["dtype"] == "fp32" else 2
        packed = n * 33 / 32
        if op == "pack":
            return {"bytes": b * n + packed + 2 * n, "flops": 2 * n}   # read, packed, values
        if op == "norm":                                               # X (R, S), Y (packed, values)
            return {"bytes": b * n * (3 if case["residual"] else 1) + 2 * n + (packed + 2 * n if case["save"] else 0),
                    "flops": 4 * n}
        return {"bytes": b * n * (3 if case["residual"] else 2) + 2 * n, "flops": 9 * n}
    M, K, r = case["M"], case["K"], case["r"]
    n, halves = (case["N"], 1) if op == "linear_back" else (case["F"], 2)
    nf4 = halves * n * K * (0.5 + 1 / 64 + 4 / 16384)
    adapters, t = 2 * halves * r * (K + n), 2 * halves * M * r
    gemm, low = 2 * halves * M * K * n, 2 * halves * M * r * (K + n)
    if op == "swiglu":
        out = 2 * M * n + (t + 2 * M * n * 33 / 32 + 4 * M * n if case["save"] else 0)     # H (T, packed, values)
        return {"bytes": 2 * M * K + nf4 + adapters + out, "flops": gemm + low}
    back = M * K * 33 / 32 + 2 * M * K + nf4 + 3 * adapters + t        # X, dX, base, adapters and their fp32 gradients, T
    return {"bytes": back + 2 * M * n + (2 * M * n * 33 / 32 if halves == 2 else 0), "flops": gemm + 2 * low}


# ---- the definitions in 64 bits --------------------------------------------------------

def _exact_mx8(x):
    """Nearest E4M3 values over a scale found by trying, ties to the even code."""
    rows, cols = x.shape
    b = torch.cat([x.double(), torch.zeros(rows, -cols % 32, dtype=torch.float64, device=x.device)], 1).view(rows, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)) - 1
    for _ in range(3):
        e = e + (448 * torch.exp2(e) < top).double()
    scale = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -117.0)).clamp_min(-117.0))
    v = b.abs() / scale
    lead = torch.full_like(v, 2.0 ** -6)                               # the power of two that leads each value
    for k in range(-5, 9):
        lead = torch.where(v >= 2.0 ** k, torch.full_like(v, 2.0 ** k), lead)
    units = v / lead * 8
    low = torch.floor(units)
    up = (units - low > 0.5) | ((units - low == 0.5) & (low % 2 == 1))
    return ((low + up.double()) / 8 * lead * scale * torch.sign(b)).view(rows, -1)[:, :cols]


def _exact_unpack(packed, cols):
    codes, scales = packed[0].long(), packed[1].double()
    mag, sign = codes % 128, 1 - 2 * (codes // 128).double()
    val = torch.where(mag < 8, mag / 512, torch.exp2((mag // 8).double() - 7) * (1 + (mag % 8) / 8)).double()
    return (sign * val * torch.exp2(scales - 127).repeat_interleave(32, 1))[:, :cols]


def _exact_base(s):
    byte = s["c2"].long()
    dec = torch.where(byte < 8, byte / 512, torch.exp2((byte // 8).double() - 7) * (1 + (byte % 8) / 8)).double()
    group = torch.arange(byte.numel(), device=byte.device) // 256
    sb = (dec * s["c1"].double()[group]).float()                    # the base's own definition rounds twice: here
    nib = torch.stack((s["codes"] % 16, s["codes"] // 16), 2).flatten()
    return (s["levels"][nib.long()].view(-1, 64) * sb[:, None]).bfloat16().double().view(-1, s["K"])    # and here


def _exact_rows(s):
    X = s["X"].double()
    if s["op"] == "pack":
        return _exact_mx8(X)
    w = s["w"].double()
    if s["op"] == "norm":
        out = {}
        if s["residual"]:
            out["S"] = X + s["R"].double()
            X = out["S"].to(s["X"].dtype).double()                     # the norm is that of the sum as it is kept
        Y = X / torch.sqrt(X.square().mean(1, keepdim=True) + EPS) * w
        return {**out, "Y": Y, **({"Y8": _exact_mx8(Y)} if s["save"] else {})}
    dY = s["dY"].double()
    rms = torch.sqrt(X.square().mean(1, keepdim=True) + EPS)
    dX = w * dY / rms - X * (X * w * dY).mean(1, keepdim=True) / rms ** 3
    if s["residual"]:
        dX = dX + s["dS"].double()
    return {"dX": dX, "dw": (X / rms * dY).sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("pack", "norm", "norm_back"):
        return _exact_rows(s)
    L1, L2, c, W = s["L1"].double(), s["L2"].double(), s["scale"], _exact_base(s)
    if case["op"] == "swiglu":
        X, F = s["X"].double(), case["F"]
        T = [X @ L1[0], X @ L1[1]]
        G = X @ W[:F].t() + c * T[0] @ L2[0]
        U = X @ W[F:].t() + c * T[1] @ L2[1]
        H = G * torch.sigmoid(G) * U
        if not case["save"]:
            return {"H": H}
        return {"H": H, "T": torch.stack(T), "GU": _exact_mx8(torch.cat((G, U)))}
    X, T = _exact_unpack(s["x8"], case["K"]), s["T"].double()
    if case["op"] == "linear_back":
        dY = s["dY"].double()
        return {"dX": dY @ W + c * dY @ L2.t() @ L1.t(), "dL1": c * X.t() @ (dY @ L2.t()), "dL2": c * T.t() @ dY}
    M, F = case["M"], case["F"]
    gu = _exact_unpack(s["gu8"], F)
    G, U, dH = gu[:M], gu[M:], s["dH"].double()
    sig = torch.sigmoid(G)
    dG, dU = dH * U * (sig + G * sig * (1 - sig)), dH * G * sig
    back = [c * dG @ L2[0].t(), c * dU @ L2[1].t()]
    return {"dX": dG @ W[:F] + dU @ W[F:] + back[0] @ L1[0].t() + back[1] @ L1[1].t(),
            "dL1": torch.stack([X.t() @ b for b in back]), "dL2": c * torch.stack([T[0].t() @ dG, T[1].t() @ dU])}
