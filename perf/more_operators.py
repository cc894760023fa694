"""The feed-forward half of a decoder layer around this library's products, as cases to measure
and compare.

Three operators, row-major (rows are tokens):

norm    s = x + residual; out = s * rsqrt(mean(s^2) + eps) * weight, with s kept for the residual
        stream; in 8 bits, out / scale as E4M3 with a scale per row, max |out| / 448 (2^-100 at
        least).  Its backward pass gives dx (with the gradient that arrives at s added) and dw.
gated   [g | u] = x w^T, out = act(g) * u, optionally with [g | u] kept; its backward pass gives
        dx and dw from dout and [g | u].
w4      x w^T with weights of 4 bits, w = (q - zero) * scale per group of features: a linear layer
        with bias and residual, or gated projections.  Two elements a byte, the first one low.

``own`` False computes the plain form: elementary torch operations in FP32, rounded once at
the end.  ``own`` True calls the library.  Inputs and outputs are the same.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_ACTS = ("relu", "gelu", "gelu_tanh", "silu")
_EPS = 1e-5


# ------------------------------------------------------------------------------ cases
def _norm(name, way, t, k, dtype="bf16", residual=True):
    return {"name": name, "op": "norm", "pass": way, "t": t, "k": k, "dtype": dtype,
            "residual": residual}


def _gated(name, way, t, n, k, act="silu", dtype="bf16", save_z=False):
    return {"name": name, "op": "gated", "pass": way, "t": t, "n": n, "k": k, "act": act,
            "dtype": dtype, "save_z": save_z}


def _w4(name, t, n, k, group, zeros=False, gated=False, dtype="bf16"):
    return {"name": name, "op": "w4", "pass": "forward", "t": t, "n": n, "k": k, "group": group,
            "zeros": zeros, "gated": gated, "dtype": dtype}


def listed():
    return [
        # The norm in front of a decoding step's projections: one row, latency alone.
        _norm("norm 1 token", "forward", 1, 4096),
        # A prompt of odd length and width for 8-bit projections, FP16, no residual yet.
        _norm("norm 777 tokens f16 8 bit", "8bit", 777, 2055, "f16", residual=False),
        # A training batch's norm with the residual stream, 8-bit output for FP8 products.
        _norm("norm 16384 tokens 8 bit", "8bit", 16384, 4096),
        # Its backward pass, the residual stream's gradient added.
        _norm("norm backward 16384", "backward", 16384, 4096),
        # Gated projections of a decoding step: bound by the weights' bytes.
        _gated("gated 1 token", "forward", 1, 8192, 4096),
        # A small decoding batch in FP16, features no multiple of a tile.
        _gated("gated 23 tokens f16", "forward", 23, 1000, 2056, "gelu", "f16"),
        # The training forward pass, pre-activations kept.
        _gated("gated 16384 tokens", "forward", 16384, 4096, 4096, save_z=True),
        # Its backward pass: dx and dw.
        _gated("gated backward 16384", "backward", 16384, 4096, 4096),
        # A down projection of a decoding step from 4-bit weights.
        _w4("w4 1 token", 1, 4096, 16384, 128),
        # A small decoding batch, small groups with zero points of their own.
        _w4("w4 8 tokens zeros", 8, 4096, 4096, 32, zeros=True),
        # Gated projections of a decoding step from 4-bit weights, FP16.
        _w4("w4 gated 3 tokens f16", 3, 8192, 4096, 64, gated=True, dtype="f16"),
        # A prompt of odd length on the same weights.
        _w4("w4 333 tokens", 333, 4096, 4096, 128),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "gated", "w4", "w4"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "norm":
        case = _norm("", rng.choice(("forward", "8bit", "backward")), _log_int(rng, 1, 16384),
                     _log_int(rng, 64, 4096), dtype, rng.random() < 0.7)
    elif op == "gated":
        t, n, k = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 512), 8 * _log_int(rng, 16, 512)
        case = _gated("", rng.choice(("forward", "backward")), t, n, k, rng.choice(_ACTS), dtype,
                      rng.random() < 0.5)
    else:
        gated = rng.random() < 0.3
        case = _w4("", _log_int(rng, 1, 512), _log_int(rng, 128, 8192), 8 * _log_int(rng, 16, 2048),
                   rng.choice((32, 64, 128)), rng.random() < 0.4, gated, dtype)
    del case["name"]
    return case


def work(case):
    t, k = case["t"], case["k"]
    if case["op"] == "norm":
        # x, (residual), weight in; out, (s) out; backward: dout, s, (ds) in, dx and dw out
        planes = 4 if case["residual"] else 2
        if case["pass"] == "backward":
            return {"bytes": 2.0 * t * k * (planes if case["residual"] else 3) + 6.0 * k,
                    "flops": 10.0 * t * k}
        moved = 2.0 * t * k * planes + 2.0 * k
        if case["pass"] == "8bit":
            moved += 4.0 * t - t * k
        return {"bytes": moved, "flops": 5.0 * t * k}
    n = case["n"]
    if case["op"] == "gated":
        product = 4.0 * t * n * k
        if case["pass"] == "forward":
            moved = t * k + 2 * n * k + t * n * (3 if case["save_z"] else 1)
            return {"bytes": 2.0 * moved, "flops": product}
        return {"bytes": 2.0 * (2 * t * k + 4 * n * k + 3 * t * n), "flops": 2 * product}
    rows = 2 * n if case["gated"] else n
    groups = -(-k // case["group"])
    moved = 0.5 * rows * k + rows * groups * (4 if case["zeros"] else 2) + 2.0 * t * (k + n)
    if not case["gated"]:
        moved += 2.0 * n + 2.0 * t * n                       # bias and residual
    return {"bytes": moved, "flops": 2.0 * t * rows * k}


# -------------------------------------------------------------------------- preparation
def prepare(case, seed):
    dev, dtype = torch.device("cuda"), _DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        """Rows a multiple of 16 bytes apart, whatever the number of columns."""
        cols = shape[-1]
        a = (torch.randn(*shape[:-1], (cols + 7) // 8 * 8, generator=gen, device=dev) * std + mean).to(dtype)
        return a[..., :cols]

    t, k = case["t"], case["k"]
    s = {"case": case, "x": normal(t, k)}
    if case["op"] == "norm":
        # hidden states: a few features far larger than the others
        loud = torch.where(torch.rand(k, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        s["x"].mul_(loud.to(dtype))
        s["weight"] = normal(k, std=0.2, mean=1.0)
        s["residual"] = normal(t, k) if case["residual"] else None
        if case["pass"] == "backward":
            s["dout"] = normal(t, k, std=0.1)
        elif case["residual"]:
            s["sum"] = torch.empty_like(s["x"])              # the residual stream
        return s
    n = case["n"]
    if case["op"] == "gated":
        s["w"] = normal(2 * n, k, std=1.0 / math.sqrt(k))
        if case["pass"] == "backward":
            s["z"] = normal(t, 2 * n)
            s["dout"] = normal(t, n)
        elif case["save_z"]:
            s["z"] = normal(t, 2 * n, std=0.0)
        return s
    rows = 2 * n if case["gated"] else n
    size, half = (rows, -(-k // case["group"])), (k + 1) // 2
    q = (torch.randn(rows, k + k % 2, generator=gen, device=dev) * 2.7 + 8.0).round().clamp(0, 15)
    q = q.to(torch.uint8)
    packed = torch.zeros(rows, (half + 15) // 16 * 16, dtype=torch.uint8, device=dev)
    packed[:, :half] = q[:, 0::2] | (q[:, 1::2] << 4)
    s["w"] = packed[:, :half]
    s["scales"] = ((0.5 + torch.rand(size, generator=gen, device=dev)) / (2.7 * math.sqrt(k))).to(dtype)
    s["zeros"] = None
    if case["zeros"]:
        s["zeros"] = (7.5 + torch.randn(size, generator=gen, device=dev)).to(dtype)
    if not case["gated"]:
        s["bias"] = normal(n, std=0.2)
        s["residual"] = normal(t, n)
    return s


# ---------------------------------------------------------------------------- plain form
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_norm(s, c):
    x, weight, dtype = s["x"].float(), s["weight"].float(), s["x"].dtype
    if c["pass"] == "backward":
        r = torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS)
        dout = s["dout"].float()
        g = dout * weight
        dx = r * (g - x * r * r * (g * x).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return {"dx": dx.to(dtype), "dw": (dout * x * r).sum(0)}
    res = {}
    if s["residual"] is not None:
        x = x + s["residual"].float()
        res["sum"] = x.to(dtype)
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS) * weight
    if c["pass"] == "forward":
        return {**res, "out": y.to(dtype)}
    scale = (y.abs().amax(1) / 448.0).clamp(min=2.0 ** -100)
    return {**res, "out": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}


def _plain_gated(s, c):
    n, dtype, w = c["n"], s["x"].dtype, s["w"].float()
    if c["pass"] == "forward":
        z = s["x"].float() @ w.t()
        out = (_act(z[:, :n], c["act"]) * z[:, n:]).to(dtype)
        return {"out": out, **({"z": z.to(dtype)} if c["save_z"] else {})}
    g, u, dout = s["z"][:, :n].float(), s["z"][:, n:].float(), s["dout"].float()
    dz = torch.cat((dout * u * _act_slope(g, c["act"]), dout * _act(g, c["act"])), 1)
    return {"dx": (dz @ w).to(dtype), "dw": (dz.t() @ s["x"].float()).to(dtype)}


def _plain_w4(s, c):
    n, k, dtype = c["n"], c["k"], s["x"].dtype
    q = torch.stack((s["w"] & 15, s["w"] >> 4), 2).flatten(1)[:, :k].float()
    group = torch.arange(k, device=q.device) // c["group"]
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, group]
    z = s["x"].float() @ ((q - zero) * s["scales"].float()[:, group]).t()
    if c["gated"]:
        return {"out": (_act(z[:, :n], "silu") * z[:, n:]).to(dtype)}
    return {"out": (z + s["bias"].float() + s["residual"].float()).to(dtype)}


# ------------------------------------------------------------------------------ one pass
_handles = {}


def _handle():
    import mixed_precision_tensor_gb300 as tcg
    device = torch.cuda.current_device()
    if device not in _handles:
        _handles[device] = tcg.Handle()
    return tcg, _handles[device]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "gated": _plain_gated, "w4": _plain_w4}[c["op"]](s, c)
    tcg, h = _handle()
    if c["op"] == "norm":
        if c["pass"] == "backward":
            dx, dw = tcg.rms_norm_backward(h, s["dout"], s["x"], s["weight"], eps=_EPS, dsum=s["residual"])
            return {"dx": dx, "dw": dw}
        kept = s.get("sum")
        if kept is not None:  # rows as far apart as those of x, a multiple of 16 bytes
            kept = torch.empty_strided(kept.shape, s["x"].stride(), dtype=kept.dtype, device=kept.device)
        res = {} if kept is None else {"sum": kept}
        if c["pass"] == "forward":
            return {**res, "out": tcg.rms_norm(h, s["x"], s["weight"], eps=_EPS, residual=s["residual"],
                                               sum_out=kept)}
        out, scale = tcg.rms_norm_8bit(h, s["x"], s["weight"], eps=_EPS, residual=s["residual"], sum_out=kept)
        return {**res, "out": out, "scale": scale}
    if c["op"] == "gated":
        if c["pass"] == "backward":
            dx, dw = tcg.gated_linear_backward(h, s["dout"], s["x"], s["w"], s["z"], act=c["act"])
            return {"dx": dx, "dw": dw}
        z = s.get("z")
        out = tcg.gated_linear(h, s["x"], s["w"], act=c["act"], z=z)
        return {"out": out, "z": z} if c["save_z"] else {"out": out}
    if c["gated"]:
        return {"out": tcg.linear_4bit(h, s["x"], s["w"], s["scales"], c["group"], zeros=s["zeros"],
                                       act="silu", gated=True)}
    return {"out": tcg.linear_4bit(h, s["x"], s["w"], s["scales"], c["group"], zeros=s["zeros"],
                                   bias=s["bias"], residual=s["residual"])}


# --------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    """The outputs in FP64, from the definitions; None where that takes too long."""
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    f = {name: a.double() for name, a in s.items()
         if isinstance(a, torch.Tensor) and a.is_floating_point()}
    if case["op"] == "norm":
        return _exact_norm(case, f)
    n, k = case["n"], case["k"]
    if case["op"] == "gated":
        if case["pass"] == "backward":
            with torch.enable_grad():
                z = f["z"].clone().requires_grad_(True)
                dz, = torch.autograd.grad(_exact_act(z[:, :n], case["act"]) * z[:, n:], z, f["dout"])
            return {"dx": torch.einsum("tn,nk->tk", dz, f["w"]), "dw": torch.einsum("tn,tk->nk", dz, f["x"])}
        g, u = (torch.einsum("tk,nk->tn", f["x"], w) for w in (f["w"][:n], f["w"][n:]))
        out = {"out": _exact_act(g, case["act"]) * u}
        return {**out, "z": torch.cat((g, u), 1)} if case["save_z"] else out
    # a group of features at a time: scale times (the product with q less zero times x's sum)
    rows = s["w"].shape[0]
    z = torch.zeros(case["t"], rows, dtype=torch.float64, device=s["w"].device)
    q = torch.zeros(rows, k + k % 2, dtype=torch.float64, device=s["w"].device)
    q[:, 0::2], q[:, 1::2] = (s["w"] % 16).double(), (s["w"] // 16).double()
    for i in range(f["scales"].shape[1]):
        at = slice(i * case["group"], min(k, (i + 1) * case["group"]))
        x = f["x"][:, at]
        zero = f["zeros"][:, i] if case["zeros"] else torch.full_like(z[0], 8.0)
        z += f["scales"][:, i] * (x @ q[:, at].t() - x.sum(1, keepdim=True) * zero)
    if case["gated"]:
        return {"out": _exact_act(z[:, :n], "silu") * z[:, n:]}
    return {"out": z + f["bias"] + f["residual"]}


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z ** 2))
    return z * torch.special.expit(z)


def _exact_norm(case, f):
    x, k = f["x"], case["k"]
    if case["pass"] == "backward":
        with torch.enable_grad():
            xg, wg = x.clone().requires_grad_(True), f["weight"].clone().requires_grad_(True)
            y = xg / torch.sqrt(xg.square().sum(1, keepdim=True) / k + _EPS) * wg
            dx, dw = torch.autograd.grad(y, (xg, wg), f["dout"])
        return {"dx": dx + f["residual"] if case["residual"] else dx, "dw": dw}
    res = {}
    if case["residual"]:
        x = x + f["residual"]
        res["sum"] = x
    y = x / torch.sqrt(x.square().sum(1, keepdim=True) / k + _EPS) * f["weight"]
    if case["pass"] == "forward":
        return {**res, "out": y}
    scale = (torch.linalg.vector_norm(y, float("inf"), dim=1) / 448.0).clamp(min=2.0 ** -100)
    return {**res, "out": y / scale[:, None], "scale": scale}
