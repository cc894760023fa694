"""The language-model products of this library, as cases to measure and compare.

Three operators, row-major (rows are tokens):

linear          out = act(x w^T + bias) + residual, optionally with the pre-activation z; its
                backward pass gives dx, dw and dbias from dout and z.
grouped_linear  the same with rows sorted by expert: rows offsets[e] .. offsets[e + 1] - 1 meet
                the weights w[e]; rows that no expert takes come out zero.  Its backward pass
                gives dx, dw (one matrix per expert, zero for an expert without rows) and dbias.
xent            the softmax cross entropy of the logits x w^T without keeping the logits: each
                row's loss and log-sum-exp, and in training dx and dw for the rows' upstream
                gradients.  Rows whose target is negative are ignored: loss and gradient zero.

``own`` False computes the plain form: elementary torch operations in FP32, rounded once at
the end.  ``own`` True calls the library.  Inputs and outputs are the same.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------------------ cases
def _linear(name, t, n, k, act, dtype="bf16", residual=False, save_z=False):
    return {"name": name, "op": "linear", "pass": "forward", "t": t, "n": n, "k": k, "act": act,
            "dtype": dtype, "residual": residual, "save_z": save_z}


def _linear_backward(name, t, n, k, act, dtype="bf16"):
    return {"name": name, "op": "linear", "pass": "backward", "t": t, "n": n, "k": k, "act": act,
            "dtype": dtype}


def _grouped(name, way, t, e, n, k, act, spread, dtype="bf16", spare=0):
    return {"name": name, "op": "grouped", "pass": way, "t": t, "e": e, "n": n, "k": k, "act": act,
            "spread": spread, "spare": spare, "dtype": dtype}


def _xent(name, way, t, v, k, dtype="bf16"):
    return {"name": name, "op": "xent", "pass": way, "t": t, "v": v, "k": k, "dtype": dtype}


def listed():
    return [
        # One token through a projection: a decoding step's latency, bound by the weights' bytes.
        _linear("linear 1 token", 1, 4096, 4096, "silu"),
        # A small decoding batch through a down projection with the residual stream added.
        _linear("linear 23 tokens", 23, 4096, 16384, "none", residual=True),
        # A prompt of odd length in FP16, features no multiple of a tile.
        _linear("linear 777 tokens f16", 777, 1000, 2056, "relu", "f16", residual=True),
        # The training forward pass of a projection with GELU, pre-activation kept.
        _linear("linear 16384 tokens", 16384, 4096, 4096, "gelu", save_z=True),
        # Its backward pass: dx, dw, dbias.
        _linear_backward("linear backward 16384", 16384, 4096, 4096, "gelu_tanh"),
        # A decoding step through experts: a few rows, most experts without any.
        _grouped("grouped 8 rows of 64", "forward", 8, 64, 2048, 4096, "none", 1.0),
        # A short prompt, ragged and partly idle experts, odd features, rows to spare, FP16.
        _grouped("grouped 397 rows f16", "forward", 397, 16, 520, 1032, "gelu", 1.5, "f16", 20),
        # The training forward pass of an expert layer with a skewed router.
        _grouped("grouped 16384 rows", "forward", 16384, 64, 2048, 4096, "silu", 1.0),
        # The backward pass of an expert layer: dx, dw per expert, dbias per expert.
        _grouped("grouped backward 16384", "backward", 16384, 32, 2048, 2048, "silu", 1.0),
        # Scoring one token against a vocabulary: bound by the head's bytes.
        _xent("xent 1 token", "forward", 1, 32003, 4096),
        # A small fine-tuning step in FP16 with an odd vocabulary.
        _xent("xent 1000 tokens f16", "training", 1000, 50021, 1024, "f16"),
        # A training step's head: loss, dx and dw over a large vocabulary.
        _xent("xent 4096 tokens", "training", 4096, 100000, 4096),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "grouped", "grouped", "xent"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    act = rng.choice(_ACTS)
    if op == "linear":
        t, n, k = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 1024), 8 * _log_int(rng, 16, 1024)
        if rng.random() < 0.5:
            case = _linear("", t, n, k, act, dtype, rng.random() < 0.5, rng.random() < 0.5)
        else:
            case = _linear_backward("", t, n, k, act, dtype)
    elif op == "grouped":
        way = rng.choice(("forward", "backward"))
        t, e = _log_int(rng, 1, 16384), _log_int(rng, 2, 64)
        n, k = 8 * _log_int(rng, 16, 512), 8 * _log_int(rng, 16, 512)
        if way == "backward":  # dw is as large as all experts' weights
            e = min(e, 32)
        case = _grouped("", way, t, e, n, k, act, round(rng.uniform(0.0, 1.5), 2), dtype,
                        rng.choice((0, 0, rng.randrange(1, 40))))
    else:
        way = rng.choice(("forward", "training"))
        t, v, k = _log_int(rng, 1, 4096), _log_int(rng, 1000, 100000), 8 * _log_int(rng, 16, 512)
        case = _xent("", way, t, v, k, dtype)
    del case["name"]
    return case


def work(case):
    t, k = case["t"], case["k"]
    if case["op"] == "xent":
        v = case["v"]
        product = 2.0 * t * v * k
        if case["pass"] == "forward":
            return {"bytes": 2.0 * (t * k + v * k) + 16.0 * t, "flops": product}
        # the logits, dx and dw: three products, whatever a form without the logits adds
        return {"bytes": 4.0 * (t * k + v * k) + 20.0 * t, "flops": 3 * product}
    n, gs = case["n"], case["op"] == "grouped"
    used = sum(1 for s in _sizes(case, 1) if s) if gs else 1
    groups = case["e"] if gs else 1
    product = 2.0 * t * n * k
    rows = t + case.get("spare", 0)
    if case["pass"] == "forward":
        moved = t * k + used * n * (k + 1) + rows * n
        moved += t * n if case.get("residual") else 0
        moved += rows * n if case.get("save_z") else 0
        return {"bytes": 2.0 * moved, "flops": product}
    # x, dout, z and the used weights in; dx, dw and dbias (FP32) out
    moved = t * k + 2 * t * n + used * n * k + rows * k + groups * n * k
    return {"bytes": 2.0 * moved + 4.0 * groups * n, "flops": 2 * product}


def _sizes(case, seed):
    """Rows of each expert: shares exp(spread * normal), drawn row by row."""
    r = random.Random(1000003 * seed + 7)
    e = case["e"]
    share = [math.exp(case["spread"] * r.gauss(0.0, 1.0)) for _ in range(e)]
    sizes = [0] * e
    for i in r.choices(range(e), weights=share, k=case["t"]):
        sizes[i] += 1
    return sizes


# -------------------------------------------------------------------------- preparation
def prepare(case, seed):
    dev, dtype = torch.device("cuda"), _DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=dtype):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    t, k = case["t"], case["k"]
    s = {"case": case}
    if case["op"] == "xent":
        v = case["v"]
        s["x"] = normal(t, k)
        s["w"] = normal(v, k, std=1.5 / math.sqrt(k))       # logits of deviation 1.5
        target = torch.randint(0, v, (t,), generator=gen, device=dev)
        if t > 1:  # padding: some rows take no part
            drop = torch.rand(t, generator=gen, device=dev) < 0.03
            target = torch.where(drop, torch.full_like(target, -100), target)
        s["target"] = target
        if case["pass"] == "training":  # the mean over the tokens, weighted a little
            s["dloss"] = (1.0 + 0.1 * torch.randn(t, generator=gen, device=dev)) / t
        return s
    n = case["n"]
    if case["op"] == "grouped":
        sizes = _sizes(case, int(seed))
        rows, lead = t + case["spare"], (case["e"],)
        ends = [0]
        for size in sizes:
            ends.append(ends[-1] + size)
        s["offsets"] = torch.tensor(ends, dtype=torch.int64, device=dev)
        s["most"] = max(sizes)
    else:
        rows, lead = t, ()
    s["x"] = normal(rows, k)
    s["w"] = normal(*lead, n, k, std=1.0 / math.sqrt(k))
    if case["pass"] == "forward":
        s["bias"] = normal(*lead, n, std=0.2)
        s["residual"] = normal(rows, n) if case.get("residual") else None
    else:
        s["dout"] = normal(rows, n)
        s["z"] = normal(rows, n) if case["act"] != "none" else None
    return s


# ---------------------------------------------------------------------------- plain form
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


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


def _padded(offsets, most):
    """(row, taken), both (experts, most): the row of each expert's j-th slot, and whether
    there is one."""
    j = torch.arange(most, device=offsets.device)
    row = offsets[:-1, None] + j
    return row, row < offsets[1:, None]


def _plain_linear(s, c):
    dtype = s["x"].dtype
    if c["pass"] == "forward":
        z = s["x"].float() @ s["w"].float().t() + s["bias"].float()
        out = _act(z, c["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return {"out": out.to(dtype), **({"z": z.to(dtype)} if c["save_z"] else {})}
    dz = s["dout"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    return {"dx": (dz @ s["w"].float()).to(dtype), "dw": (dz.t() @ s["x"].float()).to(dtype),
            "dbias": dz.sum(0)}


def _plain_grouped(s, c):
    dtype, rows = s["x"].dtype, s["x"].shape[0]
    row, taken = _padded(s["offsets"], s["most"])
    at = row.clamp(max=rows - 1)

    def gather(a):  # (experts, most, features), zero where an expert has no such row
        return torch.where(taken[..., None], a.float()[at], torch.zeros((), device=a.device))

    def scatter(a):  # back to rows; the ones that no expert takes stay zero
        out = torch.zeros(rows, a.shape[-1], device=a.device)
        out[row[taken]] = a[taken]
        return out

    if c["pass"] == "forward":
        z = torch.bmm(gather(s["x"]), s["w"].float().transpose(1, 2)) + s["bias"].float()[:, None]
        return {"out": scatter(_act(z, c["act"])).to(dtype)}
    dz = gather(s["dout"])
    if c["act"] != "none":
        dz = dz * _act_slope(gather(s["z"]), c["act"])
    return {"dx": scatter(torch.bmm(dz, s["w"].float())).to(dtype),
            "dw": torch.bmm(dz.transpose(1, 2), gather(s["x"])).to(dtype), "dbias": dz.sum(1)}


def _plain_xent(s, c):
    x, w, target = s["x"].float(), s["w"].float(), s["target"]
    logits = x @ w.t()
    top = logits.max(dim=1, keepdim=True).values
    p = torch.exp(logits - top)
    total = p.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    counts = target >= 0
    at = torch.where(counts, target, torch.zeros_like(target))
    here = torch.arange(x.shape[0], device=x.device)
    loss = torch.where(counts, lse - logits[here, at], torch.zeros_like(lse))
    if c["pass"] == "forward":
        return {"loss": loss, "lse": lse}
    del logits
    p /= total
    p[here, at] -= 1.0
    p *= torch.where(counts, s["dloss"], torch.zeros_like(lse))[:, None]
    return {"loss": loss, "lse": lse, "dx": (p @ w).to(s["x"].dtype),
            "dw": (p.t() @ x).to(s["x"].dtype)}


# ------------------------------------------------------------------------------ one pass
_handles = {}


def _handle():
    """The library handle of the current stream, as a program keeps one per stream."""
    import mixed_precision_tensor_gb300 as tcg
    stream = torch.cuda.current_stream()
    if stream.cuda_stream not in _handles:
        _handles[stream.cuda_stream] = tcg.Handle(stream)
    return tcg, _handles[stream.cuda_stream]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"linear": _plain_linear, "grouped": _plain_grouped, "xent": _plain_xent}[c["op"]](s, c)
    tcg, h = _handle()
    if c["op"] == "linear":
        if c["pass"] == "forward":
            z = s["x"].new_empty(c["t"], c["n"]) if c["save_z"] else None
            out = tcg.linear(h, s["x"], s["w"], bias=s["bias"], act=c["act"],
                             residual=s["residual"], z=z)
            return {"out": out, "z": z} if c["save_z"] else {"out": out}
        dx, dw, dbias = tcg.linear_backward(h, s["dout"], s["x"], s["w"], z=s["z"], act=c["act"])
        return {"dx": dx, "dw": dw, "dbias": dbias}
    if c["op"] == "grouped":
        if c["pass"] == "forward":
            return {"out": tcg.grouped_linear(h, s["x"], s["w"], s["offsets"], bias=s["bias"],
                                              act=c["act"])}
        dx, dw, dbias = tcg.grouped_linear_backward(h, s["dout"], s["x"], s["w"], s["offsets"],
                                                    z=s["z"], act=c["act"])
        return {"dx": dx, "dw": dw, "dbias": dbias}
    loss, lse = tcg.linear_cross_entropy(h, s["x"], s["w"], s["target"])
    if c["pass"] == "forward":
        return {"loss": loss, "lse": lse}
    dx, dw = tcg.linear_cross_entropy_backward(h, s["x"], s["w"], s["target"], lse, s["dloss"])
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


# --------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    """The outputs in FP64, from the definitions; None where that takes too long."""
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    f = {name: a.double() for name, a in s.items()
         if isinstance(a, torch.Tensor) and a.is_floating_point()}
    if case["op"] == "xent":
        return _exact_xent(case, s, f)
    n, k, dev = case["n"], case["k"], s["x"].device
    forward = case["pass"] == "forward"
    rows = s["x"].shape[0]
    if case["op"] == "linear":
        spans = [(0, rows)]
        f = {name: a[None] if name in ("w", "bias") else a for name, a in f.items()}
    else:
        ends = s["offsets"].tolist()
        spans = list(zip(ends[:-1], ends[1:]))
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=dev)  # noqa: E731
    out, z_all, dx = zeros(rows, n), zeros(rows, n), zeros(rows, k)
    dw, dbias = zeros(len(spans), n, k), zeros(len(spans), n)
    for e, (a, b) in enumerate(spans):
        if a == b:
            continue
        if forward:
            z = torch.einsum("tk,nk->tn", f["x"][a:b], f["w"][e]) + f["bias"][e]
            z_all[a:b] = z
            out[a:b] = _exact_act(z, case["act"])
            continue
        dz = f["dout"][a:b]
        if case["act"] != "none":
            with torch.enable_grad():
                zg = f["z"][a:b].clone().requires_grad_(True)
                dz, = torch.autograd.grad(_exact_act(zg, case["act"]), zg, dz)
        dx[a:b] = torch.einsum("tn,nk->tk", dz, f["w"][e])
        dw[e] = torch.einsum("tn,tk->nk", dz, f["x"][a:b])
        dbias[e] = dz.sum(0)
    if forward:
        if case.get("residual"):
            out += f["residual"]
        return {"out": out, "z": z_all} if case.get("save_z") else {"out": out}
    if case["op"] == "linear":
        dw, dbias = dw[0], dbias[0]
    return {"dx": dx, "dw": dw, "dbias": dbias}


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z ** 2))
    if act == "silu":
        return z * torch.special.expit(z)
    return z * 1.0


def _exact_xent(case, s, f):
    target, train = s["target"], case["pass"] == "training"
    t, v = case["t"], case["v"]
    loss, lse, dx = [], [], []
    dw = torch.zeros_like(f["w"]) if train else None
    for a in range(0, t, 1024):  # 1024 rows of logits at a time
        b = min(t, a + 1024)
        logits = torch.einsum("tk,vk->tv", f["x"][a:b], f["w"])
        lse.append(torch.logsumexp(logits, dim=1))
        tt = target[a:b]
        hot = (torch.arange(v, device=tt.device)[None] == tt[:, None]).double()
        loss.append(torch.where(tt >= 0, lse[-1] - (logits * hot).sum(1), lse[-1] * 0.0))
        if train:
            g = (torch.softmax(logits, dim=1) - hot) * torch.where(tt >= 0, f["dloss"][a:b],
                                                                   lse[-1] * 0.0)[:, None]
            dx.append(torch.einsum("tv,vk->tk", g, f["w"]))
            dw += torch.einsum("tv,tk->vk", g, f["x"][a:b])
    res = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    return {**res, "dx": torch.cat(dx), "dw": dw} if train else res
