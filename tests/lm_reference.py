"""The language-model products in FP64 torch, from their formulas, and the element-wise
error bounds that the library is held to.  Test code only.

u is the unit roundoff of the 16-bit type (2^-8 BF16, 2^-11 FP16).  A product of K terms is
accumulated within K 2^-23 of the sum of the terms' magnitudes.  exp and erfc carry a
few 2^-22 relative, or 1.5e-7 absolute (the erfc approximation's bound).
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
FN = 1e-6          # activation and its slope, relative to max(1, |z|)


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return (0.5 * torch.special.erfc(-z / math.sqrt(2.0))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def linear(x, w, bias, name, residual, beta, alpha, out_dtype):
    """(out, z, bound of out, bound of z before its rounding)."""
    xd, wd = x.double(), w.double()
    k = x.shape[1]
    z = alpha * (xd @ wd.t()) + (bias.double() if bias is not None else 0.0)
    ez = (k + 4) * 2.0 ** -23 * (abs(alpha) * (xd.abs() @ wd.abs().t())
                                 + (bias.double().abs() if bias is not None else 0.0))
    out = act(z, name)
    e = 1.2 * ez                                 # no slope exceeds 1.13
    if name in ("gelu", "gelu_tanh", "silu"):
        e = e + FN * z.abs().clamp(min=1.0)
    if residual is not None:
        out = out + beta * residual.double()
        e = e + 2.0 ** -23 * (out.abs() + abs(beta) * residual.double().abs())
    e = e + U[out_dtype] * (out.abs() + e) + TINY[out_dtype]
    return out, z, e, ez


def linear_backward(dout, x, w, z, name):
    """((dx, dw, dbias), their bounds)."""
    dtype = x.dtype
    u, tiny = U[dtype], TINY[dtype]
    d, xd, wd = dout.double(), x.double(), w.double()
    t, n = d.shape
    s = slope(z.double(), name) if name != "none" else torch.ones_like(d)
    dz = d * s
    # error of dz before its rounding, and after it
    e0 = d.abs() * FN * (1 + z.double().abs()) if name not in ("none", "relu") else d.abs() * 0.0
    e1 = e0 + (u * (dz.abs() + e0) + tiny if name != "none" else 0.0)
    mag = dz.abs() + e1
    dx, dw, db = dz @ wd, dz.t() @ xd, dz.sum(0)
    ex = e1 @ wd.abs() + (n + 4) * 2.0 ** -23 * (mag @ wd.abs())
    ew = e1.t() @ xd.abs() + (t + 4) * 2.0 ** -23 * (mag.t() @ xd.abs())
    eb = e0.sum(0) + (t + 4) * 2.0 ** -24 * mag.sum(0) + 1e-30
    return (dx, dw, db), (ex + u * (dx.abs() + ex) + tiny, ew + u * (dw.abs() + ew) + tiny, eb)


def xent(x, w, targets, ignore):
    """(loss, lse, their common bound, logits, which rows count)."""
    xd, wd = x.double(), w.double()
    v, k = w.shape
    logits = xd @ wd.t()
    el = (k + 4) * 2.0 ** -23 * (xd.abs() @ wd.abs().t()).max(1).values
    lse = torch.logsumexp(logits, 1)
    counts = (targets != ignore) & (targets >= 0) & (targets < v)
    at = torch.where(counts, targets, torch.zeros_like(targets))
    loss = torch.where(counts, lse - logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    adds = 64 + v / 2048                      # longest chain of additions and rescalings
    bound = 2 * el + (adds + 16) * 2.0 ** -23 + 8 * 2.0 ** -23 * (logits.abs().max(1).values + 1)
    return loss, lse, bound, logits, counts


def xent_backward(x, w, targets, ignore, dloss):
    """((dx, dw), their bounds)."""
    dtype = x.dtype
    u, tiny = U[dtype], TINY[dtype]
    loss, lse, el, logits, counts = xent(x, w, targets, ignore)
    t, v = logits.shape
    p = torch.exp(logits - lse[:, None])
    hot = torch.zeros_like(p)
    rows = counts.nonzero()[:, 0]
    hot[rows, targets[rows]] = 1.0
    g = torch.where(counts, dloss.double(), torch.zeros_like(lse))[:, None]
    G = g * (p - hot)
    eg = g.abs() * (p * (3 * el[:, None] + 1e-6) + hot * 2.0 ** -23)
    eg = eg + u * (G.abs() + eg)
    if dtype == torch.float16:               # held as multiples of 2^-24 / 2^13 of max |dloss|
        eg = eg + g.abs().max() * 2.0 ** -37
    mag = G.abs() + eg
    xd, wd = x.double(), w.double()
    dx, dw = G @ wd, G.t() @ xd
    ex = eg @ wd.abs() + (v + 4) * 2.0 ** -23 * (mag @ wd.abs())
    ew = eg.t() @ xd.abs() + (t + 4) * 2.0 ** -23 * (mag.t() @ xd.abs())
    return (dx, dw), (ex + u * (dx.abs() + ex) + tiny, ew + u * (dw.abs() + ew) + tiny)


def within(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    over = (got - want).abs()[fine] - torch.broadcast_to(bound, want.shape)[fine]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} outside the bound, " \
                           f"worst by {worst:.3g}"
