"""The operators around a decoder layer's products in FP64 torch, from their formulas, and the
element-wise error bounds that the library is held to.  Test code only.

Units as in lm_reference: U of a 16-bit type is half a step relative to the value, sums of K
terms are within K 2^-23 of the sum of the terms' magnitudes.  A row's sums of the norm add at most
64 terms one after the other (32 in a thread, then by halves over at most 1024 threads), each
rounding by 2^-24; with the square root's 2 units and a few products the factor r is within
NORM = 2^-17 of itself (64 2^-24 halved by the root, plus 2^-22).
"""
import torch

from lm_reference import FN, TINY, U, act, slope

NORM = 2.0 ** -17


def norm(x, weight, eps, residual, dtype):
    """(y, its bound before rounding, s, its bound)."""
    s = x.double()
    es = 0.0 * s.abs()
    if residual is not None:
        s = s + residual.double()
        es = 2.0 ** -24 * s.abs()
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * weight.double()
    return y, NORM * y.abs(), s, es + U[dtype] * (s.abs() + es) + TINY[dtype]


def norm_8bit(y):
    """(scale, its bound) of rows y; a stored value stands for its own within half a step: 2^-4 of
    itself, or 2^-10 of the scale below the smallest normal number."""
    scale = (y.abs().amax(1) / 448.0).clamp(min=2.0 ** -100)
    return scale, 2 * NORM * scale


def norm_backward(dout, x, weight, eps, dsum):
    """((dx, dw), their bounds, dx's with its rounding)."""
    d, xd, w = dout.double(), x.double(), weight.double()
    t, k = d.shape
    g = d * w
    r = 1.0 / torch.sqrt(xd.square().mean(1, keepdim=True) + eps)
    dot, mag = (g * xd).mean(1, keepdim=True), (g * xd).abs().mean(1, keepdim=True)
    dx = r * g - xd * r ** 3 * dot
    e = 4 * NORM * (r * g.abs() + xd.abs() * r ** 3 * mag)
    if dsum is not None:
        dx = dx + dsum.double()
        e = e + 2.0 ** -24 * dx.abs()
    dw = (d * xd * r).sum(0)
    ew = (2 * NORM + (t + 64) * 2.0 ** -24) * (d * xd * r).abs().sum(0) + 1e-30
    return (dx, dw), (e + U[x.dtype] * (dx.abs() + e) + TINY[x.dtype], ew)


def gate(g, u, eg, eu, name):
    """(act(g) u, its bound) for g and u within eg and eu."""
    a = act(g, name)
    ea = 1.2 * eg + (FN * g.abs().clamp(min=1.0) if name in ("gelu", "gelu_tanh", "silu") else 0.0)
    return a * u, ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -23 * (a * u).abs()


def gated(x, w, name, out_dtype):
    """(out, its bound, z, its bound before rounding)."""
    k, n = x.shape[1], w.shape[0] // 2
    z = x.double() @ w.double().t()
    ez = (k + 4) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t())
    out, e = gate(z[:, :n], z[:, n:], ez[:, :n], ez[:, n:], name)
    return out, e + U[out_dtype] * (out.abs() + e) + TINY[out_dtype], z, ez


def gated_backward(dout, x, w, z, name):
    """((dx, dw), their bounds)."""
    dtype = x.dtype
    u_, tiny = U[dtype], TINY[dtype]
    n = dout.shape[1]
    d, g, u = dout.double(), z[:, :n].double(), z[:, n:].double()
    dz = torch.cat((d * u * slope(g, name), d * act(g, name)), 1)
    fn = FN * (1 + g.abs()) if name not in ("none", "relu") else 0.0 * g
    e0 = torch.cat((d.abs() * u.abs() * fn, d.abs() * fn), 1) + 2.0 ** -22 * dz.abs()
    e1 = e0 + u_ * (dz.abs() + e0) + tiny
    mag = dz.abs() + e1
    xd, wd = x.double(), w.double()
    dx, dw = dz @ wd, dz.t() @ xd
    ex = e1 @ wd.abs() + (2 * n + 4) * 2.0 ** -23 * (mag @ wd.abs())
    ew = e1.t() @ xd.abs() + (x.shape[0] + 4) * 2.0 ** -23 * (mag.t() @ xd.abs())
    return (dx, dw), (ex + u_ * (dx.abs() + ex) + tiny, ew + u_ * (dw.abs() + ew) + tiny)


def unpack(w, k):
    """(rows, k) of 0 .. 15."""
    return torch.stack((w & 15, w >> 4), 2).flatten(1)[:, :k]


def pack(q):
    """(rows, ceil(k / 2)) bytes; the half after an odd k holds 15, which takes no part."""
    if q.shape[1] % 2:
        q = torch.cat((q, torch.full_like(q[:, :1], 15)), 1)
    return q[:, 0::2] | (q[:, 1::2] << 4)


def weights_4bit(w, k, scales, zeros, group):
    """(W, the magnitude that a group's products are summed with: 16 + q of a weight, and 16 and the
    zero, which are taken away again)."""
    at = torch.arange(k, device=w.device) // group
    q, s = unpack(w, k).double(), scales.double()[:, at]
    zero = torch.full_like(q, 8.0) if zeros is None else zeros.double()[:, at]
    return (q - zero) * s, (32 + q + zero.abs()) * s.abs()


def linear_4bit(x, w, scales, zeros, group, bias, name, residual, beta, gated_, out_dtype):
    """(out, its bound).  A group's sums of at most `group` terms are within their 2^-23 each of the
    magnitudes' sum; all groups' results, at most k, are added with the magnitudes of W."""
    t, k = x.shape
    W, mag = weights_4bit(w, k, scales, zeros, group)
    xd = x.double()
    z = xd @ W.t()
    ez = 2.0 ** -23 * ((min(k, group) + 8) * (xd.abs() @ mag.t()) + (k + 8) * (xd.abs() @ W.abs().t()))
    if t > 48:                               # the weights may be rounded to x's type, once or in two parts
        u, tiny = U[x.dtype] * (1 + 2.0 ** -10), TINY[x.dtype]
        ez = ez + (u * u if gated_ else u) * (xd.abs() @ W.abs().t()) + tiny * xd.abs().sum(1, keepdim=True)
        ez = ez + (k + 8) * 2.0 ** -23 * (xd.abs() @ W.abs().t())
    if gated_:
        n = z.shape[1] // 2
        out, e = gate(z[:, :n], z[:, n:], ez[:, :n], ez[:, n:], name)
    else:
        if bias is not None:
            z = z + bias.double()
            ez = ez + 2.0 ** -23 * z.abs()
        out = act(z, name)
        e = 1.2 * ez + (FN * z.abs().clamp(min=1.0) if name in ("gelu", "gelu_tanh", "silu") else 0.0)
        if residual is not None:
            out = out + beta * residual.double()
            e = e + 2.0 ** -23 * (out.abs() + abs(beta) * residual.double().abs())
    return out, e + U[out_dtype] * (out.abs() + e) + TINY[out_dtype]
