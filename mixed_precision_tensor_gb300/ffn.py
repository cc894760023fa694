"""The feed-forward half of a decoder layer on torch CUDA tensors: the root-mean-square norm with
the residual stream, gated projections, and projections with 4-bit weights (include/tcg.h, section
"The feed-forward half of a layer").

    hidden = rms_norm(h, x, weight, residual=stream, sum_out=stream)
    x = linear(h, gated_linear(h, hidden, w_gate_up), w_down)        # or linear_4bit

Tensors, streams and the workspace are as in the module ``lm``: row-major FP16 or BF16 matrices, a
row a token, unit stride along the features, rows any multiple of 16 bytes apart.  The workspace
holds dz in :func:`gated_linear_backward` and, for many tokens, the weights of
:func:`linear_4bit` expanded to 16 bits; its sizes are ``tcg_gemm_gated_workspace_size``,
``tcg_gated_backward_workspace_size``, ``tcg_rms_norm_backward_workspace_size`` and
``tcg_gemm_4bit_workspace_size``.
"""
from __future__ import annotations

import torch

import mixed_precision_tensor_gb300 as _tcg

from .lm import (_IN, _TYPES, _act, _elsewhere, _empty, _epilogue, _hold, _input, _lib, _matrix, _out,
                 _rows, _vector, _want)

_E4M3 = torch.float8_e4m3fn


def _norm_args(x, weight, eps, more, what):
    """Sizes, type, device, and the leading dimensions of x and of `more`, another matrix like it."""
    t, k, dtype, dev = _input(x)
    _vector(weight, "weight", (k,), (dtype, torch.float32), dev)
    if not eps >= 0.0:
        raise ValueError(f"eps must not be negative, got {eps}")
    return t, k, dtype, dev, _rows(x, "x", t, k, dtype, dev), \
        8 if more is None else _rows(more, what, t, k, dtype, dev)


def _norm(handle, what, x, weight, eps, residual, sum_out, args, out, ldo, out_code, scale):
    t, k, dtype, dev, ldx, ldr = args
    lds = 8 if sum_out is None else _rows(sum_out, "sum_out", t, k, dtype, dev)
    s = _lib().tcg_rms_norm(
        handle.h, t, k, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
        None if sum_out is None else sum_out.data_ptr(), lds, weight.data_ptr(), _TYPES[weight.dtype], eps,
        _IN[dtype], out.data_ptr(), out_code, ldo, None if scale is None else scale.data_ptr())
    if _elsewhere(handle, dev):
        _hold(handle, x, weight, residual, sum_out, out, scale)
    if s:
        raise _tcg.TcgError(s, what)


def rms_norm(handle, x, weight, eps=1e-6, residual=None, sum_out=None, out=None):
    """out = s / sqrt(mean(s^2) + eps) * weight along each row, s = x + residual.

    x, residual, out: (tokens, k) of one type; weight: (k,) of x's type or FP32; sum_out: (tokens,
    k), receives s rounded to x's type, the residual stream (it may be ``residual`` or ``x``
    itself; out is formed from the unrounded s).  out is made if None and may be ``x`` or
    ``residual``, if sum_out is not the same; what is in another's place has its rows there too.  k is at most 32768.  Returns out.
    """
    args = _norm_args(x, weight, eps, residual, "residual")
    t, k, dtype, dev = args[:4]
    out, ldo = _matrix(handle, out, "out", t, k, dtype, dev)
    _norm(handle, "rms_norm", x, weight, eps, residual, sum_out, args, out, ldo, _IN[dtype], None)
    return out


def rms_norm_8bit(handle, x, weight, eps=1e-6, residual=None, sum_out=None, out=None, scale=None):
    """(out, scale): :func:`rms_norm` in 8 bits, out (tokens, k) torch.float8_e4m3fn and scale
    (tokens,) FP32, which stand for out * scale[:, None].

    scale is a row's largest magnitude over 448, at least 2^-100.  The FP8 products of
    :func:`gemm_rowmajor` take out as it is; multiplying their result's rows by scale is the caller's.
    """
    args = _norm_args(x, weight, eps, residual, "residual")
    t, k, dtype, dev = args[:4]
    out, ldo = _matrix(handle, out, "out", t, k, _E4M3, dev)
    if scale is None:
        scale = _empty(handle, (t,), torch.float32, dev)
    else:
        _vector(scale, "scale", (t,), (torch.float32,), dev)
    _norm(handle, "rms_norm_8bit", x, weight, eps, residual, sum_out, args, out, ldo, _tcg.TCG_R_8F_E4M3, scale)
    return out, scale


def rms_norm_backward(handle, dout, x, weight, eps=1e-6, dsum=None, want=("dx", "dw"), dx=None, dw=None):
    """(dx, dw) of :func:`rms_norm` for dout, the gradient of its output.

    x is what was normalised (sum_out, where there was a residual); dsum, the gradient that arrives
    at sum_out from elsewhere, is added to dx, which is the gradient of x and of the residual alike
    (it may be ``dout`` or ``dsum`` itself).  dw: (k,) FP32.  ``want`` names what is computed; None
    for the other.
    """
    t, k, dtype, dev, ldx, ldds = _norm_args(x, weight, eps, dsum, "dsum")
    ldd = _rows(dout, "dout", t, k, dtype, dev)
    want_dx, want_dw, bad = _want(want)
    if bad:
        raise ValueError("want names dx and dw only")
    lddx = 8
    if want_dx:
        dx, lddx = _matrix(handle, dx, "dx", t, k, dtype, dev)
    if want_dw:
        if dw is None:
            dw = _empty(handle, (k,), torch.float32, dev)
        else:
            _vector(dw, "dw", (k,), (torch.float32,), dev)
    s = _lib().tcg_rms_norm_backward(
        handle.h, t, k, dout.data_ptr(), ldd, x.data_ptr(), ldx, None if dsum is None else dsum.data_ptr(), ldds,
        weight.data_ptr(), _TYPES[weight.dtype], eps, _IN[dtype], dx.data_ptr() if want_dx else None, lddx,
        dw.data_ptr() if want_dw else None)
    if _elsewhere(handle, dev):
        _hold(handle, dout, x, weight, dsum, dx if want_dx else None, dw if want_dw else None)
    if s:
        raise _tcg.TcgError(s, "rms_norm_backward")
    return (dx if want_dx else None, dw if want_dw else None)


def _halves(w, what):
    if w.dim() != 2 or w.shape[0] % 2:
        raise ValueError(f"{what} must have an even number of rows: those of the gate, then as many others")
    return w.shape[0] // 2


def gated_linear(handle, x, w, act="silu", out=None, out_dtype=None, z=None):
    """out = act(g) * u with [g | u] = x @ w.T.

    x: (tokens, k); w: (2 n, k), the n rows that give g, then the n that give u; out: (tokens, n) of
    x's type or FP32, made if None; z: (tokens, 2 n) of x's type, receives [g | u], which
    :func:`gated_linear_backward` wants.  Sums as in :func:`linear`.  Returns out.
    """
    t, k, dtype, dev = _input(x)
    n = _halves(w, "w")
    ldw = _rows(w, "w", 2 * n, k, dtype, dev)
    ldx = _rows(x, "x", t, k, dtype, dev)
    ldz = 8 if z is None else _rows(z, "z", t, 2 * n, dtype, dev)
    out, ldo, out_code = _out(handle, out, out_dtype, t, n, dtype, dev)
    s = _lib().tcg_gemm_gated(handle.h, _act(act), n, t, k, w.data_ptr(), ldw, x.data_ptr(), ldx, _IN[dtype],
                              out.data_ptr(), out_code, ldo, None if z is None else z.data_ptr(), ldz)
    if _elsewhere(handle, dev):
        _hold(handle, x, w, out, z)
    if s:
        raise _tcg.TcgError(s, "gated_linear")
    return out


def gated_linear_backward(handle, dout, x, w, z, act="silu", want=("dx", "dw"), dx=None, dw=None):
    """(dx, dw) of :func:`gated_linear` for dout, the gradient of its output.

    With dz = [dout * u * act'(g) | dout * act(g)]: dx = dz @ w, dw = dz.T @ x.  dz is rounded to
    the type of x before the two products (in BF16 their 2-norm error is 0.0023 of the result, 0.0017
    without that rounding; in FP16 0.0003 and 0.0002).  ``want`` names what is computed; None for the other.
    """
    t, k, dtype, dev = _input(x)
    n = _halves(w, "w")
    ldw = _rows(w, "w", 2 * n, k, dtype, dev)
    ldx = _rows(x, "x", t, k, dtype, dev)
    ldd = _rows(dout, "dout", t, n, dtype, dev)
    ldz = _rows(z, "z", t, 2 * n, dtype, dev)
    want_dx, want_dw, bad = _want(want)
    if bad:
        raise ValueError("want names dx and dw only")
    lddx = lddw = 8
    if want_dx:
        dx, lddx = _matrix(handle, dx, "dx", t, k, dtype, dev)
    if want_dw:
        dw, lddw = _matrix(handle, dw, "dw", 2 * n, k, dtype, dev)
    s = _lib().tcg_gated_backward(
        handle.h, _act(act), n, t, k, dout.data_ptr(), ldd, z.data_ptr(), ldz, w.data_ptr(), ldw, x.data_ptr(),
        ldx, _IN[dtype], dx.data_ptr() if want_dx else None, lddx, dw.data_ptr() if want_dw else None, lddw)
    if _elsewhere(handle, dev):
        _hold(handle, dout, x, w, z, dx if want_dx else None, dw if want_dw else None)
    if s:
        raise _tcg.TcgError(s, "gated_linear_backward")
    return (dx if want_dx else None, dw if want_dw else None)


def linear_4bit(handle, x, w, scales, group, zeros=None, bias=None, act="none", residual=None, beta=1.0,
                gated=False, out=None, out_dtype=None):
    """:func:`linear` with weights of 4 bits: out = act(x @ W.T + bias) + beta * residual, or with
    ``gated`` :func:`gated_linear`, where

        W[i, j] = (q[i, j] - zeros[i, j // group]) * scales[i, j // group].

    w: (n, (k + 1) // 2) uint8, q[i, 2 j] in the low half of w[i, j] and q[i, 2 j + 1] in the high
    half, rows a multiple of 16 bytes apart; scales and zeros: (n, ceil(k / group)) of x's type or
    both FP32, contiguous; without zeros they are 8.  group: 32, 64 or 128.  With ``gated``, n is
    twice the features of out, and there is no bias or residual.  For float weights v,

        s = v.unflatten(1, (-1, group)).abs().amax(2) / 7
        q = (v.unflatten(1, (-1, group)) / s[..., None]).round().add(8).clamp(1, 15).flatten(1).byte()
        w = q[:, 0::2] | q[:, 1::2] << 4

    residual may be ``out`` itself.  Weights are not rounded: q less a whole number (8, or the one
    nearest to its zero) enters the product, which meets the scale in FP32.  Where zeros are no
    whole numbers, an infinity in x makes its token's outputs NaN.  Few tokens (up to 48, 64 of at
    most 2^24 weights, 128 of at most 2^21; gated 128, 256 of at most 2^21) read the packed weights,
    more expand them in the handle's workspace to 16 bits.  Returns out.
    """
    t, k, dtype, dev = _input(x)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a two-dimensional uint8 tensor")
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    rows = w.shape[0]
    n = _halves(w, "w") if gated else rows
    ldw = _rows(w, "w", rows, (k + 1) // 2, torch.uint8, dev)
    ldx = _rows(x, "x", t, k, dtype, dev)
    shape = (rows, (k + group - 1) // group)
    _vector(scales, "scales", shape, (dtype, torch.float32), dev)
    if zeros is not None:
        _vector(zeros, "zeros", shape, (scales.dtype,), dev)
    if gated and (bias is not None or residual is not None):
        raise ValueError("a gated product takes no bias and no residual")
    out, ldo, out_code = _out(handle, out, out_dtype, t, n, dtype, dev)
    e = _epilogue(_act(act), bias, (n,), residual, beta, None, t, n, dtype, out.dtype, dev)
    s = _lib().tcg_gemm_4bit(
        handle.h, n, t, k, group, w.data_ptr(), ldw, scales.data_ptr(),
        None if zeros is None else zeros.data_ptr(), _TYPES[scales.dtype], x.data_ptr(), ldx, _IN[dtype],
        out.data_ptr(), out_code, ldo, gated, e)
    if _elsewhere(handle, dev):
        _hold(handle, x, w, scales, zeros, bias, residual, out)
    if s:
        raise _tcg.TcgError(s, "linear_4bit")
    return out
