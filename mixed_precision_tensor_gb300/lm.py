"""Language-model products on torch CUDA tensors: linear layers, layers of experts, and the
cross entropy of a linear head, forward and backward (include/tcg.h, section "Language-model
products").

Row-major: a row is a token.  Inputs are FP16 or BF16, two-dimensional with unit stride
along the features; rows may be any multiple of 16 bytes apart, so feature counts that are
no multiple of 8 need padded rows.  Every call queues on the handle's stream; inputs must be
ready there, and tensors that a call allocates belong to that stream.  Where that is not the
caller's current stream, the caller may drop its tensors at once: their memory is held until
the handle's stream is done.  This module checks and marshals; all arithmetic is in the
library's kernels.

Calls do not wait for the GPU, with one exception: the handle keeps a workspace, outside
torch's allocator and until it is closed, as large as the largest that a call has needed (all
of dz in a backward pass with an activation, up to 256 MiB of the cross entropy's gradient and
an FP32 dx).  A call that needs more than any before waits for the stream and allocates anew;
while a graph is being captured it is refused instead (TCG_STATUS_ALLOC_FAILED).  To avoid
both, run the largest shapes once first, or give the handle memory of your own with
``tcg_set_workspace``, sized by ``tcg_gemm_epilogue_workspace_size``,
``tcg_linear_backward_workspace_size`` and ``tcg_xent_workspace_size``.
"""
from __future__ import annotations

import torch

import mixed_precision_tensor_gb300 as _tcg

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_IN = {torch.float16: 0, torch.bfloat16: 1}                  # TCG_R_16F, TCG_R_16BF
# the current stream's cudaStream_t by device index, without making a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _lib():
    return _tcg._lib or _tcg.load_library()


def _rows(t, what, rows, cols, dtype, device):
    """Leading dimension of a rows x cols matrix, checked."""
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must be {rows} x {cols}, got {tuple(t.shape)}")
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what} must be {dtype} on {device}, got {t.dtype} on {t.device}")
    s0, s1 = t.stride()
    per = 4 if dtype is torch.float32 else 8
    if s1 != 1 and cols > 1:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    if rows <= 1 or cols == 0:                # no stride between rows to go by
        return (cols + per - 1) // per * per or per
    if s0 < cols or s0 % per:
        raise ValueError(f"{what}: rows must be a multiple of 16 bytes apart, got {s0} elements")
    return s0


def _input(x, what="x"):
    dtype = x.dtype if isinstance(x, torch.Tensor) else None
    if dtype not in _IN:
        raise ValueError(f"{what} must be a float16 or bfloat16 tensor, got {dtype}")
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{what} must be a two-dimensional CUDA tensor")
    t, k = x.shape
    return t, k, dtype, x.device


def _act(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _empty(handle, shape, dtype, device):
    """A new tensor of the handle's stream."""
    if not _elsewhere(handle, device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(handle.stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _elsewhere(handle, device):
    """Whether the handle's stream is another one than the caller's."""
    own = handle.stream
    return own is not None and _raw_stream(device.index) != own.cuda_stream


def _hold(handle, *tensors):
    """The caller's tensors on the handle's stream: should the caller drop one, torch gives its
    memory out again only once that stream is done with it."""
    for t in tensors:
        if t is not None:
            t.record_stream(handle.stream)


def _matrix(handle, given, what, rows, cols, dtype, device):
    """A rows x cols matrix for a result -- the given one, or a new one whose rows are a
    multiple of 16 bytes apart -- and its leading dimension."""
    if given is not None:
        return given, _rows(given, what, rows, cols, dtype, device)
    per = 4 if dtype is torch.float32 else 8
    ld = (cols + per - 1) // per * per or per
    new = _empty(handle, (rows, ld), dtype, device)
    return (new if ld == cols else new[:, :cols]), ld


def _experts(w, what, e, n, k, dtype, device):
    """(leading dimension, stride between experts) of an e x n x k tensor, checked."""
    if w.shape != (e, n, k):
        raise ValueError(f"{what} must be {e} x {n} x {k}, got {tuple(w.shape)}")
    if w.dtype is not dtype or w.device != device:
        raise ValueError(f"{what} must be {dtype} on {device}")
    stride, ld, s2 = w.stride()
    if s2 != 1 and k > 1:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    if n <= 1 or k == 0:                      # no stride between rows to go by
        ld = (k + 7) // 8 * 8 or 8
    if ld < k or ld % 8:
        raise ValueError(f"{what}: rows must be a multiple of 16 bytes apart, got {ld} elements")
    if e <= 1 or n == 0 or k == 0:
        stride = max(n, 1) * ld
    elif stride <= 0 or stride % 8:
        raise ValueError(f"{what}: experts must be a multiple of 16 bytes apart")
    return ld, stride


def _vector(t, what, shape, dtypes, device):
    if t.shape != shape or t.dtype not in dtypes or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {shape} tensor of "
                         f"{' or '.join(map(str, dtypes))} on {device}")
    return t


def _epilogue(act, bias, bias_shape, residual, beta, z, rows, n, dtype, out_dtype, device):
    e = _tcg.Epilogue()
    e.activation = act
    if bias is not None:
        _vector(bias, "bias", bias_shape, (dtype, torch.float32), device)
        e.bias, e.bias_type = bias.data_ptr(), _TYPES[bias.dtype]
    if residual is not None and beta != 0.0:
        e.ldc = _rows(residual, "residual", rows, n, out_dtype, device)
        e.C, e.beta = residual.data_ptr(), beta
    if z is not None:
        e.ldz = _rows(z, "z", rows, n, dtype, device)
        e.Z = z.data_ptr()
    return e


def _out(handle, out, out_dtype, rows, n, dtype, device):
    """The output (made if None), its leading dimension and type code."""
    if out is not None:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out and out_dtype disagree")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        raise ValueError(f"the output must be {dtype} or torch.float32, got {out_dtype}")
    out, ld = _matrix(handle, out, "out", rows, n, out_dtype, device)
    return out, ld, _TYPES[out_dtype]


def linear(handle, x, w, bias=None, act="none", residual=None, beta=1.0, alpha=1.0, out=None,
           out_dtype=None, z=None):
    """out = act(alpha * x @ w.T + bias) + beta * residual.

    x: (tokens, k); w: (n, k); bias: (n,) of x's type or FP32; residual: (tokens, n) of the
    output's type (it may be ``out`` itself); out: (tokens, n) of x's type or FP32, made if
    None; z: (tokens, n) of x's type, receives the pre-activation that
    :func:`linear_backward` wants.  act: "none", "relu", "gelu", "gelu_tanh" or "silu".
    Returns out.

    FP32 outputs are as exact as the tensor core's FP32 sums, which cut off rather than round:
    for long calls (2-norm, 2048 x 2048 outputs) 4e-6 of the result at k = 4096, 2e-5 at 16384;
    calls of few tokens, whose sums are joined from segments of 512, 4e-7.
    """
    t, k, dtype, dev = _input(x)
    n = w.shape[0]
    ldw = _rows(w, "w", n, k, dtype, dev)
    ldx = _rows(x, "x", t, k, dtype, dev)
    out, ldo, out_code = _out(handle, out, out_dtype, t, n, dtype, dev)
    e = _epilogue(_act(act), bias, (n,), residual, beta, z, t, n, dtype, out.dtype, dev)
    code = _IN[dtype]
    s = _lib().tcg_gemm_epilogue(
        handle.h, 1, 0, n, t, k, alpha, w.data_ptr(), ldw, x.data_ptr(), ldx, code, out.data_ptr(),
        out_code, ldo, e)
    if _elsewhere(handle, dev):
        _hold(handle, x, w, bias, residual, out, z)
    if s:
        raise _tcg.TcgError(s, "linear")
    return out


def _backward(handle, what, dout, x, w, z, act, want, dx, dw, dbias, offsets, e, n, ldw, stride_w):
    """The one call behind the two backward passes."""
    t, k, dtype, dev = _input(x)
    ldx = _rows(x, "x", t, k, dtype, dev)
    ldd = _rows(dout, "dout", t, n, dtype, dev)
    code = _act(act)
    ldz = 8
    if code:
        if z is None:
            raise ValueError(f"z, the pre-activation of the forward pass, is needed for act={act!r}")
        ldz = _rows(z, "z", t, n, dtype, dev)
    want_dx, want_dw, want_db = _want(want)
    lddx = lddw = 8
    stride_dw = 0
    if want_dx:
        dx, lddx = _matrix(handle, dx, "dx", t, k, dtype, dev)
    if want_dw and offsets is None:
        dw, lddw = _matrix(handle, dw, "dw", n, k, dtype, dev)
    elif want_dw:
        if dw is None:
            lddw = (k + 7) // 8 * 8 or 8
            stride_dw = n * lddw
            dw = _empty(handle, (e, n, lddw), dtype, dev)
            if lddw != k:
                dw = dw[:, :, :k]
        else:
            lddw, stride_dw = _experts(dw, "dw", e, n, k, dtype, dev)
    if want_db:
        shape = (n,) if offsets is None else (e, n)
        if dbias is None:
            dbias = _empty(handle, shape, torch.float32, dev)
        else:
            _vector(dbias, "dbias", shape, (torch.float32,), dev)
    s = _lib().tcg_linear_backward(
        handle.h, code, n, t, k, e, None if offsets is None else offsets.data_ptr(), dout.data_ptr(), ldd,
        z.data_ptr() if code else None, ldz, w.data_ptr(), ldw, stride_w, x.data_ptr(), ldx, _IN[dtype],
        dx.data_ptr() if want_dx else None, lddx, dw.data_ptr() if want_dw else None, lddw, stride_dw,
        dbias.data_ptr() if want_db else None)
    if _elsewhere(handle, dev):
        _hold(handle, dout, x, w, z if code else None, offsets, dx if want_dx else None,
              dw if want_dw else None, dbias if want_db else None)
    if s:
        raise _tcg.TcgError(s, what)
    return (dx if want_dx else None, dw if want_dw else None, dbias if want_db else None)


def _want(want):
    if not set(want) <= {"dx", "dw", "dbias"}:
        raise ValueError("want names dx, dw and dbias only")
    return "dx" in want, "dw" in want, "dbias" in want


def linear_backward(handle, dout, x, w, z=None, act="none", want=("dx", "dw", "dbias"), dx=None,
                    dw=None, dbias=None):
    """Gradients of :func:`linear` (alpha = 1) for dout, the gradient of its output.

    With dz = dout * act'(z): dx = dz @ w, dw = dz.T @ x, dbias = dz.sum(0) (FP32, from the
    unrounded dz).  With an activation, dz is rounded to the type of x before the two products
    (in BF16 their 2-norm error is 0.0024 of the result, 0.0017 without that rounding).  The
    residual's gradient is beta * dout.  ``want`` names what is computed;
    the result is (dx, dw, dbias) with None for the others.  Outputs are made where not given.
    """
    _, k, dtype, dev = _input(x)
    n = w.shape[0]
    ldw = _rows(w, "w", n, k, dtype, dev)
    return _backward(handle, "linear_backward", dout, x, w, z, act, want, dx, dw, dbias, None, 1, n, ldw, 0)


def _check_offsets(offsets, e, device):
    _vector(offsets, "offsets", (e + 1,), (torch.int64,), device)


def grouped_linear(handle, x, w, offsets, bias=None, act="none", residual=None, beta=1.0, alpha=1.0,
                   out=None, out_dtype=None, z=None):
    """A layer of experts on rows sorted by expert: for every expert e and its rows
    offsets[e] .. offsets[e + 1] - 1 of x,

        out[rows] = act(alpha * x[rows] @ w[e].T + bias[e]) + beta * residual[rows].

    x: (rows, k); w: (experts, n, k); offsets: int64 CUDA tensor of experts + 1
    non-decreasing entries in 0 .. rows, read when the kernel runs (no host
    synchronisation); bias: (experts, n).  Rows of no expert come out zero.  The rest as in
    :func:`linear`.  At most 384 experts.
    """
    t, k, dtype, dev = _input(x)
    if w.dim() != 3:
        raise ValueError("w must be experts x n x k")
    e, n = w.shape[0], w.shape[1]
    ldw, stride = _experts(w, "w", e, n, k, dtype, dev)
    ldx = _rows(x, "x", t, k, dtype, dev)
    _check_offsets(offsets, e, dev)
    out, ldo, out_code = _out(handle, out, out_dtype, t, n, dtype, dev)
    ep = _epilogue(_act(act), bias, (e, n), residual, beta, z, t, n, dtype, out.dtype, dev)
    s = _lib().tcg_gemm_grouped(
        handle.h, 1, n, t, k, e, offsets.data_ptr(), alpha, w.data_ptr(), ldw, stride, x.data_ptr(),
        ldx, _IN[dtype], out.data_ptr(), out_code, ldo, ep)
    if _elsewhere(handle, dev):
        _hold(handle, x, w, offsets, bias, residual, out, z)
    if s:
        raise _tcg.TcgError(s, "grouped_linear")
    return out


def grouped_linear_backward(handle, dout, x, w, offsets, z=None, act="none",
                            want=("dx", "dw", "dbias"), dx=None, dw=None, dbias=None):
    """Gradients of :func:`grouped_linear` (alpha = 1): dx (rows, k), zero for rows of no
    expert; dw (experts, n, k), zero for an expert without rows; dbias (experts, n), FP32.
    Arguments as in :func:`linear_backward`.
    """
    if w.dim() != 3:
        raise ValueError("w must be experts x n x k")
    _, k, dtype, dev = _input(x)
    e, n = w.shape[0], w.shape[1]
    ldw, stride = _experts(w, "w", e, n, k, dtype, dev)
    _check_offsets(offsets, e, dev)
    return _backward(handle, "grouped_linear_backward", dout, x, w, z, act, want, dx, dw, dbias, offsets, e, n,
                     ldw, stride)


def _xent_args(x, w, targets):
    t, k, dtype, dev = _input(x)
    v = w.shape[0]
    ldx, ldw = _rows(x, "x", t, k, dtype, dev), _rows(w, "w", v, k, dtype, dev)
    _vector(targets, "targets", (t,), (torch.int64,), dev)
    return t, v, k, dtype, dev, ldx, ldw


def linear_cross_entropy(handle, x, w, targets, ignore_index=-100, loss=None, lse=None):
    """(loss, lse) of the softmax cross entropy of the logits x @ w.T, which are never stored:
    per row, FP32, lse = logsumexp(logits) and loss = lse - logits[target].

    x: (rows, k); w: (vocab, k); targets: (rows,) int64.  A row whose target is ignore_index
    or outside 0 .. vocab - 1 has loss 0.
    """
    t, v, k, dtype, dev, ldx, ldw = _xent_args(x, w, targets)
    loss = _empty(handle, (t,), torch.float32, dev) if loss is None else loss
    lse = _empty(handle, (t,), torch.float32, dev) if lse is None else lse
    _vector(loss, "loss", (t,), (torch.float32,), dev)
    _vector(lse, "lse", (t,), (torch.float32,), dev)
    s = _lib().tcg_xent_forward(
        handle.h, t, v, k, x.data_ptr(), ldx, w.data_ptr(), ldw, _IN[dtype], targets.data_ptr(),
        ignore_index, loss.data_ptr(), lse.data_ptr())
    if _elsewhere(handle, dev):
        _hold(handle, x, w, targets, loss, lse)
    if s:
        raise _tcg.TcgError(s, "linear_cross_entropy")
    return loss, lse


def linear_cross_entropy_backward(handle, x, w, targets, lse, dloss, ignore_index=-100,
                                  want=("dx", "dw"), dx=None, dw=None):
    """(dx, dw) of :func:`linear_cross_entropy` for dloss, the gradient of each row's loss
    (FP32; 1 / rows for a mean), and the lse that it returned.  The gradient of the logits is
    rounded to the type of x before the two products (in BF16 their 2-norm error is about 0.0023
    of the result, 0.0017 without; in FP16 0.0003 and 0.0002), times one factor for all rows:
    FP16 holds it to 2^-39 of the largest |dloss|.  ``want`` names what is computed; None for the
    other.
    """
    t, v, k, dtype, dev, ldx, ldw = _xent_args(x, w, targets)
    _vector(lse, "lse", (t,), (torch.float32,), dev)
    _vector(dloss, "dloss", (t,), (torch.float32,), dev)
    want_dx, want_dw, bad = _want(want)
    if bad:
        raise ValueError("want names dx and dw only")
    lddx = lddw = 8
    if want_dx:
        dx, lddx = _matrix(handle, dx, "dx", t, k, dtype, dev)
    if want_dw:
        dw, lddw = _matrix(handle, dw, "dw", v, k, dtype, dev)
    s = _lib().tcg_xent_backward(
        handle.h, t, v, k, x.data_ptr(), ldx, w.data_ptr(), ldw, _IN[dtype], targets.data_ptr(),
        ignore_index, lse.data_ptr(), dloss.data_ptr(), dx.data_ptr() if want_dx else None, lddx,
        dw.data_ptr() if want_dw else None, lddw)
    if _elsewhere(handle, dev):
        _hold(handle, x, w, targets, lse, dloss, dx if want_dx else None, dw if want_dw else None)
    if s:
        raise _tcg.TcgError(s, "linear_cross_entropy_backward")
    return (dx if want_dx else None, dw if want_dw else None)
