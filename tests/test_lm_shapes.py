"""Shapes that the language-model calls refuse or accept before the library sees a pointer,
without a GPU: the library is a stand-in that notes the arguments of a call."""
import pytest
import torch

import mixed_precision_tensor_gb300 as tcg
from mixed_precision_tensor_gb300 import lm

BF16 = torch.bfloat16


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


class Handle:
    h, stream = None, None


@pytest.fixture
def library(monkeypatch):
    """The stand-in, with CPU tensors taken for the GPU's."""
    made = Library()
    monkeypatch.setattr(lm, "_lib", lambda: made)
    monkeypatch.setattr(lm, "_input", lambda x, what="x": (*x.shape, x.dtype, x.device))
    return made


def zeros(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def wide(rows, cols, ld):
    """rows x cols with rows ld apart."""
    return zeros(rows, ld)[:, :cols]


@pytest.mark.parametrize("x,w", [
    (zeros(4, 64), zeros(16, 128)), (zeros(4, 128), zeros(16, 64)),
    (zeros(4, 72), wide(16, 64, 72)), (wide(4, 64, 72), zeros(16, 72)),
])
def test_backward_refuses_features_that_differ(library, x, w):
    dout = zeros(4, 16)
    for want in (("dx", "dw", "dbias"), ("dx",), ("dw",), ("dbias",)):
        with pytest.raises(ValueError, match="w must be"):
            tcg.linear_backward(Handle(), dout, x, w, want=want)
        experts = torch.stack([zeros(*w.shape)] * 3) if w.is_contiguous() else zeros(3, 16, 72)[:, :, :64]
        with pytest.raises(ValueError, match="w must be"):
            tcg.grouped_linear_backward(Handle(), dout, x, experts, torch.zeros(4, dtype=torch.int64), want=want)
    assert not library.calls


def test_backward_refuses_what_is_no_matrix(library):
    x, d, off = zeros(4, 64), zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    for w in (zeros(16), zeros(3, 16, 64)):
        with pytest.raises(ValueError, match="w must be"):
            tcg.linear_backward(Handle(), d, x, w)
    for w in (zeros(16, 64), zeros(16)):
        with pytest.raises(ValueError, match="w must be"):
            tcg.grouped_linear_backward(Handle(), d, x, w, off)
    assert not library.calls


def test_backward_passes_the_shapes_on(library):
    tcg.linear_backward(Handle(), zeros(4, 16), wide(4, 64, 72), wide(16, 64, 80))
    (name, a), = library.calls
    assert name == "tcg_linear_backward"
    assert a[2:5] == (16, 4, 64) and a[12] == 80 and a[15] == 72      # m, n, k, ldw, ldx


# -------------------------------------------------------------------------- another stream
class Stream:
    cuda_stream = 7


@pytest.mark.parametrize("current", [0, 7])
def test_tensors_of_another_stream_are_held(library, monkeypatch, current):
    """Everything whose memory a call uses is recorded with the handle's stream, where that is
    not the current one."""
    held = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: held.append((t.data_ptr(), s)))
    monkeypatch.setattr(lm, "_raw_stream", lambda index: current)
    h = Handle()
    h.stream = Stream()
    x, w, e, d, z, o = zeros(4, 64), zeros(16, 64), zeros(3, 16, 64), zeros(4, 16), zeros(4, 16), zeros(4, 16)
    b, eb, off, r = zeros(16), zeros(3, 16), torch.zeros(4, dtype=torch.int64), zeros(4, 16)
    dx, dw, de, db = zeros(4, 64), zeros(16, 64), zeros(3, 16, 64), torch.zeros(16)
    deb, t, lo, ls, dl = torch.zeros(3, 16), torch.zeros(4, dtype=torch.int64), *(torch.zeros(4) for _ in range(3))
    for call, used in (
            (lambda: tcg.linear(h, x, w, bias=b, residual=r, out=o, z=z), (x, w, b, r, o, z)),
            (lambda: tcg.grouped_linear(h, x, e, off, bias=eb, residual=r, out=o, z=z),
             (x, e, off, eb, r, o, z)),
            (lambda: tcg.linear_backward(h, d, x, w, z=z, act="silu", dx=dx, dw=dw, dbias=db),
             (d, x, w, z, dx, dw, db)),
            (lambda: tcg.grouped_linear_backward(h, d, x, e, off, z=z, act="silu", dx=dx, dw=de, dbias=deb),
             (d, x, e, off, z, dx, de, deb)),
            (lambda: tcg.linear_cross_entropy(h, x, w, t, loss=lo, lse=ls), (x, w, t, lo, ls)),
            (lambda: tcg.linear_cross_entropy_backward(h, x, w, t, ls, dl, dx=dx, dw=dw),
             (x, w, t, ls, dl, dx, dw))):
        held.clear()
        call()
        want = {a.data_ptr() for a in used} if current != 7 else set()
        assert {a for a, _ in held} == want and all(s is h.stream for _, s in held)


# ------------------------------------------------------------------ nothing in one direction
@pytest.mark.parametrize("t,n,k", [(5, 16, 0), (5, 0, 64), (5, 0, 0), (0, 16, 64), (1, 16, 0)])
def test_matrices_without_elements_are_taken(library, t, n, k):
    """A sum over nothing, or nothing to write: contiguous tensors as torch makes them, whose
    strides say nothing about rows, and leading dimensions that the library takes."""
    x, w, dout, z = zeros(t, k), zeros(n, k), zeros(t, n), zeros(t, n)
    tcg.linear(Handle(), x, w, residual=zeros(t, n), z=z, out=zeros(t, n))
    tcg.linear_backward(Handle(), dout, x, w, z=z, act="silu", dx=zeros(t, k), dw=zeros(n, k))
    (_, a), (_, b) = library.calls
    for ld, cols in ((a[8], k), (a[10], k), (a[14], n), (a[15].ldc, n), (a[15].ldz, n),
                     (b[8], n), (b[10], n), (b[12], k), (b[15], k), (b[18], k), (b[20], k)):
        assert ld >= max(cols, 1) and ld % 8 == 0


@pytest.mark.parametrize("e,n,k", [(3, 16, 0), (3, 0, 64), (1, 0, 0), (1, 16, 0)])
def test_experts_without_elements_are_taken(library, e, n, k):
    x, w, off = zeros(5, k), zeros(e, n, k), torch.zeros(e + 1, dtype=torch.int64)
    tcg.grouped_linear(Handle(), x, w, off)
    tcg.grouped_linear_backward(Handle(), zeros(5, n), x, w, off, dw=zeros(e, n, k))
    (_, a), (_, b) = library.calls
    for ld, stride in ((a[9], a[10]), (b[12], b[13]), (b[20], b[21])):
        assert ld >= max(k, 1) and ld % 8 == 0
        assert stride >= (n - 1) * ld + k and stride % 8 == 0 and (stride > 0 or e == 1)
