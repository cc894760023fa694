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
