"""4-bit products held to the accuracy that the header states, (k + 8) 2^-23 of the products'
magnitudes |W| |x|, whatever the number of tokens, with FP32 outputs so that no rounding hides it."""
import pytest
import torch

import ffn_reference as ref
import mixed_precision_tensor_gb300 as tcg
from lm_reference import within
from test_gpu_lm import gen_of, randn

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = tcg.Handle()
    yield h
    tcg.check(tcg.tcg_get_device_error(h.h), "device error word")
    h.close()


def expected(x, q, scales, zeros, group):
    """(x W^T in FP64, its bound): W = (q - zero) scale, the magnitudes those of W; FP32 values
    below 2^-126 are within 2^-149 each."""
    k = x.shape[1]
    at = torch.arange(k, device="cuda") // group
    zero = 8.0 if zeros is None else zeros.double()[:, at]
    w = (q.double() - zero) * scales.double()[:, at]
    xd = x.double()
    return xd @ w.t(), (k + 8) * (2.0 ** -23 * (xd.abs() @ w.abs().t()) + 2.0 ** -149)


def positive(g, t, k, dtype):
    """x of one sign: a group's sum of x is as large as its magnitudes' sum."""
    return (torch.rand(t, k, generator=g, device="cuda") + 0.5).to(dtype)


@pytest.mark.parametrize("t", [1, 2, 7, 40, 60, 200])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_of_zero_weights_but_one(handle, t, group, dtype):
    """What the packed form holds beside a weight, its zero, must leave no error where the
    weights themselves are next to nothing."""
    g = gen_of(t + group)
    k, n = 1184, 136
    q = torch.full((n, k), 8, dtype=torch.uint8, device="cuda")
    q[torch.arange(n), (torch.arange(n) * 67) % k] = 9
    scales = (0.5 + torch.rand(n, -(-k // group), generator=g, device="cuda")).to(dtype)
    x = positive(g, t, k, dtype)
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, group, out_dtype=F32)
    within(out, *expected(x, q, scales, None, group), "out")
