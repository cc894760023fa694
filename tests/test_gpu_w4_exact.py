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


def weights(g, n, k, group, dtype, zeros=None):
    q = torch.randint(0, 16, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    size = (n, -(-k // group))
    scales = ((0.5 + torch.rand(size, generator=g, device="cuda")) / (4.6 * k ** 0.5)).to(dtype)
    if zeros == "whole":
        return q, scales, torch.randint(0, 16, size, generator=g, device="cuda").to(dtype)
    return q, scales, (torch.randn(size, generator=g, device="cuda") * 3 + 8).to(dtype) if zeros else None


@pytest.mark.parametrize("t", [1, 8, 40])
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -40, 2.0 ** -60, 2.0 ** -75, 2.0 ** -100, 2.0 ** 60, 2.0 ** 90])
def test_small_and_large_scales(handle, t, kind, size):
    """BF16 x of ordinary size and scales of any: the products are what has to fit FP32."""
    g = gen_of(31)
    q, scales, zeros = weights(g, 72, 544, 64, F32, True)
    scales, zeros = (scales * size).to(kind), zeros.to(kind)
    x = randn(g, t, 544)
    for zero in (None, zeros):
        out = tcg.linear_4bit(handle, x, ref.pack(q), scales, 64, zeros=zero, out_dtype=F32)
        want, bound = expected(x, q, scales, zero, 64)
        if zero is not None:        # the zero's part is taken besides
            at = torch.arange(544, device="cuda") // 64
            bound = bound + 552 * 2.0 ** -23 * (x.double().abs() @ (
                ((8 - zero.double()).abs() + 16) * scales.double())[:, at].t())
        within(out, want, bound, "out")


@pytest.mark.parametrize("t", [1, 8, 40])
@pytest.mark.parametrize("size", [2.0 ** -110, 2.0 ** -80, 2.0 ** -57, 2.0 ** 63, 2.0 ** 100, 2.0 ** 120])
def test_small_and_large_rows(handle, t, size):
    """BF16 x over the type's range."""
    g = gen_of(32)
    q, scales, _ = weights(g, 72, 544, 64, BF16)
    x = (randn(g, t, 544, dtype=F32) / 8 * size).to(BF16)
    within(tcg.linear_4bit(handle, x, ref.pack(q), scales, 64, out_dtype=F32), *expected(x, q, scales, None, 64), "out")


@pytest.mark.parametrize("t", [2, 8, 40])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_infinity_in_x(handle, t, dtype):
    """An infinite entry meets a weight: infinite with its sign, NaN where the weight is zero."""
    g = gen_of(33)
    q, scales, _ = weights(g, 72, 544, 32, dtype)
    x = randn(g, t, 544, dtype=dtype)
    x[1, 77] = float("inf")
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, 32)
    sign = q[:, 77].double() - 8
    assert torch.equal(torch.isnan(out[1]), sign == 0) and bool((sign == 0).any())
    assert torch.equal(out[1][sign != 0].double(), sign[sign != 0] * float("inf"))
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()


def expected_with_zeros(x, q, scales, zeros, group):
    """expected(), a weight's magnitude with what is left of its zero beside the nearest whole number of
    0 .. 15: |q - c| + |c - zero|."""
    k = x.shape[1]
    at = torch.arange(k, device="cuda") // group
    zero, s = zeros.double()[:, at], scales.double()[:, at].abs()
    c = zero.clamp(0, 15).round()
    want, _ = expected(x, q, scales, zeros, group)
    return want, (k + 8) * (2.0 ** -23 * (x.double().abs() @ (((q - c).abs() + (c - zero).abs()) * s).t()) + 2.0 ** -149)


@pytest.mark.parametrize("t", [1, 2, 7, 40, 60])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_weights_at_their_zeros(handle, t, group, dtype):
    """Zeros from 0 to 15: rows of weights that are nearly all at theirs are no difference of large
    sums, where x has a few entries far larger than the others."""
    g = gen_of(t + group + 1)
    k, n = 1184, 136
    scales = (0.5 + torch.rand(n, -(-k // group), generator=g, device="cuda")).to(dtype)
    zeros = (torch.rand(n, -(-k // group), generator=g, device="cuda") * 15).round().to(dtype)
    q = zeros.repeat_interleave(group, 1)[:, :k].to(torch.uint8)
    at = (torch.arange(n, device="cuda"), (torch.arange(n, device="cuda") * 67) % k)
    q[at] = (q[at] + 1) % 16
    x = positive(g, t, k, F32)
    x = torch.where(torch.rand(k, generator=g, device="cuda") < 0.05, 3000 * x, x).to(dtype)
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, group, zeros=zeros, out_dtype=F32)
    within(out, *expected_with_zeros(x, q, scales, zeros, group), "out")


@pytest.mark.parametrize("t", [1, 8, 40, 60])
@pytest.mark.parametrize("dtype,kind", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_zeros_of_any_size(handle, t, dtype, kind, group):
    """Zeros that are no whole numbers, and beyond 0 .. 15."""
    g = gen_of(35)
    q, scales, _ = weights(g, 72, 544, group, kind)
    zeros = (torch.randn(scales.shape, generator=g, device="cuda") * 12 + 8).to(kind)
    zeros[5] = 1000.25
    x = positive(g, t, 544, dtype)
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, group, zeros=zeros, out_dtype=F32)
    within(out, *expected_with_zeros(x, q, scales, zeros, group), "out")


@pytest.mark.parametrize("t", [2, 8, 40])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_infinity_in_x_with_zeros(handle, t, dtype):
    """As without zeros, where they are whole numbers."""
    g = gen_of(36)
    q, scales, zeros = weights(g, 72, 544, 32, dtype, "whole")
    x = randn(g, t, 544, dtype=dtype)
    x[1, 77] = float("-inf")
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, 32, zeros=zeros)
    sign = zeros[:, 77 // 32].double() - q[:, 77].double()
    assert torch.equal(torch.isnan(out[1]), sign == 0) and bool((sign == 0).any())
    assert torch.equal(out[1][sign != 0].double(), sign[sign != 0] * float("inf"))
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()
