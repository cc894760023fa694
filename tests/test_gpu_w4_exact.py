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


# ------------------------------------------------------------------- more tokens, weights expanded
# (tokens, features, k): whole tiles and pieces of them, K no multiple of a block or a group, one block
# and many, 64 tokens and more, several tiles of tokens
EXPANDED = [(129, 520, 1184), (200, 72, 8224), (333, 264, 544), (60, 4128, 4128), (70, 1032, 4160), (700, 136, 1000),
            (257, 8, 32), (130, 2056, 2112), (1100, 300, 4096)]


def expanded(t, rows, k, gated):
    h = tcg.Handle()
    size = tcg.tcg_gemm_4bit_workspace_size(h.h, rows // 2 if gated else rows, t, k, gated)
    h.close()
    return size > 0


@pytest.mark.parametrize("t,n,k", EXPANDED)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,kind", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
def test_many_tokens(handle, t, n, k, group, dtype, kind):
    """Prompts are as exact as single tokens."""
    g = gen_of(t + n + k + group)
    assert expanded(t, n, k, False)
    for zero in (False, True, "whole"):
        q, scales, zeros = weights(g, n, k, group, kind, zero)
        x = randn(g, t, k, dtype=dtype)
        out = tcg.linear_4bit(handle, x, padded_bytes(ref.pack(q)), scales, group, zeros=zeros, out_dtype=F32)
        within(out, *(expected_with_zeros if zero else expected)(x, q, scales, zeros, group), "out")


@pytest.mark.parametrize("t,n,k", [(129, 1040, 1184), (300, 36, 8224), (333, 264, 544), (700, 68, 1000), (260, 1032, 2112)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_tokens_gated(handle, t, n, k, group, dtype):
    g = gen_of(t + n + k + group)
    assert expanded(t, 2 * n, k, True)
    for zero in (False, True):
        q, scales, zeros = weights(g, 2 * n, k, group, dtype, zero)
        x = randn(g, t, k, dtype=dtype)
        out = tcg.linear_4bit(handle, x, padded_bytes(ref.pack(q)), scales, group, zeros=zeros, act="silu", gated=True,
                              out_dtype=F32)
        z, e = (expected_with_zeros if zero else expected)(x, q, scales, zeros, group)
        within(out, *ref.gate(z[:, :n], z[:, n:], e[:, :n], e[:, n:], "silu"), "out")


def padded_bytes(w):
    """Rows a multiple of 16 bytes apart."""
    big = torch.full((w.shape[0], -(-w.shape[1] // 16) * 16), 255, dtype=torch.uint8, device="cuda")
    big[:, :w.shape[1]] = w
    return big[:, :w.shape[1]]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -18, 2.0 ** 18, 2.0 ** 40])
def test_many_tokens_with_small_and_large_scales(handle, dtype, size):
    """Weights beyond the 16-bit type's range, products within FP32's."""
    g = gen_of(41)
    q, scales, _ = weights(g, 264, 544, 64, F32)
    x = randn(g, 200, 544, dtype=dtype)
    scales *= size
    scales[7] *= 2.0 ** 12
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, 64, out_dtype=F32)
    within(out, *expected(x, q, scales, None, 64), "out")


@pytest.mark.parametrize("zero", [None, "whole"])
@pytest.mark.parametrize("gated", [False, True])
def test_many_tokens_with_an_infinity(handle, zero, gated):
    g = gen_of(42)
    q, scales, zeros = weights(g, 72, 544, 32, BF16, zero)
    x = randn(g, 200, 544)
    x[1, 77] = float("inf")
    out = tcg.linear_4bit(handle, x, ref.pack(q), scales, 32, zeros=zeros, gated=gated)
    sign = q[:, 77].double() - (8 if zero is None else zeros[:, 77 // 32].double())
    want = torch.where(sign == 0, float("nan"), sign * float("inf"))
    if gated:
        want = want[:36] * want[36:]
    assert torch.equal(torch.isnan(out[1]), torch.isnan(want)) and bool(torch.isnan(want).any())
    assert torch.equal(out[1][~torch.isnan(want)].double(), want[~torch.isnan(want)])
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()


def test_scales_without_a_number_are_their_rows_alone(handle):
    g = gen_of(43)
    q, scales, zeros = weights(g, 72, 544, 32, BF16, True)
    x = randn(g, 200, 544)
    want = tcg.linear_4bit(handle, x, ref.pack(q), scales, 32, zeros=zeros)
    scales[7, 3], zeros[20, 0] = float("nan"), float("nan")
    got = tcg.linear_4bit(handle, x, ref.pack(q), scales, 32, zeros=zeros)
    rest = [i for i in range(72) if i not in (7, 20)]
    assert torch.isnan(got[:, [7, 20]]).all() and torch.equal(got[:, rest], want[:, rest])
