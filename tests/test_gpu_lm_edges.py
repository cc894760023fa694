"""Edges of the language-model products: nothing to sum, nothing to write, values far apart."""
import math

import pytest
import torch

import lm_reference as ref
import mixed_precision_tensor_gb300 as tcg
from test_gpu_lm import BF16, F16, F32, gen_of, offsets_of, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = tcg.Handle()
    yield h
    tcg.check(tcg.tcg_get_device_error(h.h), "device error word")
    h.close()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_experts_without_any_rows(handle, dtype, act):
    """No tokens at all: zero weight and bias gradients for every expert, dx of no rows."""
    g = gen_of(1)
    e, n, k = 5, 200, 136
    w, off = randn(g, e, n, k, dtype=dtype), offsets_of([0] * e, 0)
    x, d, z = (torch.empty(0, c, dtype=dtype, device="cuda") for c in (k, n, n))
    assert tcg.grouped_linear(handle, x, w, off, act=act).shape == (0, n)
    dw = torch.full((e, n, k), float("nan"), dtype=dtype, device="cuda")
    db = torch.full((e, n), float("nan"), device="cuda")
    dx, _, _ = tcg.grouped_linear_backward(handle, d, x, w, off, z=z, act=act, dw=dw, dbias=db)
    assert dx.shape == (0, k) and (dw == 0).all() and (db == 0).all()
    ty = tcg.TCG_R_16BF if dtype is BF16 else tcg.TCG_R_16F
    dw.fill_(float("nan"))
    tcg.check(tcg.tcg_gemm_grouped_k(handle.h, k, n, 0, e, off, 1.0, None, k, None, n, ty, dw, ty, k, n * k))
    assert (dw == 0).all()
    tcg.check(tcg.tcg_get_device_error(handle.h))


def test_nothing_to_sum_or_to_write(handle):
    """Contiguous tensors without elements: the bias alone, zero gradients, or no output."""
    g = gen_of(2)
    empty = lambda *shape: torch.empty(*shape, dtype=BF16, device="cuda")  # noqa: E731
    bias, e_bias, res = randn(g, 256), randn(g, 3, 256), randn(g, 45, 256)
    off = offsets_of([20, 0, 25], 0)
    out = tcg.linear(handle, empty(45, 0), empty(256, 0), bias=bias, residual=res)
    assert torch.equal(out, (bias.float() + res.float()).to(BF16))
    out = tcg.grouped_linear(handle, empty(45, 0), empty(3, 256, 0), off, bias=e_bias)
    assert torch.equal(out, torch.cat([e_bias[0].expand(20, 256), e_bias[2].expand(25, 256)]))
    d = randn(g, 45, 256)
    dx, dw, db = tcg.linear_backward(handle, d, empty(45, 0), empty(256, 0))
    assert dx.shape == (45, 0) and dw.shape == (256, 0)
    off_by = (db.double() - d.double().sum(0)).abs()
    assert (off_by <= (45 + 4) * 2.0 ** -24 * d.double().abs().sum(0)).all()   # FP32 additions
    dx, dw, db = tcg.linear_backward(handle, empty(45, 0), randn(g, 45, 64), empty(0, 64))
    assert dx.shape == (45, 64) and not dx.any() and dw.shape == (0, 64) and db.shape == (0,)
    dx, dw, db = tcg.grouped_linear_backward(handle, empty(45, 0), randn(g, 45, 64), empty(3, 0, 64), off)
    assert not dx.any() and dw.shape == (3, 0, 64) and db.shape == (3, 0)
    assert tcg.linear(handle, randn(g, 45, 64), empty(0, 64)).shape == (45, 0)
    tcg.check(tcg.tcg_get_device_error(handle.h))


@pytest.mark.parametrize("t", [1, 2, 3, 20, 200])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("top", [91, 103, 117])
def test_log_sum_exp_of_large_logits(handle, t, dtype, top):
    """Whole logits of 50 below `top` to `top` over a large vocabulary, as a few tokens, tokens on
    the columns and tokens on the rows.

    Products and sums of the logits are exact.  The sum of exponentials is off by 1.5 2^-22 of
    itself for exp, as much for each of at most four rescalings that change the maximum, and
    2^-24 for each of at most 110 additions in a row; the logarithm by 2^-20; and lse, between
    64 and 128, is rounded to 2^-17 apart: 1.3e-5, less than 2^-16 together."""
    g = gen_of(t + top)
    v, k = 100003, 16
    x, w = torch.zeros(t, k, dtype=dtype, device="cuda"), torch.zeros(v, k, dtype=dtype, device="cuda")
    x[:, 0] = 1
    x[:, 1] = torch.arange(t, device="cuda") % 3 - 1
    w[:, 0] = torch.randint(top - 50, top, (v,), generator=g, device="cuda").to(dtype)
    w[:, 1] = torch.randint(-1, 1, (v,), generator=g, device="cuda").to(dtype)
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target)
    logits = x.double() @ w.double().t()
    want = torch.logsumexp(logits, 1)
    assert float((lse.double() - want).abs().max()) <= 2.0 ** -16
    off = loss.double() - (want - logits.gather(1, target[:, None])[:, 0])
    assert float(off.abs().max()) <= 2.0 ** -16 + 2.0 ** -18


@pytest.mark.parametrize("t", [3, 200])
@pytest.mark.parametrize("top", [101, 103, 116])
def test_gradient_of_a_certain_row(handle, t, top):
    """A target 50 above everything else: its probability is one less 2e-17, and exp is within
    2^-22 of itself, so the gradient of the logits has nothing above that."""
    v, k = 5003, 16
    x, w = torch.zeros(t, k, dtype=BF16, device="cuda"), torch.zeros(v, k, dtype=BF16, device="cuda")
    x[:, 0] = 1
    w[:, 0] = top - 50
    w[7, 0] = top
    target = torch.full((t,), 7, device="cuda")
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    assert (lse == top).all()
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, torch.ones(t, device="cuda"))
    assert float(dx.abs().max()) <= top * 2.0 ** -21 and float(dw.abs().max()) <= t * 2.0 ** -21


@pytest.mark.parametrize("t", [1, 40, 300])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gelu_is_right_to_its_own_size(handle, t, dtype):
    """FP32 outputs of GELU over its whole left tail, and its slope, relative to themselves.

    Phi(-|z|): 1.3e-6 of itself (the fit, 1 / x and exp of 2^-22 each, the polynomial's FP32
    sums) and z^2 7.5e-8 (exp's argument, rounded twice); one more rounding for the product."""
    z = torch.linspace(-12, 12, 4801, device="cuda").to(dtype)
    n, k = z.shape[0], 8
    x = torch.zeros(t, k, dtype=dtype, device="cuda")
    w = torch.zeros(n, k, dtype=dtype, device="cuda")
    x[:, 0], w[:, 0] = 1, z
    out = tcg.linear(handle, x, w, act="gelu", out_dtype=F32)
    zd = z.double()
    want = ref.act(zd, "gelu")
    bound = (2e-6 + 1e-7 * zd * zd) * want.abs() + 2.0 ** -120
    assert ((out.double() - want).abs() <= bound).all()
    # one token's bias gradient is the slope in FP32: Phi + z phi
    dout = torch.ones(1, 4808, dtype=dtype, device="cuda")[:, :n]
    zrow = torch.zeros(1, 4808, dtype=dtype, device="cuda")
    zrow[0, :n] = z
    db = tcg.linear_backward(handle, dout, x[:1], w, z=zrow[:, :n], act="gelu", want=("dbias",))[2]
    tail = 0.5 * torch.special.erfc(-zd / math.sqrt(2.0))
    phi = zd.abs() * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    bound = (2e-6 + 1e-7 * zd * zd) * (tail + phi) + 2.0 ** -120
    assert ((db.double() - ref.slope(zd, "gelu")).abs() <= bound).all()


@pytest.mark.parametrize("group_m", [1, 3, 1024])
def test_tile_order_does_not_change_results(cuda_device, group_m):
    """More rows of tiles walked together than there are, or fewer: the same bits."""
    g = gen_of(6)
    x, w, we = randn(g, 700, 264), randn(g, 1000, 264, std=1 / 16), randn(g, 3, 520, 264, std=1 / 16)
    off = offsets_of([300, 0, 350], 20)
    h = tcg.Handle()
    want = tcg.linear(h, x, w, act="silu"), tcg.grouped_linear(h, x, we, off), \
        *tcg.grouped_linear_backward(h, randn(g, 700, 520), x, we, off)[:1]
    g = gen_of(6)
    x, w, we = randn(g, 700, 264), randn(g, 1000, 264, std=1 / 16), randn(g, 3, 520, 264, std=1 / 16)
    tcg.check(tcg.tcg_set_kernel_options(h.h, 2, group_m))
    got = tcg.linear(h, x, w, act="silu"), tcg.grouped_linear(h, x, we, off), \
        *tcg.grouped_linear_backward(h, randn(g, 700, 520), x, we, off)[:1]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


@pytest.mark.parametrize("t", [3, 20, 300])
@pytest.mark.parametrize("k", [1024, 4096, 8192])
@pytest.mark.parametrize("logit", [24.0, 40.0, 100.0])
def test_gradient_of_certain_rows_over_a_long_sum(handle, t, k, logit):
    """Rows whose target stands out: 1 - p is the rest's probability, so dx has to vanish but
    for what the logits that it is formed from differ by from those of lse.

    Over 32 rows both come from the same sums: lse is rounded (2^-24 of itself), exp is within
    2^-22, and so is what is taken from it.  With fewer rows the sums are in another order:
    segments of 512 of K, 32 additions each, cut off at 2^-23 of the terms (all of one sign)."""
    g = gen_of(k + t)
    v = 3001
    x, w = randn(g, t, k), randn(g, v, k, std=0.5 * k ** -0.5)
    w[:t] = (logit * x.float() / x.float().square().sum(1, keepdim=True)).to(BF16)
    target = torch.arange(t, device="cuda")
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    dx, _ = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, torch.ones(t, device="cuda"))
    logits = x.double() @ w.double().t()
    p = torch.softmax(logits, 1)
    rest = p.sum(1) - p[target, target]
    off = lse.double() * 2.0 ** -23 + 2.0 ** -21
    if t <= 32:
        off = off + 2 * (32 + k / 512) * 2.0 ** -23 * (x.double().abs() * w[:t].double().abs()).sum(1)
    bound = 1.01 * (off + 2 * rest) * w.double().abs().max()
    assert (dx.double().abs() <= bound[:, None]).all(), float((dx.double().abs().amax(1) / bound).max())


@pytest.mark.parametrize("t", [1, 5, 200])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dloss", [1 + 2.0 ** -8 + 2.0 ** -12, (1 + 2.0 ** -8 + 2.0 ** -12) / 200, 1.0])
def test_gradients_of_a_mean_balance(handle, t, dtype, dloss):
    """A row's gradients of the logits sum to zero.  Equal logits and one upstream gradient for
    all rows: what is left are the roundings of 1 / vocab (times the vocabulary) and of
    1 - 1 / vocab, whatever the upstream gradient's own bits; FP32 adds less than 2^-18."""
    v, k = 2731, 16                           # 1 / 2731 = 1.4998 2^-12
    x, w = torch.zeros(t, k, dtype=dtype, device="cuda"), torch.zeros(v, k, dtype=dtype, device="cuda")
    w[:, 0] = 1
    target = torch.arange(t, device="cuda")
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    d = torch.full((t,), dloss, device="cuda")
    dx, _ = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, d, want=("dx",))
    near = lambda y: abs(float(torch.tensor(y, dtype=torch.float64).to(dtype)) - y)  # noqa: E731
    bound = dloss * (near(2.0 ** 12 / v) * v / 2.0 ** 12 + near(1 - 1 / v) + 2.0 ** -18)
    assert float(dx[:, 0].double().abs().max()) <= bound * (1 + ref.U[dtype]) + ref.TINY[dtype]
