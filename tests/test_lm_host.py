"""The language-model products without a GPU: argument checks, and the reference formulas
against central differences."""
import pytest
import torch

import lm_reference as ref
import mixed_precision_tensor_gb300 as tcg

PA, PB, PD, PX = 0x10000, 0x20000, 0x30000, 0x40000
F16, BF16, F32, E4M3 = tcg.TCG_R_16F, tcg.TCG_R_16BF, tcg.TCG_R_32F, tcg.TCG_R_8F_E4M3
N, T = tcg.TCG_OP_N, tcg.TCG_OP_T
INV, NSUP, OK = (tcg.TCG_STATUS_INVALID_VALUE, tcg.TCG_STATUS_NOT_SUPPORTED, tcg.TCG_STATUS_SUCCESS)


@pytest.fixture(scope="module")
def handle():
    from mixed_precision_tensor_gb300 import _build
    _build.build()
    h = tcg.tcg_create()
    yield h
    assert tcg.tcg_destroy(h) == OK


def epi(**kw):
    return tcg.Epilogue(**kw)


def product(h, transa=T, transb=N, m=64, n=64, k=64, A=PA, lda=64, B=PB, ldb=64, at=BF16, D=PD, dt=BF16,
            ldd=64, e=None):
    return tcg.tcg_gemm_epilogue(h, transa, transb, m, n, k, 1.0, A, lda, B, ldb, at, D, dt, ldd, e)


@pytest.mark.parametrize("kw,status", [
    (dict(transa=2), INV), (dict(transb=-1), INV), (dict(m=-1), INV), (dict(n=-1), INV),
    (dict(k=-1), INV), (dict(at=9), INV), (dict(dt=9), INV),
    (dict(at=F32), NSUP), (dict(at=E4M3), NSUP), (dict(at=F16, dt=BF16), NSUP), (dict(dt=E4M3), NSUP),
    (dict(lda=56), INV), (dict(lda=68), INV), (dict(ldb=60), INV), (dict(ldd=60), INV),
    (dict(dt=F32, ldd=66), INV), (dict(transa=N, m=128, ldd=128), INV), (dict(transb=T, n=128), INV),
    (dict(A=None), INV), (dict(B=None), INV), (dict(D=None), INV), (dict(A=PA + 2), INV),
    (dict(D=PD + 8), INV), (dict(m=1 << 31, lda=64, ldd=1 << 31), NSUP), (dict(m=0), OK), (dict(n=0), OK),
    (dict(e=epi(activation=5)), INV), (dict(e=epi(activation=-1)), INV),
    (dict(e=epi(bias=PX, bias_type=7)), INV), (dict(e=epi(bias=PX, bias_type=F16)), NSUP),
    (dict(e=epi(bias=PX + 1, bias_type=BF16)), INV), (dict(e=epi(beta=1.0)), INV),
    (dict(e=epi(beta=1.0, C=PX, ldc=60)), INV), (dict(e=epi(beta=1.0, C=PX + 4, ldc=64)), INV),
    (dict(e=epi(Z=PX, ldz=63)), INV), (dict(e=epi(Z=PX + 8, ldz=64)), INV),
])
def test_epilogue_product_refuses(handle, kw, status):
    assert product(handle, **kw) == status


def test_null_handle():
    assert product(None) == INV
    assert tcg.tcg_xent_forward(None, 1, 8, 8, PA, 8, PB, 8, BF16, PX, -1, PD, PD) == INV


def grouped(h, m=64, n=64, k=64, groups=4, offsets=PX, lda=64, stride=4096, ldb=64, at=BF16, ldd=64, e=None):
    return tcg.tcg_gemm_grouped(h, T, m, n, k, groups, offsets, 1.0, PA, lda, stride, PB, ldb, at, PD, at,
                                ldd, e)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), INV), (dict(groups=385), NSUP), (dict(offsets=None), INV), (dict(offsets=PX + 4), INV),
    (dict(stride=0), INV), (dict(stride=4092), INV), (dict(lda=56), INV), (dict(at=F32), NSUP),
    (dict(n=0), OK), (dict(e=epi(activation=9)), INV),
])
def test_grouped_product_refuses(handle, kw, status):
    assert grouped(handle, **kw) == status


def grouped_k(h, m=64, n=64, k=64, groups=4, offsets=PX, lda=64, ldb=64, at=BF16, dt=BF16, ldd=64,
              stride=4096, D=PD):
    return tcg.tcg_gemm_grouped_k(h, m, n, k, groups, offsets, 1.0, PA, lda, PB, ldb, at, D, dt, ldd, stride)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), INV), (dict(groups=385), NSUP), (dict(offsets=None), INV), (dict(stride=4032), INV),
    (dict(stride=4100), INV), (dict(lda=56), INV), (dict(ldb=60), INV), (dict(ldd=60), INV),
    (dict(at=E4M3), NSUP), (dict(dt=F16), NSUP), (dict(D=None), INV), (dict(m=0), OK), (dict(k=-1), INV),
])
def test_grouped_weight_gradient_refuses(handle, kw, status):
    assert grouped_k(handle, **kw) == status


def backward(h, act=1, m=64, n=64, groups=1, offsets=None, dD=PA, lddd=64, Z=PB, ldz=64, ty=BF16, dZ=PD,
             lddz=64, dbias=PX):
    return tcg.tcg_epilogue_backward(h, act, m, n, groups, offsets, dD, lddd, Z, ldz, ty, dZ, lddz, dbias)


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), INV), (dict(ty=F32), NSUP), (dict(ty=8), INV), (dict(groups=2), INV), (dict(Z=None), INV),
    (dict(lddd=60), INV), (dict(ldz=56), INV), (dict(lddz=56), INV), (dict(dD=None), INV),
    (dict(dbias=PX + 2), INV), (dict(groups=0, offsets=PX), INV), (dict(groups=385, offsets=PX), NSUP),
    (dict(m=0), OK), (dict(dZ=None, dbias=None), OK),
])
def test_epilogue_gradient_refuses(handle, kw, status):
    assert backward(handle, **kw) == status


def layer_backward(h, act=1, m=64, n=64, k=64, groups=1, offsets=None, dD=PA, lddd=64, Z=PB, ldz=64, W=PD,
                   ldw=64, stride=4096, X=PA, ldx=64, ty=BF16, dX=PB, lddx=64, dW=PD, lddw=64, strided=4096,
                   dbias=PX):
    return tcg.tcg_linear_backward(h, act, m, n, k, groups, offsets, dD, lddd, Z, ldz, W, ldw, stride, X, ldx,
                                   ty, dX, lddx, dW, lddw, strided, dbias)


@pytest.mark.parametrize("kw,status", [
    (dict(act=-1), INV), (dict(act=5), INV), (dict(ty=F32), NSUP), (dict(ty=9), INV), (dict(m=-1), INV),
    (dict(n=-1), INV), (dict(k=-1), INV), (dict(k=(1 << 30) + 8, ldw=1 << 31, ldx=1 << 31, lddx=1 << 31,
                                               lddw=1 << 31), NSUP),
    (dict(groups=2), INV), (dict(groups=0, offsets=PX), INV), (dict(groups=385, offsets=PX), NSUP),
    (dict(groups=2, offsets=PX + 4), INV), (dict(groups=2, offsets=PX, stride=0), INV),
    (dict(groups=2, offsets=PX, stride=4100), INV), (dict(groups=2, offsets=PX, strided=4032), INV),
    (dict(groups=2, offsets=PX, strided=4100), INV), (dict(dD=None), INV), (dict(dD=PA + 4), INV),
    (dict(lddd=60), INV), (dict(Z=None), INV), (dict(ldz=56), INV), (dict(W=None), INV), (dict(W=PD + 8), INV),
    (dict(ldw=56), INV), (dict(X=None), INV), (dict(X=PA + 2), INV), (dict(ldx=60), INV),
    (dict(dX=PB + 4), INV), (dict(lddx=60), INV), (dict(dW=PD + 4), INV), (dict(lddw=56), INV),
    (dict(dbias=PX + 2), INV),
])
def test_layer_gradient_refuses(handle, kw, status):
    assert layer_backward(handle, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(vocab=0), INV), (dict(k=0), INV), (dict(ldx=56), INV), (dict(ldw=60), INV),
    (dict(ty=F32), NSUP), (dict(ty=7), INV), (dict(X=None), INV), (dict(W=PB + 4), INV),
    (dict(targets=None), INV), (dict(targets=PX + 4), INV), (dict(loss=None), INV), (dict(rows=0), OK),
])
def test_cross_entropy_refuses(handle, kw, status):
    a = dict(rows=4, vocab=100, k=64, X=PA, ldx=64, W=PB, ldw=64, ty=BF16, targets=PX, loss=PD, lse=PD)
    a.update(kw)
    assert tcg.tcg_xent_forward(handle, a["rows"], a["vocab"], a["k"], a["X"], a["ldx"], a["W"], a["ldw"],
                                a["ty"], a["targets"], -100, a["loss"], a["lse"]) == status
    if "loss" in kw or kw == dict(rows=0):
        return
    assert tcg.tcg_xent_backward(handle, a["rows"], a["vocab"], a["k"], a["X"], a["ldx"], a["W"], a["ldw"],
                                 a["ty"], a["targets"], -100, PD, PD, PA, 64, PB, 64) == status


def test_python_calls_refuse_what_the_library_cannot_see():
    """Shapes, types and places are checked before any pointer is taken."""
    h = object()
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tcg.linear(h, x, x)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        tcg.linear(h, x.float(), x)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        tcg.linear_cross_entropy(h, None, x, None)
    m = torch.zeros(4, 8, dtype=torch.bfloat16, device="meta")
    from mixed_precision_tensor_gb300 import lm
    for bad, kw in ((m[:, :4], "must be"), (m.float(), "bfloat16"), (m.t(), "must be")):
        with pytest.raises(ValueError, match=kw):
            lm._rows(bad, "w", 4, 8, torch.bfloat16, m.device)
    with pytest.raises(ValueError, match="16 bytes"):
        lm._rows(torch.zeros(4, 12, dtype=torch.bfloat16, device="meta")[:, :8], "w", 4, 8, torch.bfloat16,
                 m.device)
    with pytest.raises(ValueError, match="unit stride"):
        lm._rows(torch.zeros(8, 4, dtype=torch.bfloat16, device="meta").t(), "w", 4, 8, torch.bfloat16,
                 m.device)
    with pytest.raises(ValueError, match="act must be"):
        lm._act("swish")
    with pytest.raises(ValueError, match="want"):
        lm._want(("dx", "db"))


# ------------------------------------------------ the reference's gradients and differences
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_against_differences(name):
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.013
    h = 1e-6
    diff = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
    assert float((ref.slope(z, name) - diff).abs().max()) < 1e-8


def test_linear_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    t, n, k = 7, 5, 6
    x, w = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((t, k), (n, k)))
    b, d = torch.randn(n, generator=g, dtype=torch.float64), torch.randn(t, n, generator=g, dtype=torch.float64)

    def f(x, w, b):
        return float((ref.act(x @ w.t() + b, "gelu") * d).sum())

    z = x @ w.t() + b
    dz = d * ref.slope(z, "gelu")
    grads = (dz @ w, dz.t() @ x, dz.sum(0))
    for i, v in enumerate((x, w, b)):
        e = torch.randn(v.shape, generator=g, dtype=torch.float64)
        up, lo = [x, w, b], [x, w, b]
        up[i], lo[i] = v + 1e-6 * e, v - 1e-6 * e
        assert abs((f(*up) - f(*lo)) / 2e-6 - float((grads[i] * e).sum())) < 1e-6


def test_cross_entropy_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    t, v, k = 6, 11, 5
    x, w = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((t, k), (v, k)))
    target, c = torch.tensor([0, 10, -100, 4, 11, 5]), torch.randn(t, generator=g, dtype=torch.float64)

    def f(x, w):
        return float((ref.xent(x, w, target, -100)[0] * c).sum())

    logits = x @ w.t()
    counts = (target >= 0) & (target < v)
    hot = torch.zeros(t, v, dtype=torch.float64)
    hot[counts, target[counts]] = 1.0
    G = torch.where(counts, c, torch.zeros_like(c))[:, None] * (torch.softmax(logits, 1) - hot)
    for i, grad in enumerate((G @ w, G.t() @ x)):
        e = torch.randn((x, w)[i].shape, generator=g, dtype=torch.float64)
        up, lo = [x, w], [x, w]
        up[i], lo[i] = up[i] + 1e-6 * e, lo[i] - 1e-6 * e
        assert abs((f(*up) - f(*lo)) / 2e-6 - float((grad * e).sum())) < 1e-6
