"""The norm, the gated projections and the 4-bit products without a GPU: argument checks of the
library and of the Python calls, and the reference's gradients against differences."""
import pytest
import torch

import ffn_reference as ref
import mixed_precision_tensor_gb300 as tcg
from mixed_precision_tensor_gb300 import ffn, lm

PA, PB, PD, PX, PW = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
F16, BF16, F32, E4M3 = tcg.TCG_R_16F, tcg.TCG_R_16BF, tcg.TCG_R_32F, tcg.TCG_R_8F_E4M3
INV, NSUP, OK = (tcg.TCG_STATUS_INVALID_VALUE, tcg.TCG_STATUS_NOT_SUPPORTED, tcg.TCG_STATUS_SUCCESS)


@pytest.fixture(scope="module")
def handle():
    from mixed_precision_tensor_gb300 import _build
    _build.build()
    h = tcg.tcg_create()
    yield h
    assert tcg.tcg_destroy(h) == OK


# --------------------------------------------------------------------------- the library
def norm(h, rows=4, k=64, X=PA, ldx=64, R=None, ldr=64, S=None, lds=64, W=PW, wt=BF16, eps=1e-6, t=BF16, Y=PD,
         yt=BF16, ldy=64, scale=None):
    return tcg.tcg_rms_norm(h, rows, k, X, ldx, R, ldr, S, lds, W, wt, eps, t, Y, yt, ldy, scale)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(k=0), INV), (dict(k=-8), INV), (dict(t=9), INV), (dict(wt=9), INV), (dict(yt=-1), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(t=F32), NSUP), (dict(t=E4M3), NSUP), (dict(wt=F16), NSUP),
    (dict(yt=F32), NSUP), (dict(yt=F16), NSUP), (dict(k=32769, ldx=32776, ldy=32776), NSUP), (dict(ldx=56), INV),
    (dict(ldx=68), INV), (dict(ldy=56), INV), (dict(R=PB, ldr=60), INV), (dict(R=PB + 2), INV), (dict(S=PB, lds=63), INV),
    (dict(S=PB + 8), INV), (dict(X=None), INV), (dict(X=PA + 8), INV), (dict(Y=None), INV), (dict(Y=PD + 8), INV),
    (dict(W=None), INV), (dict(W=PW + 4), INV), (dict(yt=E4M3), INV), (dict(yt=E4M3, scale=PX + 2), INV),
    (dict(yt=E4M3, scale=PX, ldy=72), INV), (dict(rows=0), OK), (dict(rows=0, X=None, Y=None, W=None), OK),
])
def test_norm_refuses(handle, kw, status):
    assert norm(handle, **kw) == status
    assert norm(None, **kw) == INV


def norm_backward(h, rows=4, k=64, dY=PA, lddy=64, X=PB, ldx=64, dS=None, ldds=64, W=PW, wt=BF16, eps=1e-6, t=BF16,
                  dX=PD, lddx=64, dW=PX):
    return tcg.tcg_rms_norm_backward(h, rows, k, dY, lddy, X, ldx, dS, ldds, W, wt, eps, t, dX, lddx, dW)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INV), (dict(k=0), INV), (dict(t=9), INV), (dict(t=F32), NSUP), (dict(wt=F16), NSUP),
    (dict(eps=-0.5), INV), (dict(k=40000, lddy=40000, ldx=40000, lddx=40000), NSUP), (dict(lddy=56), INV),
    (dict(ldx=60), INV), (dict(dS=PX, ldds=63), INV), (dict(dS=PX + 2), INV), (dict(lddx=56), INV), (dict(dX=PD + 8), INV),
    (dict(dW=PX + 2), INV), (dict(dY=None), INV), (dict(X=None), INV), (dict(W=None), INV), (dict(W=PW + 8), INV),
    (dict(dX=None, dW=None), OK), (dict(rows=0, dW=None), OK),
])
def test_norm_backward_refuses(handle, kw, status):
    assert norm_backward(handle, **kw) == status
    assert norm_backward(None, **kw) == INV


def gated(h, act=4, m=64, n=8, k=64, A=PA, lda=64, B=PB, ldb=64, at=BF16, D=PD, dt=BF16, ldd=64, Z=None, ldz=128):
    return tcg.tcg_gemm_gated(h, act, m, n, k, A, lda, B, ldb, at, D, dt, ldd, Z, ldz)


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), INV), (dict(act=-1), INV), (dict(m=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV), (dict(at=9), INV),
    (dict(dt=9), INV), (dict(at=F32), NSUP), (dict(at=E4M3), NSUP), (dict(at=F16, dt=BF16), NSUP), (dict(dt=E4M3), NSUP),
    (dict(lda=56), INV), (dict(lda=68), INV), (dict(ldb=60), INV), (dict(ldd=60), INV), (dict(dt=F32, ldd=66), INV),
    (dict(Z=PX, ldz=120), INV), (dict(Z=PX + 8), INV), (dict(A=None), INV), (dict(A=PA + 2), INV), (dict(B=None), INV),
    (dict(D=None), INV), (dict(D=PD + 8), INV), (dict(m=1 << 30, ldd=1 << 30), NSUP), (dict(m=0), OK), (dict(n=0), OK),
])
def test_gated_product_refuses(handle, kw, status):
    assert gated(handle, **kw) == status
    assert gated(None, **kw) == INV


def gated_backward(h, act=4, m=64, n=8, k=64, dD=PA, lddd=64, Z=PB, ldz=128, W=PW, ldw=64, X=PX, ldx=64, t=BF16,
                   dX=PD, lddx=64, dW=PD + 0x100000, lddw=64):
    return tcg.tcg_gated_backward(h, act, m, n, k, dD, lddd, Z, ldz, W, ldw, X, ldx, t, dX, lddx, dW, lddw)


@pytest.mark.parametrize("kw,status", [
    (dict(act=5), INV), (dict(m=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV), (dict(t=9), INV), (dict(t=F32), NSUP),
    (dict(lddd=56), INV), (dict(ldz=120), INV), (dict(ldw=60), INV), (dict(ldx=60), INV), (dict(lddx=56), INV),
    (dict(lddw=56), INV), (dict(dD=None), INV), (dict(Z=None), INV), (dict(W=None), INV), (dict(X=None), INV),
    (dict(dD=PA + 2), INV), (dict(Z=PB + 8), INV), (dict(dX=PD + 2), INV), (dict(dX=None, dW=None), OK),
    (dict(n=0, dW=None), OK), (dict(m=0, dX=None), OK), (dict(m=1 << 30, lddd=1 << 30, ldz=1 << 31), NSUP),
])
def test_gated_gradient_refuses(handle, kw, status):
    assert gated_backward(handle, **kw) == status
    assert gated_backward(None, **kw) == INV


def packed(h, m=64, n=8, k=64, group=32, A=PA, lda=32, scales=PX, zeros=None, st=BF16, B=PB, ldb=64, bt=BF16, D=PD,
           dt=BF16, ldd=64, gate=0, e=None):
    return tcg.tcg_gemm_4bit(h, m, n, k, group, A, lda, scales, zeros, st, B, ldb, bt, D, dt, ldd, gate, e)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV), (dict(st=9), INV), (dict(bt=9), INV), (dict(dt=9), INV),
    (dict(bt=F32), NSUP), (dict(bt=E4M3), NSUP), (dict(dt=F16), NSUP), (dict(st=F16), NSUP), (dict(st=E4M3), NSUP),
    (dict(group=16), NSUP), (dict(group=0), NSUP), (dict(group=256), NSUP), (dict(lda=24), INV), (dict(lda=40), INV),
    (dict(k=65, ldb=72), INV), (dict(ldb=56), INV), (dict(ldd=56), INV), (dict(A=None), INV), (dict(A=PA + 8), INV),
    (dict(B=None), INV), (dict(B=PB + 2), INV), (dict(D=None), INV), (dict(D=PD + 8), INV), (dict(scales=None), INV),
    (dict(scales=PX + 1), INV), (dict(zeros=PX + 1), INV), (dict(st=F32, scales=PX + 2), INV),
    (dict(e=tcg.Epilogue(Z=PX, ldz=64)), NSUP), (dict(e=tcg.Epilogue(activation=7)), INV),
    (dict(e=tcg.Epilogue(beta=1.0)), INV), (dict(gate=1, e=tcg.Epilogue(bias=PX, bias_type=F32)), NSUP),
    (dict(gate=1, e=tcg.Epilogue(beta=1.0, C=PX, ldc=64)), NSUP), (dict(m=0), OK), (dict(n=0), OK),
])
def test_packed_product_refuses(handle, kw, status):
    assert packed(handle, **kw) == status
    assert packed(None, **kw) == INV


def test_workspace_queries_refuse(handle):
    import ctypes
    size = ctypes.c_size_t(0)
    lib = tcg.load_library()
    assert lib.tcg_gemm_gated_workspace_size(handle, -1, 1, 1, size) == INV
    assert lib.tcg_gemm_gated_workspace_size(handle, 1, 1, 1, None) == INV
    assert lib.tcg_gated_backward_workspace_size(handle, 1, -1, 1, 1, 1, size) == INV
    assert lib.tcg_rms_norm_backward_workspace_size(handle, 1, 0, size) == INV
    assert lib.tcg_rms_norm_backward_workspace_size(handle, 1, 40000, size) == NSUP
    assert lib.tcg_gemm_4bit_workspace_size(handle, 1, 1, -1, 0, size) == INV
    assert lib.tcg_gemm_4bit_workspace_size(handle, 1, 1, 8, 0, None) == INV
    for m, n, k, gate in ((4096, 48, 65536, 0), (4096, 64, 4096, 0), (65536, 128, 4096, 1), (512, 128, 4096, 0), (256, 256, 4096, 1)):
        assert lib.tcg_gemm_4bit_workspace_size(handle, m, n, k, gate, size) == OK and size.value == 0


# ------------------------------------------------------------------------- the Python calls
class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


class Handle:
    h, stream = None, None


@pytest.fixture
def library(monkeypatch):
    """A stand-in that notes its arguments, with CPU tensors taken for the GPU's."""
    made = Library()
    monkeypatch.setattr(ffn, "_lib", lambda: made)
    monkeypatch.setattr(ffn, "_input", lambda x, what="x": (*x.shape, x.dtype, x.device))
    return made


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_cpu_tensors_are_refused():
    x, w = zeros(4, 64), zeros(64)
    for call in (lambda: tcg.rms_norm(None, x, w), lambda: tcg.rms_norm_8bit(None, x, w),
                 lambda: tcg.rms_norm_backward(None, x, x, w), lambda: tcg.gated_linear(None, x, zeros(16, 64)),
                 lambda: tcg.gated_linear_backward(None, zeros(4, 8), x, zeros(16, 64), zeros(4, 16)),
                 lambda: tcg.linear_4bit(None, x, zeros(8, 32, dtype=torch.uint8), zeros(8, 2), 32)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("kw,what", [
    (dict(weight=zeros(63)), "weight"), (dict(weight=zeros(64, dtype=torch.float16)), "weight"),
    (dict(weight=zeros(128)[::2]), "weight"), (dict(eps=-1e-6), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(residual=zeros(3, 64)), "residual"), (dict(residual=zeros(4, 64).half()), "residual"),
    (dict(sum_out=zeros(4, 65)[:, :64]), "sum_out"), (dict(out=zeros(4, 64).half()), "out"), (dict(out=zeros(4, 72)), "out"),
])
def test_norm_arguments(library, kw, what):
    args = dict(weight=zeros(64)) | kw
    with pytest.raises(ValueError, match=what):
        tcg.rms_norm(Handle(), zeros(4, 64), args.pop("weight"), **args)
    assert not library.calls


def test_norm_8bit_arguments(library):
    x, w = zeros(4, 40), zeros(40)
    for kw, what in ((dict(out=zeros(4, 40)), "out"), (dict(scale=zeros(4)), "scale"), (dict(scale=zeros(5).float()), "scale"),
                     (dict(out=torch.zeros(4, 40).to(torch.float8_e4m3fn)), "16 bytes")):
        with pytest.raises(ValueError, match=what):
            tcg.rms_norm_8bit(Handle(), x, w, **kw)
    assert not library.calls
    out, scale = tcg.rms_norm_8bit(Handle(), x, w)
    assert out.shape == (4, 40) and out.stride(0) == 48 and scale.dtype is torch.float32
    (name, a), = library.calls
    assert name == "tcg_rms_norm" and a[1:3] == (4, 40) and a[14:16] == (E4M3, 48)


def test_backward_arguments(library):
    x, w = zeros(4, 64), zeros(64)
    for kw, what in ((dict(dout=zeros(4, 63)), "dout"), (dict(want=("dbias",)), "want"), (dict(dw=zeros(64)), "dw"),
                     (dict(dsum=zeros(5, 64)), "dsum"), (dict(dx=zeros(4, 64).half()), "dx")):
        args = dict(dout=zeros(4, 64)) | kw
        with pytest.raises(ValueError, match=what):
            tcg.rms_norm_backward(Handle(), args.pop("dout"), x, w, **args)
    gw, z, d = zeros(16, 64), zeros(4, 16), zeros(4, 8)
    for args, what in (((zeros(4, 9), x, gw, z), "dout"), ((d, x, zeros(15, 64), z), "even"), ((d, x, gw, zeros(4, 15)), "z"),
                       ((d, x, zeros(16, 56), z), "w must")):
        with pytest.raises(ValueError, match=what):
            tcg.gated_linear_backward(Handle(), *args)
    with pytest.raises(ValueError, match="want"):
        tcg.gated_linear_backward(Handle(), d, x, gw, z, want=("dbias",))
    with pytest.raises(ValueError, match="act"):
        tcg.gated_linear_backward(Handle(), d, x, gw, z, act="swish")
    assert not library.calls


def test_gated_arguments(library):
    x = zeros(4, 64)
    for args, kw, what in (((zeros(15, 64),), {}, "even"), ((zeros(2, 8, 64),), {}, "even"), ((zeros(16, 72),), {}, "w must"),
                           ((zeros(16, 64),), dict(z=zeros(4, 8)), "z"), ((zeros(16, 64),), dict(out=zeros(4, 16)), "out"),
                           ((zeros(16, 64),), dict(out_dtype=torch.float16), "output")):
        with pytest.raises(ValueError, match=what):
            tcg.gated_linear(Handle(), x, *args, **kw)
    assert not library.calls


def test_4bit_arguments(library):
    x, w, s = zeros(4, 64), zeros(8, 32, dtype=torch.uint8), zeros(8, 2)
    for args, kw, what in (((w, s, 48), {}, "group"), ((w, s, 64), {}, "scales"), ((w.char(), s, 32), {}, "w must"),
                           ((zeros(8, 31, dtype=torch.uint8), s, 32), {}, "w must"), ((w, s.half(), 32), {}, "scales"),
                           ((w, s, 32), dict(zeros=s.float()), "zeros"), ((w, s, 32), dict(bias=zeros(9)), "bias"),
                           ((zeros(7, 32, dtype=torch.uint8), zeros(7, 2), 32), dict(gated=True), "even"),
                           ((w, s, 32), dict(gated=True, bias=zeros(4)), "gated"),
                           ((w, s, 32), dict(gated=True, residual=zeros(4, 4)), "gated"), ((None, s, 32), {}, "w must"),
                           ((w, s, 32), dict(residual=zeros(4, 7)), "residual"), ((w, s, 32), dict(act="swish"), "act")):
        with pytest.raises(ValueError, match=what):
            tcg.linear_4bit(Handle(), x, *args, **kw)
    assert not library.calls


def test_rows_that_are_held(library, monkeypatch):
    """Tensors of another stream than the caller's are recorded there, all that a call touches."""
    held = []
    monkeypatch.setattr(ffn, "_elsewhere", lambda handle, device: True)
    monkeypatch.setattr(ffn, "_hold", lambda handle, *t: held.append([a for a in t if a is not None]))
    x, r, k, w, o = zeros(4, 64), zeros(4, 64), zeros(4, 64), zeros(64), zeros(4, 64)
    tcg.rms_norm(Handle(), x, w, residual=r, sum_out=k, out=o)
    assert all(any(a is b for b in held[-1]) for a in (x, r, k, w, o))
    gw, z = zeros(16, 64), zeros(4, 16)
    out = tcg.gated_linear(Handle(), x, gw, z=z, out=zeros(4, 8))
    assert all(any(a is b for b in held[-1]) for a in (x, gw, z, out))
    q, s, b = zeros(8, 32, dtype=torch.uint8), zeros(8, 2), zeros(8)
    out = tcg.linear_4bit(Handle(), x, q, s, 32, zeros=s, bias=b, residual=zeros(4, 8), out=zeros(4, 8))
    assert all(any(a is b_ for b_ in held[-1]) for a in (x, q, s, b, out))


# ------------------------------------------------------------------- the reference itself
def central(f, x, step=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).flatten()
        e[i] = step
        e = e.view_as(x)
        g.view(-1)[i] = (f(x + e) - f(x - e)) / (2 * step)
    return g


def test_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(0)
    x, w, d, ds = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 5), (5,), (3, 5), (3, 5)))
    x, w, d, ds = (v.to(torch.bfloat16) for v in (x, w, d, ds))
    (dx, dw), _ = ref.norm_backward(d, x, w, 1e-5, ds)

    def loss(xx, ww):
        y = xx / torch.sqrt(xx.square().mean(1, keepdim=True) + 1e-5) * ww
        return (y * d.double()).sum() + (xx * ds.double()).sum()
    assert torch.allclose(dx, central(lambda v: loss(v, w.double()), x.double()), atol=1e-7)
    assert torch.allclose(dw, central(lambda v: loss(x.double(), v), w.double()), atol=1e-7)


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
def test_gated_gradient_against_differences(name):
    g = torch.Generator().manual_seed(1)
    x, w, d = (torch.randn(*s, generator=g).to(torch.bfloat16) for s in ((3, 4), (6, 4), (3, 3)))
    z = x.double() @ w.double().t()
    (dx, dw), _ = ref.gated_backward(d, x, w, z, name)

    def loss(xx, ww):
        zz = xx @ ww.t()
        return (ref.act(zz[:, :3], name) * zz[:, 3:] * d.double()).sum()
    assert torch.allclose(dx, central(lambda v: loss(v, w.double()), x.double()), atol=1e-6)
    assert torch.allclose(dw, central(lambda v: loss(x.double(), v), w.double()), atol=1e-6)


def test_packing_of_the_documentation():
    """The expression in linear_4bit's text gives weights within half a scale of the originals."""
    g = torch.Generator().manual_seed(2)
    v, group = torch.randn(6, 128, generator=g), 32
    s = v.unflatten(1, (-1, group)).abs().amax(2) / 7
    q = (v.unflatten(1, (-1, group)) / s[..., None]).round().add(8).clamp(1, 15).flatten(1).byte()
    w = q[:, 0::2] | q[:, 1::2] << 4
    assert torch.equal(ref.unpack(w, 128), q) and torch.equal(ref.pack(q), w)
    W, _ = ref.weights_4bit(w, 128, s, None, group)
    assert ((W - v.double()).abs() <= 0.5 * s.double().repeat_interleave(group, 1) * (1 + 1e-5)).all()
