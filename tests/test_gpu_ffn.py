"""The norm, the gated projections and the 4-bit products on the GPU against FP64
(ffn_reference), at the sizes, masks and layouts where they can go wrong."""
import pytest
import torch

import ffn_reference as ref
import mixed_precision_tensor_gb300 as tcg
from lm_reference import TINY, U, within
from test_gpu_lm import gen_of, padded, randn, same_bits

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = tcg.Handle()
    yield h
    tcg.check(tcg.tcg_get_device_error(h.h), "device error word")
    h.close()


def untouched(buf, cols):
    """Nothing between the rows of a padded() buffer was written."""
    full = torch.as_strided(buf, (buf.shape[0], buf.stride(0)), (buf.stride(0), 1))
    return torch.isnan(full[:, cols:].float()).all()


# -------------------------------------------------------------------------------- norm
NORM_SIZES = [(1, 1), (1, 7), (3, 8), (9, 64), (1, 256), (700, 255), (20, 257), (8, 512), (33, 513), (1, 4096),
              (5, 1000), (300, 4096), (2000, 72), (777, 2055), (3, 16384), (4, 16392), (2, 32768), (1, 32761),
              (20000, 8), (2500, 520)]


@pytest.mark.parametrize("t,k", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_norm_forward(handle, t, k, dtype):
    g = gen_of(t * 13 + k)
    x = padded(randn(g, t, k, dtype=dtype))
    res = padded(randn(g, t, k, dtype=dtype)) if (t + k) % 3 else None
    weight = randn(g, k, dtype=F32 if k % 2 else dtype)
    kept = padded(torch.zeros_like(x)) if k % 4 else None
    out = padded(torch.zeros_like(x))
    assert tcg.rms_norm(handle, x, weight, eps=1e-5, residual=res, sum_out=kept, out=out) is out
    y, ey, s, es = ref.norm(x, weight, 1e-5, res, dtype)
    within(out, y, ey + U[dtype] * (y.abs() + ey) + TINY[dtype], "out")
    assert untouched(out, k)
    if kept is not None:
        within(kept, s, es, "sum")
        assert untouched(kept, k)


@pytest.mark.parametrize("t,k", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_norm_8bit(handle, t, k, dtype):
    g = gen_of(t * 17 + k)
    x = padded(randn(g, t, k, dtype=dtype))
    if t > 2:
        x[1] = 0.0
        x[2] *= 30.0
    weight = randn(g, k, dtype=dtype if k % 2 else F32)
    res = padded(randn(g, t, k, dtype=dtype, std=0.0 if t > 2 else 1.0)) if k % 3 else None
    out = padded(torch.zeros(t, k, device="cuda").to(E4M3), 16) if k % 5 else None
    out, scale = tcg.rms_norm_8bit(handle, x, weight, eps=1e-5, residual=res, out=out)
    assert out.dtype is E4M3 and out.shape == (t, k) and scale.shape == (t,) and out.stride(0) % 16 == 0
    y, ey, _, _ = ref.norm(x, weight, 1e-5, res, dtype)
    want, bound = ref.norm_8bit(y)
    within(scale, want, bound, "scale")
    stands = out.double() * scale.double()[:, None]
    within(stands, y, (2.0 ** -4 + 2.0 ** -20) * (y.abs() + ey) + 2.0 ** -10 * scale.double()[:, None] + ey, "out")
    if k % 5:
        assert untouched(out, k)


@pytest.mark.parametrize("t,k", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_norm_backward(handle, t, k, dtype):
    g = gen_of(t * 19 + k)
    x, dout = padded(randn(g, t, k, dtype=dtype)), padded(randn(g, t, k, dtype=dtype, std=0.5))
    dsum = padded(randn(g, t, k, dtype=dtype)) if (t + k) % 2 else None
    weight = randn(g, k, dtype=F32 if t % 2 else dtype)
    dx = padded(torch.zeros_like(x))
    got = tcg.rms_norm_backward(handle, dout, x, weight, eps=1e-5, dsum=dsum, dx=dx)
    assert got[0] is dx and got[1].dtype is F32
    want, bound = ref.norm_backward(dout, x, weight, 1e-5, dsum)
    within(dx, want[0], bound[0], "dx")
    within(got[1], want[1], bound[1], "dw")
    assert untouched(dx, k)
    alone = tcg.rms_norm_backward(handle, dout, x, weight, eps=1e-5, dsum=dsum, want=("dx",))
    assert alone[1] is None and same_bits(alone[0], dx)
    alone = tcg.rms_norm_backward(handle, dout, x, weight, eps=1e-5, dsum=dsum, want=("dw",))
    assert alone[0] is None and same_bits(alone[1], got[1])


@pytest.mark.parametrize("t,k", [(1, 264), (40, 4096), (1000, 72)])
def test_norm_in_place(handle, t, k):
    g = gen_of(k)
    x, res, weight = randn(g, t, k), randn(g, t, k), randn(g, k)
    kept = torch.empty_like(x)
    out = tcg.rms_norm(handle, x, weight, residual=res, sum_out=kept)
    for into in ("residual", "x"):
        a, b = x.clone(), res.clone()
        got = tcg.rms_norm(handle, a, weight, residual=b, sum_out=b if into == "residual" else a,
                           out=a if into == "residual" else b)
        assert same_bits(got, out) and same_bits(b if into == "residual" else a, kept)
    dout = randn(g, t, k)
    want = tcg.rms_norm_backward(handle, dout, x, weight, dsum=res)
    for into in ("dout", "dsum"):
        a, b = dout.clone(), res.clone()
        got = tcg.rms_norm_backward(handle, a, x, weight, dsum=b, dx=a if into == "dout" else b)
        assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])


@pytest.mark.parametrize("k", [200, 4104])
def test_norm_rows_without_a_number(handle, k):
    """NaN and infinities stay in their rows, zero rows come out zero."""
    g = gen_of(2)
    x, weight = randn(g, 6, k), randn(g, k)
    x[0, 3], x[2, 5], x[4] = float("nan"), float("inf"), 0.0
    out = tcg.rms_norm(handle, x, weight)
    q, scale = tcg.rms_norm_8bit(handle, x, weight)
    y = ref.norm(x, weight, 1e-6, None, BF16)[0]
    assert torch.isnan(out[0]).all() and torch.isnan(out[2, 5])
    assert (out[2, :5] == 0).all() and (out[2, 6:] == 0).all()
    assert torch.isnan(scale[[0, 2]]).all() and torch.isnan(q[[0, 2]].float()).all()
    assert (out[4] == 0).all() and (q[4].float() == 0).all() and scale[4] == 2.0 ** -100
    for i in (1, 3, 5):
        within(out[i], y[i], (U[BF16] + 2 * ref.NORM) * y[i].abs() + TINY[BF16])
        assert torch.isfinite(scale[i])


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e15])
def test_norm_of_small_and_large_rows(handle, size):
    g = gen_of(4)
    x = randn(g, 5, 1000, dtype=F32).mul(size).to(BF16)
    weight = randn(g, 1000)
    eps = 1e-5 if size < 1e-20 else 0.0
    out, scale = tcg.rms_norm_8bit(handle, x, weight, eps=eps)
    y = ref.norm(x, weight, eps, None, BF16)[0]
    within(scale, *ref.norm_8bit(y))
    within(out.double() * scale.double()[:, None], y,
           (2.0 ** -4 + 2 * ref.NORM) * y.abs() + 2.0 ** -10 * scale.double()[:, None])


def test_norm_refuses_a_weight_between_places(handle):
    x, room = torch.ones(3, 64, dtype=BF16, device="cuda"), torch.ones(65, dtype=BF16, device="cuda")
    for call in (tcg.rms_norm, tcg.rms_norm_8bit, lambda h, a, w: tcg.rms_norm_backward(h, a, a, w)):
        with pytest.raises(tcg.TcgError):
            call(handle, x, room[1:])


def test_norm_without_rows(handle):
    x, weight = torch.empty(0, 40, dtype=BF16, device="cuda"), torch.ones(40, dtype=BF16, device="cuda")
    assert tcg.rms_norm(handle, x, weight).shape == (0, 40)
    q, scale = tcg.rms_norm_8bit(handle, x, weight)
    assert q.shape == (0, 40) and scale.shape == (0,)
    dw = torch.full((40,), 3.0, device="cuda")
    dx, got = tcg.rms_norm_backward(handle, x, x, weight, dw=dw)
    assert dx.shape == (0, 40) and got is dw and (dw == 0).all()


# ------------------------------------------------------------------------------- gated
GATED_SIZES = [(1, 8, 8), (1, 4096, 1024), (2, 301, 523), (4, 1000, 264), (3, 5, 13), (5, 40, 300), (17, 300, 1000),
               (33, 256, 64), (64, 1000, 1032), (100, 520, 200), (100, 72, 4096), (129, 2056, 264), (257, 513, 127),
               (300, 77, 2048), (700, 1288, 320), (200, 1000, 4096), (2000, 2048, 256), (5, 256, 20000),
               (1, 17, 8200), (1500, 250, 8192), (24, 4096, 4096), (40, 16, 72), (1, 100, 7), (600, 130, 640)]


@pytest.mark.parametrize("t,n,k", GATED_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated_forward(handle, t, n, k, dtype):
    g = gen_of(t * 31 + n * 7 + k)
    act = ACTS[(t + n + k) % 5]
    out_dtype = F32 if (t + k) % 3 == 0 else dtype
    x, w = padded(randn(g, t, k, dtype=dtype)), padded(randn(g, 2 * n, k, dtype=dtype, std=k ** -0.5))
    z = padded(torch.zeros(t, 2 * n, dtype=dtype, device="cuda"))
    out = padded(torch.zeros(t, n, dtype=out_dtype, device="cuda"))
    assert tcg.gated_linear(handle, x, w, act=act, out=out, z=z) is out
    tcg.check(tcg.tcg_get_device_error(handle.h))
    want, eo, zw, ez = ref.gated(x, w, act, out_dtype)
    within(out, want, eo, "out")
    within(z, zw, ez + U[dtype] * (zw.abs() + ez) + TINY[dtype], "z")
    assert untouched(out, n) and untouched(z, 2 * n)
    assert same_bits(tcg.gated_linear(handle, x, w, act=act, out_dtype=out_dtype), out)


@pytest.mark.parametrize("t,n,k", GATED_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated_backward(handle, t, n, k, dtype):
    g = gen_of(t * 37 + n * 7 + k)
    act = ACTS[(t + n) % 5]
    x, w = padded(randn(g, t, k, dtype=dtype)), padded(randn(g, 2 * n, k, dtype=dtype, std=k ** -0.5))
    z, dout = padded(randn(g, t, 2 * n, dtype=dtype)), padded(randn(g, t, n, dtype=dtype))
    dx, dw = padded(torch.zeros_like(x)), padded(torch.zeros_like(w))
    got = tcg.gated_linear_backward(handle, dout, x, w, z, act=act, dx=dx, dw=dw)
    assert got[0] is dx and got[1] is dw
    tcg.check(tcg.tcg_get_device_error(handle.h))
    want, bound = ref.gated_backward(dout, x, w, z, act)
    within(dx, want[0], bound[0], "dx")
    within(dw, want[1], bound[1], "dw")
    assert untouched(dx, k) and untouched(dw, k)
    alone = tcg.gated_linear_backward(handle, dout, x, w, z, act=act, want=("dw",))
    assert alone[0] is None and same_bits(alone[1], dw)


@pytest.mark.parametrize("t,n,k", [(0, 16, 8), (3, 0, 8), (3, 16, 0), (70, 24, 0), (300, 24, 0)])
def test_gated_without_elements(handle, t, n, k):
    x = torch.empty(t, max(k, 8), dtype=BF16, device="cuda")[:, :k]
    w = torch.empty(2 * n, max(k, 8), dtype=BF16, device="cuda")[:, :k]
    z = torch.full((t, max(2 * n, 8)), float("nan"), dtype=BF16, device="cuda")[:, :2 * n]
    out = tcg.gated_linear(handle, x, w, z=z)
    assert out.shape == (t, n) and (out == 0).all() and (z == 0).all()
    dx, dw = tcg.gated_linear_backward(handle, torch.zeros(t, max(n, 8), dtype=BF16, device="cuda")[:, :n], x, w,
                                       z)
    assert dx.shape == (t, k) and dw.shape == (2 * n, k) and (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("t", [1, 40, 300])
def test_gated_keeps_rows_apart(handle, t):
    """A token with NaN changes no other token."""
    g = gen_of(8)
    x, w = randn(g, t + 1, 320), randn(g, 2 * 264, 320, std=0.05)
    want = tcg.gated_linear(handle, x, w)
    x[t // 2] = float("nan")
    got = tcg.gated_linear(handle, x, w)
    assert torch.isnan(got[t // 2]).all()
    rest = [i for i in range(t + 1) if i != t // 2]
    assert same_bits(got[rest], want[rest])


# ------------------------------------------------------------------------------- 4 bits
W4_SIZES = [(1, 32, 128), (1, 8, 32), (1, 4096, 4096), (2, 100, 31), (3, 33, 257), (4, 1000, 1000), (8, 40, 5000), (9, 64, 40),
            (16, 300, 2048), (17, 512, 384), (32, 77, 100), (33, 200, 777), (64, 1000, 1032), (65, 136, 200),
            (100, 512, 1024), (300, 1000, 520), (7, 6, 16384), (1, 3, 20000), (1, 1, 1), (5, 2, 33), (130, 40, 36), (128, 200, 1000),
            (48, 4128, 4104), (64, 2000, 8300), (129, 1100, 1064), (256, 100, 520), (300, 2200, 1032)]


def draw_4bit(g, rows, k, group, dtype, zeros, apart=True):
    q = torch.randint(0, 16, (rows, k), generator=g, device="cuda", dtype=torch.uint8)
    w = ref.pack(q)
    half = w.shape[1]
    ld = -(-half // 16) * 16 + (16 if apart else 0)
    big = torch.full((rows, ld), 255, dtype=torch.uint8, device="cuda")
    big[:, :half] = w
    size = (rows, -(-k // group))
    scales = ((0.5 + torch.rand(size, generator=g, device="cuda")) / (4.6 * k ** 0.5)).to(dtype)
    zero = (torch.randn(size, generator=g, device="cuda") * 3 + 8).to(dtype) if zeros else None
    return big[:, :half], scales, zero


@pytest.mark.parametrize("t,n,k", W4_SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_4bit(handle, t, n, k, group, dtype):
    g = gen_of(t * 31 + n * 7 + k + group)
    act = ACTS[(t + n + k) % 5]
    out_dtype = F32 if (t + k) % 3 == 0 else dtype
    x = padded(randn(g, t, k, dtype=dtype))
    w, scales, zeros = draw_4bit(g, n, k, group, F32 if n % 2 else dtype, (t + group // 32) % 2)
    bias = randn(g, n, dtype=dtype if n % 2 else F32) if k % 2 else None
    res = padded(randn(g, t, n, dtype=out_dtype)) if n % 4 else None
    out = padded(torch.zeros(t, n, dtype=out_dtype, device="cuda"))
    assert tcg.linear_4bit(handle, x, w, scales, group, zeros=zeros, bias=bias, act=act, residual=res, beta=0.5,
                           out=out) is out
    want, bound = ref.linear_4bit(x, w, scales, zeros, group, bias, act, res, 0.5, False, out_dtype)
    within(out, want, bound, "out")
    assert untouched(out, n)


@pytest.mark.parametrize("t,n,k", W4_SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gated_4bit(handle, t, n, k, dtype):
    g = gen_of(t * 41 + n * 7 + k)
    group = (32, 64, 128)[(n + k) % 3]
    act = ACTS[(t + k) % 5]
    out_dtype = F32 if (t + n) % 3 == 0 else dtype
    x = padded(randn(g, t, k, dtype=dtype))
    w, scales, zeros = draw_4bit(g, 2 * n, k, group, dtype, n % 2)
    out = padded(torch.zeros(t, n, dtype=out_dtype, device="cuda"))
    tcg.linear_4bit(handle, x, w, scales, group, zeros=zeros, act=act, gated=True, out=out)
    want, bound = ref.linear_4bit(x, w, scales, zeros, group, None, act, None, 0.0, True, out_dtype)
    within(out, want, bound, "out")
    assert untouched(out, n)


def test_4bit_every_weight_at_every_place(handle):
    """Products with one-hot rows of x give the weights themselves, exactly: 16 values at 256 places."""
    k = 256
    q = ((torch.arange(k, device="cuda")[None] + torch.arange(16, device="cuda")[:, None]) % 16).to(torch.uint8)
    ones = torch.ones(16, k // 32, device="cuda")
    for dtype in (BF16, F16):
        for t in (8, 32, 64, 256):
            for first in range(0, k, t):
                x = torch.zeros(t, k, dtype=dtype, device="cuda")
                x[torch.arange(t), first + torch.arange(t)] = 1.0
                out = tcg.linear_4bit(handle, x, ref.pack(q), ones, 32, out_dtype=F32)
                assert torch.equal(out, (q[:, first:first + t].float() - 8).t())


@pytest.mark.parametrize("t,n,k", [(0, 16, 8), (3, 0, 8), (3, 16, 0), (70, 24, 0)])
def test_4bit_without_elements(handle, t, n, k):
    x = torch.empty(t, max(k, 8), dtype=BF16, device="cuda")[:, :k]
    w = torch.empty(n, 16, dtype=torch.uint8, device="cuda")[:, :(k + 1) // 2]
    scales = torch.ones(n, -(-k // 32), dtype=BF16, device="cuda")
    bias = torch.arange(n, dtype=F32, device="cuda")
    out = tcg.linear_4bit(handle, x, w, scales, 32, bias=bias)
    assert out.shape == (t, n)
    if k == 0:
        assert torch.equal(out.float(), bias.expand(t, n))


@pytest.mark.parametrize("t", [1, 12, 40, 300])
def test_4bit_keeps_rows_apart(handle, t):
    g = gen_of(9)
    x = randn(g, t + 1, 520)
    w, scales, zeros = draw_4bit(g, 264, 520, 64, BF16, True)
    want = tcg.linear_4bit(handle, x, w, scales, 64, zeros=zeros)
    x[t // 2] = float("inf")
    got = tcg.linear_4bit(handle, x, w, scales, 64, zeros=zeros)
    rest = [i for i in range(t + 1) if i != t // 2]
    assert same_bits(got[rest], want[rest])


@pytest.mark.parametrize("size", [2.0 ** -50, 2.0 ** -30, 2.0 ** 40, 2.0 ** 60])
def test_4bit_of_small_and_large_rows(handle, size):
    """BF16 as far as its range goes, beside a row of ordinary size."""
    g = gen_of(10)
    x = randn(g, 3, 520)
    x[1] = (x[1].float() / 8 * size).to(BF16)
    w, scales, zeros = draw_4bit(g, 72, 520, 64, BF16, True)
    out = tcg.linear_4bit(handle, x, w, scales, 64, zeros=zeros, out_dtype=F32)
    within(out, *ref.linear_4bit(x, w, scales, zeros, 64, None, "none", None, 0.0, False, F32), "out")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_4bit_scales_without_a_number(handle, dtype):
    """A NaN among the scales or zeros of a row is that row's alone."""
    g = gen_of(14)
    x = randn(g, 5, 264, dtype=dtype)
    w, scales, zeros = draw_4bit(g, 40, 264, 32, dtype, True)
    want = tcg.linear_4bit(handle, x, w, scales, 32, zeros=zeros)
    scales[7, 3], zeros[20, 0] = float("nan"), float("nan")
    got = tcg.linear_4bit(handle, x, w, scales, 32, zeros=zeros)
    rest = [i for i in range(40) if i not in (7, 20)]
    assert torch.isnan(got[:, [7, 20]]).all() and same_bits(got[:, rest], want[:, rest])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_4bit_scales_anywhere(handle, group, kind):
    """Scales and zeros that start at any element, where a stage's are not one aligned load."""
    g = gen_of(15)
    t, n, k = 5, 72, 1024
    x = randn(g, t, k)
    w, scales, zeros = draw_4bit(g, n, k, group, kind, True)
    want = tcg.linear_4bit(handle, x, w, scales, group, zeros=zeros)

    def moved(a):
        room = torch.full((a.numel() + 1,), float("nan"), dtype=a.dtype, device="cuda")
        room[1:] = a.flatten()
        return room[1:].view(a.shape)
    assert same_bits(tcg.linear_4bit(handle, x, w, moved(scales), group, zeros=zeros), want)
    assert same_bits(tcg.linear_4bit(handle, x, w, scales, group, zeros=moved(zeros)), want)


# ------------------------------------------------------------- places past 2^31 elements
def test_norm_far_rows(handle):
    g = gen_of(16)
    t, k = 66000, 32768                       # 2.16e9 elements
    x = torch.zeros(t, k, dtype=BF16, device="cuda")
    x[-3:] = randn(g, 3, k)
    weight, kept = randn(g, k), x[-3:].clone()
    q, scale = tcg.rms_norm_8bit(handle, x, weight)
    alone, alone_scale = tcg.rms_norm_8bit(handle, kept, weight)
    assert same_bits(q[-3:], alone) and same_bits(scale[-3:], alone_scale) and (scale[:-3] == 2.0 ** -100).all()
    del q
    tcg.rms_norm(handle, x, weight, out=x)
    assert same_bits(x[-3:], tcg.rms_norm(handle, kept, weight)) and not x[:-3].any()
    x[-3:] = kept
    dx, dw = tcg.rms_norm_backward(handle, x, x, weight, dx=x)
    want = tcg.rms_norm_backward(handle, kept, kept, weight)
    assert dx is x and same_bits(dx[-3:], want[0])
    bound = 66000 * 2.0 ** -24 * ref.norm_backward(kept, kept, weight, 1e-6, None)[0][1].abs() + 1e-6
    within(dw, want[1].double(), bound, "dw")


def test_gated_far_tokens(handle):
    g = gen_of(17)
    t, n, k = 140000, 8192, 64                # z: 2.29e9 elements
    x = torch.zeros(t, k, dtype=BF16, device="cuda")
    x[-300:] = randn(g, 300, k)
    w = randn(g, 2 * n, k, std=0.125)
    z = torch.full((t, 2 * n), 7.0, dtype=BF16, device="cuda")
    out = tcg.gated_linear(handle, x, w, z=z)
    want, eo, zw, ez = ref.gated(x[-300:], w, "silu", BF16)
    within(out[-300:], want, eo, "out")
    within(z[-300:], zw, ez + U[BF16] * (zw.abs() + ez) + TINY[BF16], "z")
    assert not out[:-300].any() and not z[:-300].any()
    dx, dw = tcg.gated_linear_backward(handle, out, x, w, z)
    (dxw, dww), (ex, ew) = ref.gated_backward(out[-300:], x[-300:], w, z[-300:], "silu")
    within(dx[-300:], dxw, ex, "dx")
    within(dw, dww, ew + (t * 2.0 ** -23) * ew, "dw")
    assert not dx[:-300].any()


@pytest.mark.parametrize("t", [2, 70])
def test_4bit_far_rows(handle, t):
    g = gen_of(18)
    n, k, group = 66000, 65536, 128           # 2.16e9 bytes of weights, 4.3e9 elements
    x = randn(g, t, k)
    w = torch.full((n, k // 2), 0x88, dtype=torch.uint8, device="cuda")      # q = 8: zero
    scales = torch.ones(n, k // group, dtype=BF16, device="cuda")
    last, s, _ = draw_4bit(g, 64, k, group, BF16, False, apart=False)
    w[-64:], scales[-64:] = last, s
    out = tcg.linear_4bit(handle, x, w, scales, group, out_dtype=F32)
    want, bound = ref.linear_4bit(x, last, s, None, group, None, "none", None, 0.0, False, F32)
    within(out[:, -64:], want, bound, "out")
    assert not out[:, :-64].any()


# ---------------------------------------------------------------------------- together
def test_layer_step(handle):
    """The feed-forward half of a layer forward and backward, as a training step runs it, against
    FP64 through autograd: relative 2-norm, each 16-bit rounding on the way (five forward, four more
    backward) adding at most half a step, U, of its own result."""
    g = gen_of(11)
    t, d, f = 333, 264, 520
    x, stream = randn(g, t, d), randn(g, t, d)
    weight = randn(g, d, std=0.2) + 1
    w1, w2 = randn(g, 2 * f, d, std=d ** -0.5), randn(g, d, f, std=f ** -0.5)
    z, s = torch.empty(t, 2 * f, dtype=BF16, device="cuda"), torch.empty_like(x)
    h = tcg.rms_norm(handle, x, weight, residual=stream, sum_out=s)
    a = tcg.gated_linear(handle, h, w1, z=z)
    y = tcg.linear(handle, a, w2, residual=s)
    dy = randn(g, t, d)
    da, dw2, _ = tcg.linear_backward(handle, dy, a, w2, want=("dx", "dw"))
    dh, dw1 = tcg.gated_linear_backward(handle, da, h, w1, z)
    dx, dweight = tcg.rms_norm_backward(handle, dh, s, weight, dsum=dy)

    leaves = [v.double().requires_grad_(True) for v in (x, weight, w1, w2)]
    xd, wd, w1d, w2d = leaves
    sd = xd + stream.double()
    hd = sd / torch.sqrt(sd.square().mean(1, keepdim=True) + 1e-6) * wd
    zd = hd @ w1d.t()
    yd = (zd[:, :f] * torch.sigmoid(zd[:, :f]) * zd[:, f:]) @ w2d.t() + sd
    grads = torch.autograd.grad(yd, leaves, dy.double())
    for got, want, roundings in ((y, yd.detach(), 5), (dw2, grads[3], 6), (dw1, grads[2], 9), (dx, grads[0], 9),
                                 (dweight, grads[1], 9)):
        assert float((got.double() - want).norm() / want.norm()) < roundings * U[BF16]


def test_decode_step(handle):
    """A token through the norm and 4-bit projections, and the 8-bit norm through the FP8 product."""
    g = gen_of(12)
    d, f = 512, 1040
    x, stream, weight = randn(g, 1, d), randn(g, 1, d), randn(g, d, std=0.2) + 1
    w1, s1, _ = draw_4bit(g, 2 * f, d, 64, BF16, False)
    w2, s2, z2 = draw_4bit(g, d, f, 32, BF16, True)
    s = stream.clone()
    h = tcg.rms_norm(handle, x, weight, residual=s, sum_out=s)
    a = tcg.linear_4bit(handle, h, w1, s1, 64, act="silu", gated=True)
    y = tcg.linear_4bit(handle, a, w2, s2, 32, zeros=z2, residual=s, out=s)
    sd = x.double() + stream.double()
    hd = sd / torch.sqrt(sd.square().mean(1, keepdim=True) + 1e-6) * weight.double()
    zd = hd @ ref.weights_4bit(w1, d, s1, None, 64)[0].t()
    yd = (zd[:, :f] * torch.sigmoid(zd[:, :f]) * zd[:, f:]) @ ref.weights_4bit(w2, f, s2, z2, 32)[0].t() + sd
    assert y is s and float((y.double() - yd).norm() / yd.norm()) < 5 * U[BF16]

    x = randn(g, 200, d)
    q, scale = tcg.rms_norm_8bit(handle, x, weight)
    w8 = randn(g, d, 256, dtype=F32).to(E4M3)
    out = torch.empty(200, 256, device="cuda")
    tcg.gemm_rowmajor(handle, q, w8, out)
    out *= scale[:, None]
    y = ref.norm(x, weight, 1e-6, None, BF16)[0]
    want = y @ w8.double()
    assert float((out.double() - want).norm() / want.norm()) < 2.0 ** -4


# ------------------------------------------------------------- streams, graphs, memory
def calls(h, s):
    """One call of each kind, into the buffers of s."""
    tcg.rms_norm(h, s["x"], s["weight"], residual=s["res"], sum_out=s["sum"], out=s["h"])
    tcg.rms_norm_8bit(h, s["x"], s["weight"], out=s["q"], scale=s["scale"])
    tcg.gated_linear(h, s["h"], s["w1"], out=s["a"], z=s["z"])
    tcg.gated_linear_backward(h, s["a"], s["h"], s["w1"], s["z"], dx=s["dx"], dw=s["dw1"])
    tcg.rms_norm_backward(h, s["dx"], s["sum"], s["weight"], dx=s["dxn"], dw=s["dwn"])
    tcg.linear_4bit(h, s["x"], s["w4"], s["s4"], 64, out=s["y"])


OUTS = ("sum", "h", "q", "scale", "a", "z", "dx", "dw1", "dxn", "dwn", "y")


def buffers(t, d, f, seed):
    g = gen_of(seed)
    new = lambda *shape, dtype=BF16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"x": randn(g, t, d), "res": randn(g, t, d), "weight": randn(g, d), "w1": randn(g, 2 * f, d, std=d ** -0.5)}
    s["w4"], s["s4"], _ = draw_4bit(g, f, d, 64, BF16, False)
    s |= {"sum": new(t, d), "h": new(t, d), "q": new(t, -(-d // 16) * 16).to(E4M3)[:, :d], "scale": new(t, dtype=F32), "a": new(t, f),
          "z": new(t, 2 * f), "dx": new(t, d), "dw1": new(2 * f, d), "dxn": new(t, d), "dwn": new(d, dtype=F32),
          "y": new(t, f)}
    return s


@pytest.mark.parametrize("t", [1, 20, 500])
def test_captured_and_replayed(cuda_device, t):
    h = tcg.Handle()
    s = buffers(t, 520, 264, t)
    calls(h, s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUTS}
    for k in OUTS:
        s[k].zero_()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    h.set_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls(h, s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k in OUTS:
        assert same_bits(s[k], want[k]), k
    tcg.check(tcg.tcg_get_device_error(h.h))
    del graph
    h.close()


def test_other_stream_and_dropped_inputs(cuda_device):
    """A handle on a stream of its own; the caller drops its tensors at once."""
    side = torch.cuda.Stream()
    h, plain = tcg.Handle(side), tcg.Handle()
    s = buffers(300, 1032, 520, 1)
    calls(plain, s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUTS}
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    x = s["x"].clone()
    side.wait_stream(torch.cuda.current_stream())
    out = tcg.rms_norm(h, x, s["weight"], residual=s["res"])
    a = tcg.gated_linear(h, out, s["w1"])
    y = tcg.linear_4bit(h, x, s["w4"], s["s4"], 64)
    del x, out
    junk = [torch.full_like(s["x"], 7.0) for _ in range(4)]
    torch.cuda.synchronize()
    assert same_bits(a, want["a"]) and same_bits(y, want["y"]) and junk
    h.close()
    plain.close()


def test_two_streams_at_once(cuda_device):
    """Two handles on streams of their own, their calls under way together."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    plain, handles = tcg.Handle(), [tcg.Handle(s) for s in streams]
    sets = [buffers(t, 1032, 520, t) for t in (200, 20)]
    want = []
    for s in sets:
        calls(plain, s)
        torch.cuda.synchronize()
        want.append({k: s[k].clone() for k in OUTS})
    for s in sets:
        for k in OUTS:
            s[k].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for h, s in zip(handles, sets):
            calls(h, s)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        for k in OUTS:
            assert same_bits(s[k], w[k]), k
    for h in (*handles, plain):
        tcg.check(tcg.tcg_get_device_error(h.h))
        h.close()


def test_capture_does_not_grow_the_workspace(cuda_device):
    stream = torch.cuda.Stream()
    h = tcg.Handle(stream)
    s = buffers(200, 520, 264, 3)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        tcg.rms_norm(h, s["x"], s["weight"], out=s["h"])
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    refused = []
    with torch.cuda.graph(graph, stream=stream):
        tcg.rms_norm(h, s["x"], s["weight"], out=s["h"])
        for call in (lambda: tcg.gated_linear_backward(h, s["a"], s["h"], s["w1"], s["z"], dx=s["dx"], dw=s["dw1"]),
                     lambda: tcg.rms_norm_backward(h, s["dx"], s["sum"], s["weight"], dx=s["dxn"], dw=s["dwn"]),
                     lambda: tcg.linear_4bit(h, s["x"], s["w4"], s["s4"], 64, out=s["y"])):
            try:
                call()
            except tcg.TcgError as e:
                refused.append(e.status)
    assert refused == [tcg.TCG_STATUS_ALLOC_FAILED] * 3
    del graph
    h.close()


@pytest.mark.parametrize("t", [1, 20, 500])
def test_wait_that_runs_out(cuda_device, t):
    """A load that never comes ends a gated product with an error, and the next call is right."""
    h = tcg.Handle()
    s = buffers(t, 520, 264, 6)
    tcg.gated_linear(h, s["x"], s["w1"], out=s["a"])
    tcg.check(tcg.tcg_get_device_error(h.h))
    want = s["a"].clone()
    tcg.tcg_set_debug(h.h, 2_000_000, 1)
    tcg.gated_linear(h, s["x"], s["w1"], out=s["a"])
    assert tcg.tcg_get_device_error(h.h) == tcg.TCG_STATUS_TIMEOUT
    tcg.tcg_set_debug(h.h)
    tcg.gated_linear(h, s["x"], s["w1"], out=s["a"])
    tcg.check(tcg.tcg_get_device_error(h.h))
    assert same_bits(s["a"], want)
    h.close()


@pytest.mark.parametrize("t", [1, 20, 500])
def test_given_workspace_is_enough(cuda_device, t):
    h = tcg.Handle()
    d, f = 1032, 2056
    s = buffers(t, d, f, 5)
    calls(h, s)
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in OUTS}
    sizes = (tcg.tcg_gemm_gated_workspace_size(h.h, f, t, d), tcg.tcg_gated_backward_workspace_size(h.h, f, t, d),
             tcg.tcg_rms_norm_backward_workspace_size(h.h, t, d), tcg.tcg_gemm_4bit_workspace_size(h.h, f, t, d))
    own = tcg.Handle()
    room = torch.full((max(sizes) + 256,), 77, dtype=torch.uint8, device="cuda")
    tcg.check(tcg.tcg_set_workspace(own.h, room.data_ptr(), max(sizes)))
    calls(own, s)
    torch.cuda.synchronize()
    for k in OUTS:
        assert same_bits(s[k], want[k]), k
    assert (room[max(sizes):] == 77).all()
    h.close()
    own.close()
