"""The language-model products on the GPU against FP64 (lm_reference), at the sizes,
masks and layouts where they can go wrong."""
import math

import pytest
import torch

import lm_reference as ref
import mixed_precision_tensor_gb300 as tcg

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = tcg.Handle()
    yield h
    tcg.check(tcg.tcg_get_device_error(h.h), "device error word")
    h.close()


def randn(gen, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def padded(t, extra=8):
    """The same matrix with its rows further apart, NaN between them."""
    per = 16 // t.element_size()
    ld = -(-t.shape[-1] // per) * per + extra
    big = torch.full((*t.shape[:-1], ld), float("nan"), dtype=t.dtype, device=t.device)
    big[..., :t.shape[-1]] = t
    return big[..., :t.shape[-1]]


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------------------ linear
SIZES = [(1, 8, 8), (1, 4096, 4096), (4, 301, 523), (8, 1000, 264), (6, 40, 300), (2, 13, 5), (3, 264, 72), (17, 300, 1000), (33, 256, 64),
         (64, 1000, 1032), (100, 520, 200), (129, 2056, 264), (257, 513, 127), (300, 77, 2048),
         (700, 1288, 320), (200, 1000, 4096), (2000, 4096, 256), (5, 256, 20000), (2, 1032, 8200), (4, 2056, 5000),
         (100, 512, 8192), (90, 1000, 4104), (45, 2000, 4096), (1500, 1000, 4096)]


@pytest.mark.parametrize("t,n,k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_forward(handle, t, n, k, dtype):
    g = gen_of(t * 31 + n * 7 + k)
    act = ACTS[(t + n + k) % 5]
    out_dtype = F32 if (t + k) % 3 == 0 else dtype
    x, w = padded(randn(g, t, k, dtype=dtype)), padded(randn(g, n, k, dtype=dtype, std=k ** -0.5))
    bias = randn(g, n, dtype=F32 if n % 2 else dtype)
    res = padded(randn(g, t, n, dtype=out_dtype))
    z = padded(torch.zeros(t, n, dtype=dtype, device="cuda"))
    out = padded(torch.zeros(t, n, dtype=out_dtype, device="cuda"))
    assert tcg.linear(handle, x, w, bias=bias, act=act, residual=res, beta=0.5, alpha=1.25, out=out,
                      z=z) is out
    tcg.check(tcg.tcg_get_device_error(handle.h))
    want, zw, eo, ez = ref.linear(x, w, bias, act, res, 0.5, 1.25, out_dtype)
    ref.within(out, want, eo, "out")
    ref.within(z, zw, ez + ref.U[dtype] * (zw.abs() + ez) + ref.TINY[dtype], "z")
    for buf, cols in ((out, n), (z, n)):      # nothing between the rows was written
        full = torch.as_strided(buf, (t, buf.stride(0)), (buf.stride(0), 1))
        assert torch.isnan(full[:, cols:]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
def test_linear_activations(handle, act, dtype, out_dtype):
    g = gen_of(5)
    x, w = randn(g, 70, 96, dtype=dtype), randn(g, 312, 96, dtype=dtype, std=0.4)
    out = tcg.linear(handle, x, w, act=act, out_dtype=out_dtype)
    want, _, eo, _ = ref.linear(x, w, None, act, None, 0.0, 1.0, out_dtype)
    ref.within(out, want, eo, act)


def test_linear_extreme_values(handle):
    """Pre-activations from -60000 to 60000, infinities and NaN: each stays in its row."""
    k = 64
    x = torch.zeros(40, k, dtype=BF16, device="cuda")
    x[:, 0] = torch.tensor([(-1.0) ** i * 2.0 ** (i % 17 - 4) for i in range(40)])
    x[7, 3], x[9, 3], x[11, 3] = float("nan"), float("inf"), float("-inf")
    w = torch.zeros(256, k, dtype=BF16, device="cuda")
    w[:, 0] = torch.linspace(0.0, 14.0, 256)
    w[:, 3] = 1.0
    for act in ACTS:
        out = tcg.linear(handle, x, w, act=act, out_dtype=F32)
        want, _, eo, _ = ref.linear(x, w, None, act, None, 0.0, 1.0, F32)
        keep = [i for i in range(40) if i not in (7, 9, 11)]
        ref.within(out[keep], want[keep], eo[keep], act)
        assert torch.isnan(out[7]).all()
        assert (out[9] == float("inf")).all()
        if act == "relu":
            assert (out[11] == 0).all()


def test_linear_integers_are_exact(handle):
    g = gen_of(11)
    for t in (1, 20, 50, 130, 600):
        x = torch.randint(-2, 3, (t, 520), generator=g, device="cuda").to(BF16)
        w = torch.randint(-2, 3, (776, 520), generator=g, device="cuda").to(BF16)
        b = torch.randint(-4, 5, (776,), generator=g, device="cuda").float()
        out = tcg.linear(handle, x, w, bias=b, out_dtype=F32)
        assert torch.equal(out.double(), x.double() @ w.double().t() + b.double())


def test_linear_in_place_residual_and_empty(handle):
    g = gen_of(3)
    x, w = randn(g, 45, 128), randn(g, 256, 128, std=0.1)
    out = randn(g, 45, 256)
    want, _, eo, _ = ref.linear(x, w, None, "silu", out.clone(), 1.0, 1.0, BF16)
    tcg.linear(handle, x, w, act="silu", residual=out, out=out)
    ref.within(out, want, eo)
    assert tcg.linear(handle, x[:0], w).shape == (0, 256)
    bias = randn(g, 256)
    none = tcg.linear(handle, x[:, :0], w[:, :0], bias=bias)   # nothing to sum: the bias alone
    assert torch.equal(none, bias.expand(45, 256))


@pytest.mark.parametrize("t,n,k", [(1, 2048, 4096), (4, 300, 1000), (12, 2048, 4096), (40, 512, 8192),
                                   (200, 300, 16384)])
def test_linear_is_deterministic(handle, t, n, k):
    g = gen_of(t)
    x, w = randn(g, t, k), randn(g, n, k, std=k ** -0.5)
    # tiles cut along K keep partial sums; a few tokens need none
    assert (tcg.tcg_gemm_epilogue_workspace_size(handle.h, 1, 0, n, t, k) > 0) == (t > 4)
    first = tcg.linear(handle, x, w, out_dtype=F32)
    for _ in range(5):
        assert same_bits(tcg.linear(handle, x, w, out_dtype=F32), first)


@pytest.mark.parametrize("t,n,k", [(1, 264, 72), (2, 13, 5), (33, 256, 512), (257, 520, 136),
                                   (1000, 1000, 264), (4099, 256, 320)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_backward(handle, t, n, k, dtype):
    g = gen_of(t + n + k)
    act = ACTS[(t + n) % 5]
    x, w = padded(randn(g, t, k, dtype=dtype)), padded(randn(g, n, k, dtype=dtype, std=k ** -0.5))
    dout, z = padded(randn(g, t, n, dtype=dtype)), padded(randn(g, t, n, dtype=dtype, std=2.0))
    got = tcg.linear_backward(handle, dout, x, w, z=z, act=act)
    tcg.check(tcg.tcg_get_device_error(handle.h))
    want, bounds = ref.linear_backward(dout, x, w, z, act)
    for name, a, b, e in zip(("dx", "dw", "dbias"), got, want, bounds):
        ref.within(a, b, e, f"{name} {act}")


@pytest.mark.parametrize("act", ACTS)
def test_activation_slopes(handle, act):
    """dbias of a single token is dout act'(z) in FP32: z over the whole range, zero included."""
    z = torch.cat([torch.linspace(-30, 30, 4000, device="cuda"),
                   torch.tensor([0.0, -0.0, 1e-20, -1e-20, 100.0, -100.0, 3e4, -3e4],
                                device="cuda")])[None].to(BF16)
    n = z.shape[1]
    dout = torch.full((1, n), 1.0, dtype=BF16, device="cuda")
    w = torch.zeros(n, 8, dtype=BF16, device="cuda")
    x = torch.zeros(1, 8, dtype=BF16, device="cuda")
    db = tcg.linear_backward(handle, dout, x, w, z=z, act=act, want=("dbias",))[2]
    want = ref.slope(z.double(), act)[0]
    assert float((db.double() - want).abs().max()) <= ref.FN * 4


def test_linear_backward_wants(handle):
    g = gen_of(2)
    x, w, d = randn(g, 50, 64), randn(g, 72, 64), randn(g, 50, 72)
    full = tcg.linear_backward(handle, d, x, w)
    for want in (("dx",), ("dw",), ("dbias",), ("dx", "dbias")):
        got = tcg.linear_backward(handle, d, x, w, want=want)
        for name, a, b in zip(("dx", "dw", "dbias"), got, full):
            assert (a is None) == (name not in want)
            assert a is None or same_bits(a, b)
    dx, dw, db = tcg.linear_backward(handle, d[:0], x[:0], w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("experts", [0, 5])
def test_layer_backward_in_the_callers_workspace(cuda_device, act, experts):
    """The workspace that the library asks for is enough, and one that is smaller is refused
    before anything is queued."""
    g = gen_of(8)
    t, n, k = 300, 264, 1160
    x, d, z = randn(g, t, k), randn(g, t, n), randn(g, t, n)
    w = randn(g, *((experts,) if experts else ()), n, k)
    off = offsets_of([100, 0, 7, 150, 43], 0) if experts else None
    h = tcg.Handle()
    run = (lambda **kw: tcg.grouped_linear_backward(h, d, x, w, off, z=z, act=act, **kw)) if experts else \
        (lambda **kw: tcg.linear_backward(h, d, x, w, z=z, act=act, **kw))
    want = run()
    for outputs in ("dx", "dw", "dbias"), ("dx",), ("dw",), ("dbias",):
        need = tcg.tcg_linear_backward_workspace_size(
            h.h, ACTS.index(act), n, t, k, experts, "dx" in outputs, "dw" in outputs, "dbias" in outputs)
        if not need:
            continue
        space = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
        tcg.check(tcg.tcg_set_workspace(h.h, space, need))
        got = run(want=outputs)
        for name, a, b in zip(("dx", "dw", "dbias"), got, want):
            assert a is None or same_bits(a, b), name
        assert bool((space[need:] == 0xff).all())
        tcg.check(tcg.tcg_set_workspace(h.h, space, need - 256))
        before = tcg.tcg_launch_count(h.h)
        with pytest.raises(tcg.TcgError):
            run(want=outputs)
        assert tcg.tcg_launch_count(h.h) == before
        tcg.check(tcg.tcg_set_workspace(h.h, None, 0))
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


# ----------------------------------------------------------------------------- grouped
GROUPS = [[5], [0, 3, 0], [1, 1, 1, 1], [64, 0, 65, 63, 1], [300, 7, 0, 129], [0, 0, 0],
          [33, 128, 256, 2, 90], [3] * 70, [1] * 200 + [0] * 184, [700, 1, 64, 127]]


def offsets_of(sizes, lead):
    o = [lead]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("i", range(len(GROUPS)))
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lead,spare", [(0, 0), (3, 41)])
def test_grouped_forward_and_backward(handle, i, dtype, lead, spare):
    sizes, act = GROUPS[i], ACTS[i % 5]
    e, rows = len(sizes), sum(sizes) + lead + spare
    n, k = [(264, 72), (520, 136), (13, 5), (256, 200)][i % 4]
    g = gen_of(i)
    off = offsets_of(sizes, lead)
    x, w = padded(randn(g, rows, k, dtype=dtype)), padded(randn(g, e, n, k, dtype=dtype, std=k ** -0.5))
    dout, z = randn(g, rows, n, dtype=dtype), randn(g, rows, n, dtype=dtype)
    dout, z = padded(dout), padded(z)
    bias = randn(g, e, n, dtype=F32 if i % 2 else dtype)
    res = padded(randn(g, rows, n, dtype=dtype))
    # rows of no expert hold NaN: it must not reach anything
    ends = off.tolist()
    for a in (x, dout, z, res):
        a[:ends[0]] = float("nan")
        a[ends[-1]:] = float("nan")
    zo = padded(torch.ones(rows, n, dtype=dtype, device="cuda"))
    out = tcg.grouped_linear(handle, x, w, off, bias=bias, act=act, residual=res, z=zo)
    dx, dw, db = tcg.grouped_linear_backward(handle, dout, x, w, off, z=z, act=act)
    tcg.check(tcg.tcg_get_device_error(handle.h))
    for a in (out, zo, dx):
        assert not a[:ends[0]].any() and not a[ends[-1]:].any()
    for j in range(e):
        a, b = ends[j], ends[j + 1]
        if a == b:
            assert not dw[j].any() and not db[j].any()
            continue
        want, zw, eo, ez = ref.linear(x[a:b], w[j], bias[j], act, res[a:b], 1.0, 1.0, dtype)
        ref.within(out[a:b], want, eo, f"out of expert {j}")
        ref.within(zo[a:b], zw, ez + ref.U[dtype] * (zw.abs() + ez) + ref.TINY[dtype], "z")
        grads, bounds = ref.linear_backward(dout[a:b], x[a:b], w[j], z[a:b], act)
        for name, got, gw, eb in zip(("dx", "dw", "dbias"), (dx[a:b], dw[j], db[j]), grads, bounds):
            ref.within(got, gw, eb, f"{name} of expert {j}")


def test_grouped_backward_from_its_parts(handle):
    """The epilogue's gradient and the two products, called one by one, give the bits of the
    one call behind grouped_linear_backward."""
    g = gen_of(9)
    e, t, n, k = 5, 300, 264, 136
    x, d, z, w = randn(g, t, k), randn(g, t, n), randn(g, t, n), randn(g, e, n, k)
    off = offsets_of([100, 0, 7, 150, 43], 0)
    want = tcg.grouped_linear_backward(handle, d, x, w, off, z=z, act="gelu")
    dz, dx, dw = torch.empty_like(d), torch.empty_like(x), torch.empty_like(w)
    db = torch.empty(e, n, device="cuda")
    ty = tcg.TCG_R_16BF
    tcg.check(tcg.tcg_epilogue_backward(handle.h, ACTS.index("gelu"), n, t, e, off, d, n, z, n, ty, dz, n, db))
    tcg.check(tcg.tcg_gemm_grouped(handle.h, 0, k, t, n, e, off, 1.0, w, k, n * k, dz, n, ty, dx, ty, k))
    tcg.check(tcg.tcg_gemm_grouped_k(handle.h, k, n, t, e, off, 1.0, x, k, dz, n, ty, dw, ty, k, n * k))
    tcg.check(tcg.tcg_get_device_error(handle.h))
    for name, a, b in zip(("dx", "dw", "dbias"), (dx, dw, db), want):
        assert same_bits(a, b), name
    dzw = d.double() * ref.slope(z.double(), "gelu")
    err = d.double().abs() * ref.FN * (1 + z.double().abs())
    ref.within(dz, dzw, err + ref.U[BF16] * (dzw.abs() + err) + ref.TINY[BF16], "dz")


@pytest.mark.parametrize("size", list(range(1, 70)) + [127, 128, 129, 191])
def test_grouped_weight_gradient_tails(handle, size):
    """Every length of a group's last tokens, at every offset of its start, with NaN all
    around: integers, so the sums are exact."""
    g = gen_of(size)
    lead = size % 7
    rows = lead + size + 9
    x = torch.full((rows, 136), float("nan"), dtype=BF16, device="cuda")
    d = torch.full((rows, 200), float("nan"), dtype=BF16, device="cuda")
    x[lead:lead + size] = torch.randint(-2, 3, (size, 136), generator=g, device="cuda").to(BF16)
    d[lead:lead + size] = torch.randint(-2, 3, (size, 200), generator=g, device="cuda").to(BF16)
    w = torch.zeros(1, 200, 136, dtype=BF16, device="cuda")
    off = torch.tensor([lead, lead + size], dtype=torch.int64, device="cuda")
    dw = tcg.grouped_linear_backward(handle, d, x, w, off, want=("dw",))[1][0]
    want = d[lead:lead + size].double().t() @ x[lead:lead + size].double()
    assert torch.equal(dw.double(), want.to(BF16).double())


def test_grouped_neighbours_do_not_mix(handle):
    """NaN in one expert's rows reaches that expert's outputs only."""
    g = gen_of(1)
    sizes = [30, 50, 20]
    off = offsets_of(sizes, 0)
    x, w, d = randn(g, 100, 128), randn(g, 3, 256, 128, std=0.1), randn(g, 100, 256)
    x[30:80] = float("nan")
    out = tcg.grouped_linear(handle, x, w, off)
    dx, dw, db = tcg.grouped_linear_backward(handle, d, x, w, off)
    assert torch.isfinite(out[:30].float()).all() and torch.isfinite(out[80:].float()).all()
    assert torch.isnan(out[30:80].float()).all() and torch.isnan(dw[1].float()).all()
    assert torch.isfinite(dw[0].float()).all() and torch.isfinite(dw[2].float()).all()
    assert torch.isfinite(dx.float()).all() and torch.isfinite(db).all()


def test_grouped_offsets_out_of_range_stay_in_bounds(handle):
    """Offsets below 0 or past the rows are taken as the nearest end."""
    g = gen_of(4)
    x, w = randn(g, 40, 64), randn(g, 3, 72, 64)
    wild = torch.tensor([-5, 10, 10, 10 ** 12], dtype=torch.int64, device="cuda")
    tame = torch.tensor([0, 10, 10, 40], dtype=torch.int64, device="cuda")
    assert same_bits(tcg.grouped_linear(handle, x, w, wild), tcg.grouped_linear(handle, x, w, tame))
    d = randn(g, 40, 72)
    for a, b in zip(tcg.grouped_linear_backward(handle, d, x, w, wild),
                    tcg.grouped_linear_backward(handle, d, x, w, tame)):
        assert same_bits(a, b)


@pytest.mark.parametrize("sizes", [[0, 1, 0, 0, 2, 0, 0, 1], [0, 7, 0, 0, 5, 1, 0, 2], [0] * 20 + [3, 0, 5] + [0] * 9,
                                   [0, 20, 0, 0, 11, 1, 0, 2]])
def test_grouped_few_rows(handle, sizes):
    """A pass over the weights (a row for two experts), or tiles cut along K."""
    g = gen_of(9)
    rows = sum(sizes)
    off = offsets_of(sizes, 0)
    e = len(sizes)
    x, w = randn(g, rows, 4096), randn(g, e, 256, 4096, std=1 / 64)
    cut = tcg.tcg_gemm_epilogue_workspace_size(handle.h, 1, 0, 256, rows, 4096, e) > 0
    assert cut == (e == 8 and rows > 4)
    first = tcg.grouped_linear(handle, x, w, off, act="silu", out_dtype=F32)
    for _ in range(4):
        assert same_bits(tcg.grouped_linear(handle, x, w, off, act="silu", out_dtype=F32), first)
    for j in range(e):
        a, b = off[j].item(), off[j + 1].item()
        if b > a:
            want, _, eo, _ = ref.linear(x[a:b], w[j], None, "silu", None, 0.0, 1.0, F32)
            ref.within(first[a:b], want, eo)


@pytest.mark.parametrize("sizes", [[40, 0, 70, 66], [130, 0, 101], [60], [1, 128, 3, 2], [200, 1], [25] * 8])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_tiles_of_few_experts(handle, sizes, dtype):
    """Few tiles of a long K: pieces of one tile on several pairs, alike from call to call."""
    g = gen_of(len(sizes))
    rows, e, n, k = sum(sizes), len(sizes), 264, 2312
    off = offsets_of(sizes, 0)
    x, w = randn(g, rows, k, dtype=dtype), randn(g, e, n, k, dtype=dtype, std=k ** -0.5)
    bias, z = randn(g, e, n, dtype=F32), torch.empty(rows, n, dtype=dtype, device="cuda")
    first = tcg.grouped_linear(handle, x, w, off, bias=bias, act="gelu", z=z)
    for _ in range(4):
        assert same_bits(tcg.grouped_linear(handle, x, w, off, bias=bias, act="gelu"), first)
    tcg.check(tcg.tcg_get_device_error(handle.h))
    for j in range(e):
        a, b = off[j].item(), off[j + 1].item()
        if b > a:
            want, zw, eo, ez = ref.linear(x[a:b], w[j], bias[j], "gelu", None, 0.0, 1.0, dtype)
            ref.within(first[a:b], want, eo)
            ref.within(z[a:b], zw, ez + ref.U[dtype] * (zw.abs() + ez) + ref.TINY[dtype], "z")


# ----------------------------------------------------------------------- cross entropy
def xent_case(t, v, k, dtype, seed=0, std=1.5):
    g = gen_of(seed + t + v + k)
    x, w = randn(g, t, k, dtype=dtype), randn(g, v, k, dtype=dtype, std=std / math.sqrt(k))
    target = torch.randint(0, v, (t,), generator=g, device="cuda")
    dloss = torch.randn(t, generator=g, device="cuda") / t
    return x, w, target, dloss


@pytest.mark.parametrize("t,v,k", [(1, 1, 8), (1, 2, 5), (1, 1000, 64), (3, 257, 72), (5, 30011, 200), (8, 999, 264),
                                   (17, 256, 200), (32, 3001, 1032), (130, 511, 64), (257, 1001, 136), (300, 5003, 256),
                                   (64, 50021, 128), (515, 300, 1000), (3, 9001, 1032)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent(handle, t, v, k, dtype):
    x, w, target, dloss = xent_case(t, v, k, dtype)
    if t > 4:
        target[1], target[2], target[3], target[4] = -100, v, -1, 0
        dloss[1] = float("nan")               # a row that does not count
    x, w = padded(x), padded(w)
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target)
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
    tcg.check(tcg.tcg_get_device_error(handle.h))
    loss_w, lse_w, bound, _, counts = ref.xent(x, w, target, -100)
    ref.within(lse, lse_w, bound, "lse")
    ref.within(loss, loss_w, bound, "loss")
    assert not loss[~counts].any()
    d = torch.where(counts, dloss, torch.zeros_like(dloss))
    (dx_w, dw_w), (ex, ew) = ref.xent_backward(x, w, target, -100, d)
    ref.within(dx, dx_w, ex, "dx")
    ref.within(dw, dw_w, ew, "dw")
    assert not dx[~counts].any()


def test_xent_in_pieces(handle):
    """Enough rows and vocabulary that the gradient goes in several pieces."""
    x, w, target, dloss = xent_case(9000, 16000, 64, BF16)
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target)
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
    launches = tcg.tcg_launch_count(handle.h)
    tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
    assert tcg.tcg_launch_count(handle.h) - launches > 6       # two pieces at least
    loss_w, lse_w, bound, _, _ = ref.xent(x, w, target, -100)
    ref.within(lse, lse_w, bound, "lse")
    (dx_w, dw_w), (ex, ew) = ref.xent_backward(x, w, target, -100, dloss)
    ref.within(dx, dx_w, ex, "dx")
    ref.within(dw, dw_w, ew, "dw")


@pytest.mark.parametrize("power", [-40, 0, 20])
def test_xent_fp16_keeps_small_gradients(handle, power):
    """Probabilities near 1 / vocab and upstream gradients of any size in FP16."""
    x, w, target, dloss = xent_case(200, 20000, 64, F16, std=0.2)
    x *= 16
    dloss = dloss * 2.0 ** power
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target)
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
    (dx_w, dw_w), (ex, ew) = ref.xent_backward(x, w, target, -100, dloss)
    ok = dx_w.abs() < 60000
    ref.within(torch.where(ok, dx.double(), dx_w), dx_w, ex, "dx")
    ok = dw_w.abs() < 60000
    ref.within(torch.where(ok, dw.double(), dw_w), dw_w, ew, "dw")


def test_xent_infinite_logits(handle):
    """Vocabulary entries at -inf have probability 0, whole tiles of them too; NaN stays in
    its row; a row that is all -inf has lse -inf like a sum over nothing."""
    t, v, k = 20, 900, 64
    x, w, target, dloss = xent_case(t, v, k, BF16)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    w[:600, 0] = float("-inf")                # two tiles and a half
    target = target % 300 + 600
    x[5, 1] = float("nan")
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target)
    logits = x.double() @ w.double().t()
    want = torch.logsumexp(logits, 1)
    keep = [i for i in range(t) if i != 5]
    assert torch.isnan(lse[5]) and torch.isnan(loss[5])
    assert float((lse.double() - want)[keep].abs().max()) < 1e-4
    w[:, 0] = float("-inf")
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target)
    assert (lse[keep] == float("-inf")).all()


def test_xent_ignores_everything(handle):
    x, w, target, dloss = xent_case(70, 400, 64, BF16)
    target[:] = 7
    loss, lse = tcg.linear_cross_entropy(handle, x, w, target, ignore_index=7)
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss, ignore_index=7)
    assert not loss.any() and not dx.any() and not dw.any()
    assert torch.isfinite(lse).all()
    dx, dw = tcg.linear_cross_entropy_backward(handle, x[:0], w, target[:0], lse[:0], dloss[:0])
    assert dx.shape == (0, 64) and not dw.any()


def test_xent_gradient_against_differences(handle):
    """Central differences of the library's own loss along random directions.

    With logits changing at rates a (|a| <= A), the loss's third derivative is at most
    2 (2 A)^3, so a step h is off by h^2 / 6 of that; the losses themselves are FP32."""
    t, v, k = 40, 600, 64
    x, w, target, _ = xent_case(t, v, k, BF16)
    x = (x * 8).round() / 8                    # so that x +- h d is exact in BF16
    x = x.clamp(-4, 4).to(BF16)
    h = 1.0 / 32
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    dx, _ = tcg.linear_cross_entropy_backward(handle, x, w, target, lse,
                                              torch.ones(t, device="cuda"))
    for seed in range(4):
        d = torch.randint(0, 2, (t, k), generator=gen_of(seed), device="cuda").to(BF16)
        up, _ = tcg.linear_cross_entropy(handle, (x.float() + h * d.float()).to(BF16), w, target)
        lo, _ = tcg.linear_cross_entropy(handle, (x.float() - h * d.float()).to(BF16), w, target)
        exact = (x.float() + h * d.float()).to(BF16).float() == x.float() + h * d.float()
        assert exact.all()
        slope = (up - lo).double() / (2 * h)
        rate = (d.double() @ w.double().t()).abs().max(1).values
        bound = h * h / 6 * 2 * (2 * rate) ** 3 + 2e-5 / h + \
            2.0 ** -7 * (dx.double().abs() @ d.double().t()).diagonal()
        off = (slope - (dx.double() * d.double()).sum(1)).abs()
        assert (off <= bound).all(), float((off - bound).max())


# -------------------------------------------------------------------- streams and errors
def test_side_stream_and_graph(cuda_device):
    g = gen_of(8)
    x, w, b = randn(g, 40, 4096), randn(g, 512, 4096, std=1 / 64), randn(g, 512)
    we, off = randn(g, 4, 256, 4096, std=1 / 64), offsets_of([10, 0, 25, 5], 0)
    target = torch.randint(0, 512, (40,), generator=g, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h = tcg.Handle(s)
    out = torch.empty(40, 512, dtype=BF16, device="cuda")
    ge = torch.empty(40, 256, dtype=BF16, device="cuda")
    loss, lse = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")

    def step():
        tcg.linear(h, x, w, bias=b, act="gelu", out=out)
        tcg.grouped_linear(h, x, we, off, out=ge)
        tcg.linear_cross_entropy(h, x, w, target, loss=loss, lse=lse)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    first = [a.clone() for a in (out, ge, loss, lse)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for a in (out, ge, loss, lse):
        a.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, f in zip((out, ge, loss, lse), first):
        assert same_bits(a, f)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


def test_timeout_is_reported_and_leaves_nothing(cuda_device):
    """A load that never comes: the bounded wait gives up, the status says so, and the next
    calls (a split one among them) are right."""
    g = gen_of(6)
    x, w = randn(g, 20, 4096), randn(g, 512, 4096, std=1 / 64)
    h = tcg.Handle()
    first = tcg.linear(h, x, w, out_dtype=F32).clone()
    tcg.check(tcg.tcg_get_device_error(h.h))
    tcg.check(tcg.tcg_set_debug(h.h, 20_000_000, 1))
    tcg.linear(h, x, w, out_dtype=F32)
    assert tcg.tcg_get_device_error(h.h) == tcg.TCG_STATUS_TIMEOUT
    tcg.check(tcg.tcg_set_debug(h.h, 0, 0))
    assert same_bits(tcg.linear(h, x, w, out_dtype=F32), first)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


def test_host_memory_and_foreign_pointers_are_refused(handle):
    g = gen_of(1)
    x, w = randn(g, 8, 64), randn(g, 64, 64)
    pinned = torch.empty(64, dtype=torch.float32, pin_memory=True)
    out = torch.empty(8, 64, dtype=BF16, device="cuda")
    before = tcg.tcg_launch_count(handle.h)
    e = tcg.Epilogue(bias=pinned.data_ptr(), bias_type=tcg.TCG_R_32F)
    assert tcg.tcg_gemm_epilogue(handle.h, 1, 0, 64, 8, 64, 1.0, w, 64, x, 64, tcg.TCG_R_16BF, out,
                                 tcg.TCG_R_16BF, 64, e) == tcg.TCG_STATUS_INVALID_VALUE
    off = torch.zeros(2, dtype=torch.int64, pin_memory=True)
    assert tcg.tcg_gemm_grouped(handle.h, 1, 64, 8, 64, 1, off, 1.0, w, 64, 4096, x, 64,
                                tcg.TCG_R_16BF, out, tcg.TCG_R_16BF, 64) == tcg.TCG_STATUS_INVALID_VALUE
    assert tcg.tcg_launch_count(handle.h) == before
