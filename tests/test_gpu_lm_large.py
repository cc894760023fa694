"""Language-model products at sizes that choose other kernels than the small tests do: many
rows per expert, gradients of the cross entropy in pieces, tiles cut in equal ranges of K."""
import pytest
import torch

import lm_reference as ref
import mixed_precision_tensor_gb300 as tcg
from test_gpu_lm import ACTS, BF16, F16, F32, gen_of, offsets_of, padded, randn, same_bits, xent_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle(cuda_device):
    h = tcg.Handle()
    yield h
    tcg.check(tcg.tcg_get_device_error(h.h), "device error word")
    h.close()


@pytest.mark.parametrize("sizes,n,k,cut", [
    ([4100, 0, 3000, 2309], 264, 136, False), ([2048, 2048], 1000, 72, False), ([9000, 1, 0, 255], 72, 4104, True),
    ([5000], 520, 4104, True), ([1024, 900, 1200], 264, 520, False), ([2100, 3011, 1100], 200, 2312, True)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lead,spare", [(0, 0), (300, 513)])
def test_experts_with_many_rows(handle, sizes, n, k, cut, dtype, lead, spare):
    """1024 rows and more for each expert: tokens on the accumulator's rows, each expert's own
    last tiles, whole tiles of rows of no expert, tiles cut along K."""
    e, rows = len(sizes), sum(sizes) + lead + spare
    act = ACTS[(n + e + lead) % 5]
    out_dtype = F32 if lead else dtype
    g = gen_of(rows + n)
    off = offsets_of(sizes, lead)
    assert (tcg.tcg_gemm_epilogue_workspace_size(handle.h, 1, 0, n, rows, k, e) > 0) == cut
    x, w = padded(randn(g, rows, k, dtype=dtype)), padded(randn(g, e, n, k, dtype=dtype, std=k ** -0.5))
    dout, z = padded(randn(g, rows, n, dtype=dtype)), padded(randn(g, rows, n, dtype=dtype))
    bias, res = randn(g, e, n, dtype=F32 if lead else dtype), padded(randn(g, rows, n, dtype=out_dtype))
    ends = off.tolist()
    for a in (x, dout, z, res):               # rows of no expert hold NaN: it must not reach anything
        a[:ends[0]] = float("nan")
        a[ends[-1]:] = float("nan")
    zo = padded(torch.ones(rows, n, dtype=dtype, device="cuda"))
    out = tcg.grouped_linear(handle, x, w, off, bias=bias, act=act, residual=res, beta=0.75, out_dtype=out_dtype,
                             z=zo)
    dx, dw, db = tcg.grouped_linear_backward(handle, dout, x, w, off, z=z, act=act)
    tcg.check(tcg.tcg_get_device_error(handle.h))
    again = tcg.grouped_linear(handle, x, w, off, bias=bias, act=act, residual=res, beta=0.75, out_dtype=out_dtype)
    assert same_bits(again, out)
    for a in (out, zo, dx):
        assert not a[:ends[0]].any() and not a[ends[-1]:].any()
    for j in range(e):
        a, b = ends[j], ends[j + 1]
        if a == b:
            assert not dw[j].any() and not db[j].any()
            continue
        want, zw, eo, ez = ref.linear(x[a:b], w[j], bias[j], act, res[a:b], 0.75, 1.0, out_dtype)
        ref.within(out[a:b], want, eo, f"out of expert {j}")
        ref.within(zo[a:b], zw, ez + ref.U[dtype] * (zw.abs() + ez) + ref.TINY[dtype], "z")
        grads, bounds = ref.linear_backward(dout[a:b], x[a:b], w[j], z[a:b], act)
        for name, got, gw, eb in zip(("dx", "dw", "dbias"), (dx[a:b], dw[j], db[j]), grads, bounds):
            ref.within(got, gw, eb, f"{name} of expert {j}")


@pytest.mark.parametrize("k", [70, 67, 64])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_cross_entropy_gradient_in_pieces(handle, dtype, k):
    """Several pieces of the vocabulary: dx summed in FP32 (of the scaled gradient in FP16) and
    rounded at the end, for feature counts that are no multiple of four as well."""
    x, w, target, dloss = xent_case(9000, 16000, k, dtype)
    target[::7] = -100
    x, w = padded(x), padded(w)
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    launches = tcg.tcg_launch_count(handle.h)
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
    assert tcg.tcg_launch_count(handle.h) - launches > 6       # two pieces at least
    tcg.check(tcg.tcg_get_device_error(handle.h))
    (dx_w, dw_w), (ex, ew) = ref.xent_backward(x, w, target, -100, dloss)
    ref.within(dx, dx_w, ex, "dx")
    ref.within(dw, dw_w, ew, "dw")
    assert not dx[::7].any()


@pytest.mark.parametrize("t,v", [(200, 5003), (3, 9001)])
def test_fp16_gradients_of_rows_far_apart(handle, t, v):
    """Upstream gradients from 1 down to 2^-40 in one FP16 call.  One power of two serves all
    rows: each entry of the logits' gradient is held to 2^-38 of the largest of them."""
    x, w, target, _ = xent_case(t, v, 136, F16)
    dloss = 2.0 ** -(torch.arange(t, device="cuda") * 41 // t).float()
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
    (dx_w, dw_w), (ex, ew) = ref.xent_backward(x, w, target, -100, dloss)
    ref.within(dx, dx_w, ex, "dx")
    ref.within(dw, dw_w, ew, "dw")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_cut_tiles_in_equal_ranges(handle, dtype):
    """Few tiles of operands that exceed half of L2, shared by tiles on both sides: sums of whole
    numbers are exact, and alike from call to call."""
    g = gen_of(12)
    t, n, k = 1000, 1024, 50021
    assert tcg.tcg_gemm_epilogue_workspace_size(handle.h, 1, 0, n, t, k) > 0

    def whole(rows, cols):
        return padded(torch.randint(-2, 3, (rows, cols), generator=g, device="cuda").to(dtype), extra=0)

    x, w = whole(t, k), whole(n, k)
    want = (x.double() @ w.double().t()).float()
    for _ in range(3):
        assert torch.equal(tcg.linear(handle, x, w, out_dtype=F32), want)
    d, x = whole(k, n), whole(k, t)                            # dw: the tokens are K
    want = (d.double().t() @ x.double()).to(dtype)
    for _ in range(3):
        assert torch.equal(tcg.linear_backward(handle, d, x, torch.zeros(n, t, dtype=dtype, device="cuda"),
                                               want=("dw",))[1], want)
    tcg.check(tcg.tcg_get_device_error(handle.h))


@pytest.mark.parametrize("rows", [4096, 4097, 70001, 300000])
@pytest.mark.parametrize("where", [0.0, 0.37, 1.0])
def test_scale_of_many_rows(handle, rows, where):
    """The largest upstream gradient may be anywhere among rows of several blocks: FP16 entries of
    its row stay in range, and the next calls find the counters as they should be."""
    x, w, target, _ = xent_case(rows, 50, 16, F16)
    at = int(where * (rows - 1))
    dloss = torch.full((rows,), 2.0 ** -6, device="cuda")
    dloss[at] = 40.0
    target[(at + 1) % rows] = -100
    dloss[(at + 1) % rows] = 1e9               # does not count
    _, lse = tcg.linear_cross_entropy(handle, x, w, target)
    first = None
    for _ in range(3):
        dx, dw = tcg.linear_cross_entropy_backward(handle, x, w, target, lse, dloss)
        assert first is None or (same_bits(dx, first[0]) and same_bits(dw, first[1]))
        first = dx, dw
    d = torch.where(target >= 0, dloss, torch.zeros_like(dloss))
    (dx_w, dw_w), (ex, ew) = ref.xent_backward(x, w, target, -100, d)
    ref.within(dx, dx_w, ex, "dx")
    ref.within(dw, dw_w, ew, "dw")
