"""The language-model products on streams of their own: handles whose first calls, workspaces
and inputs meet work that other streams still have queued."""
import pytest
import torch

import mixed_precision_tensor_gb300 as tcg
from test_gpu_lm import BF16, F32, gen_of, randn, same_bits

pytestmark = pytest.mark.gpu

BUSY = 2_000_000_000                  # clock cycles that a stream is kept busy for: about a second


def cut_product(seed=1):
    """Inputs of a product whose tiles are cut along K, and its result."""
    g = gen_of(seed)
    x, w = randn(g, 20, 4096), randn(g, 512, 4096, std=1 / 64)
    h = tcg.Handle()
    assert tcg.tcg_gemm_epilogue_workspace_size(h.h, 1, 0, 512, 20, 4096) > 0
    want = tcg.linear(h, x, w, out_dtype=F32).clone()
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()
    torch.cuda.synchronize()
    return x, w, want


def test_first_calls_while_the_default_stream_is_busy(cuda_device):
    """A new handle's arrival counters are zero before its first kernel, whatever the legacy
    default stream still has to do."""
    x, w, want = cut_product()
    side = torch.cuda.Stream()
    out = [torch.empty(20, 512, dtype=F32, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    busy = torch.cuda.current_stream()
    h = tcg.Handle(side)
    for o in out:
        tcg.linear(h, x, w, out=o)
    side.synchronize()
    assert not busy.query()
    for o in out:
        assert same_bits(o, want)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


def test_error_word_is_read_and_cleared_beside_a_busy_default_stream(cuda_device):
    """After a wait that ran out, the counters are zero again before the next kernel."""
    x, w, want = cut_product(2)
    side = torch.cuda.Stream()
    out = [torch.empty(20, 512, dtype=F32, device="cuda") for _ in range(4)]
    h = tcg.Handle(side)
    tcg.linear(h, x, w, out=out[0])
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    busy = torch.cuda.current_stream()
    tcg.check(tcg.tcg_set_debug(h.h, 20_000_000, 1))     # one load that never comes
    tcg.linear(h, x, w, out=out[0])
    assert tcg.tcg_get_device_error(h.h) == tcg.TCG_STATUS_TIMEOUT
    tcg.check(tcg.tcg_set_debug(h.h, 0, 0))
    for o in out:
        tcg.linear(h, x, w, out=o)
    side.synchronize()
    assert not busy.query()
    for o in out:
        assert same_bits(o, want)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


def test_waits_do_not_include_the_kernel_before(cuda_device):
    """A short wait limit bounds a kernel's own waits.  Two calls back to back: one pair of
    SMs busy for longer than the limit, then tiles for all of them, whose blocks are resident
    early on the SMs that the first call leaves idle."""
    g = gen_of(3)
    h = tcg.Handle()
    tcg.check(tcg.tcg_set_split_k(h.h, 1))                  # the long product stays on one pair
    x1, w1 = randn(g, 20, 1 << 20), randn(g, 64, 1 << 20)
    x2, w2 = randn(g, 600, 64), randn(g, 4096, 64)
    out1 = torch.empty(20, 64, dtype=BF16, device="cuda")
    out2 = torch.empty(600, 4096, dtype=BF16, device="cuda")
    for _ in range(2):
        tcg.linear(h, x1, w1, out=out1)
        tcg.linear(h, x2, w2, out=out2)
    torch.cuda.synchronize()
    want1, want2 = out1.clone(), out2.clone()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    tcg.linear(h, x1, w1, out=out1)
    ev[1].record()
    torch.cuda.synchronize()
    limit = ev[0].elapsed_time(ev[1]) / 4                   # ms
    assert limit > 0.2
    tcg.check(tcg.tcg_set_debug(h.h, int(limit * 1e6), 0))
    for _ in range(3):
        tcg.linear(h, x1, w1, out=out1)
        tcg.linear(h, x2, w2, out=out2)
    tcg.check(tcg.tcg_get_device_error(h.h))
    assert same_bits(out1, want1) and same_bits(out2, want2)
    h.close()


def test_graph_keeps_its_workspace(cuda_device):
    """A captured call's workspace stays where the graph found it when a later call needs more."""
    x, w, want = cut_product(4)
    g = gen_of(5)
    out = torch.empty(20, 512, dtype=F32, device="cuda")
    s = torch.cuda.Stream()
    h = tcg.Handle(s)
    with torch.cuda.stream(s):
        tcg.linear(h, x, w, out=out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tcg.linear(h, x, w, out=out)
    with torch.cuda.stream(s):
        for rows in (300, 3000, 30000):                     # each needs more than the one before
            d, xb, wb = randn(g, rows, 512), randn(g, rows, 256), randn(g, 512, 256)
            tcg.linear_backward(h, d, xb, wb, z=randn(g, rows, 512), act="silu")
            s.synchronize()
            fill = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(64)]
            out.zero_()
            for _ in range(3):
                graph.replay()
            s.synchronize()
            assert same_bits(out, want)
            del fill
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


def test_capture_does_not_grow_the_workspace(cuda_device):
    """Refused cleanly: the capture goes on, and the call works once the handle has the memory."""
    x, w, want = cut_product(6)
    out, n = torch.empty(20, 512, dtype=F32, device="cuda"), torch.zeros(1, device="cuda")
    s = torch.cuda.Stream()
    h = tcg.Handle(s)
    with torch.cuda.stream(s):
        tcg.linear(h, x[:1], w)                             # binds the handle; needs no workspace
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        before = tcg.tcg_launch_count(h.h)
        with pytest.raises(tcg.TcgError) as e:
            tcg.linear(h, x, w, out=out)
        assert e.value.status == tcg.TCG_STATUS_ALLOC_FAILED and tcg.tcg_launch_count(h.h) == before
        n += 1
    graph.replay()
    torch.cuda.synchronize()
    assert float(n) == 1
    with torch.cuda.stream(s):
        tcg.linear(h, x, w, out=out)
    s.synchronize()
    assert same_bits(out, want)
    h.close()


@pytest.mark.parametrize("t", [1, 2, 4])
def test_few_tokens_timeout_leaves_nothing(cuda_device, t):
    """A load that never comes: the bounded wait gives up, the status says so, the copies under
    way have landed before the kernel's blocks leave, and the calls right after it are right."""
    g = gen_of(7)
    x, w = randn(g, t, 4096), randn(g, 1000, 4096, std=1 / 64)
    target = torch.randint(0, 1000, (t,), generator=g, device="cuda")
    h = tcg.Handle()
    want = tcg.linear(h, x, w, out_dtype=F32).clone()
    loss = tcg.linear_cross_entropy(h, x, w, target)[0].clone()
    tcg.check(tcg.tcg_get_device_error(h.h))
    for _ in range(2):
        tcg.check(tcg.tcg_set_debug(h.h, 20_000_000, 1))
        tcg.linear(h, x, w, out_dtype=F32)
        tcg.linear_cross_entropy(h, x, w, target)
        tcg.check(tcg.tcg_set_debug(h.h, 0, 0))
        out = tcg.linear(h, x, w, out_dtype=F32)
        again = tcg.linear_cross_entropy(h, x, w, target)[0]
        assert tcg.tcg_get_device_error(h.h) == tcg.TCG_STATUS_TIMEOUT
        assert same_bits(out, want) and same_bits(again, loss)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


def test_inputs_of_another_stream_may_be_dropped(cuda_device):
    """The caller drops an input while the handle's stream has yet to read it."""
    x, w, want = cut_product(8)
    side = torch.cuda.Stream()
    out = torch.empty(20, 512, dtype=F32, device="cuda")
    h = tcg.Handle(side)
    tcg.linear(h, x, w, out=out)
    spare = [torch.full_like(a, 0.0) for a in (x, w) for _ in range(6)]   # memory that torch has in hand
    del spare
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    x2, w2 = x.clone(), w.clone()
    torch.cuda.current_stream().synchronize()               # the inputs are ready
    tcg.linear(h, x2, w2, out=out)
    del x2, w2
    other = [torch.full_like(a, float("nan")) for a in (x, w) for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    assert not side.query()
    side.synchronize()
    assert same_bits(out, want)
    del other
    h.close()
