"""4-bit products of many tokens, whose weights are expanded in the workspace: in memory of the caller's
of just the size asked for, in captured graphs, on streams of their own, and after a wait that ran out."""
import pytest
import torch

import mixed_precision_tensor_gb300 as tcg
from test_gpu_ffn import draw_4bit
from test_gpu_lm import gen_of, randn, same_bits

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# (tokens, features, k, gated, zeros): whole tiles and pieces
CASES = [(500, 264, 520, True, False), (300, 264, 4128, True, True), (200, 520, 4104, False, True),
         (700, 136, 1032, False, False)]


def data(t, n, k, gated, zeros, seed=1):
    g = gen_of(seed)
    w, scales, zero = draw_4bit(g, 2 * n if gated else n, k, 32, BF16, zeros)
    return {"x": randn(g, t, k), "w": w, "scales": scales, "zeros": zero,
            "out": torch.zeros(t, -(-n // 8) * 8, dtype=BF16, device="cuda")[:, :n]}


def call(h, s, gated, out=None):
    return tcg.linear_4bit(h, s["x"], s["w"], s["scales"], 32, zeros=s["zeros"], act="silu" if gated else "none",
                           gated=gated, out=s["out"] if out is None else out)


@pytest.mark.parametrize("t,n,k,gated,zeros", CASES)
def test_given_workspace_is_enough(cuda_device, t, n, k, gated, zeros):
    """Guarded on both sides, and full of NaN before the call."""
    h = tcg.Handle()
    s = data(t, n, k, gated, zeros)
    want = call(h, s, gated).clone()
    size = tcg.tcg_gemm_4bit_workspace_size(h.h, n, t, k, gated)
    assert size > 0
    room = torch.full((size + 512,), 255, dtype=torch.uint8, device="cuda")
    own = tcg.Handle()
    tcg.check(tcg.tcg_set_workspace(own.h, room.data_ptr() + 256, size))
    assert same_bits(call(own, s, gated), want)
    torch.cuda.synchronize()
    assert (room[:256] == 255).all() and (room[256 + size:] == 255).all()
    tcg.check(tcg.tcg_set_workspace(own.h, room.data_ptr() + 256, size - 256))
    with pytest.raises(tcg.TcgError):
        call(own, s, gated)
    h.close()
    own.close()


@pytest.mark.parametrize("t,n,k,gated,zeros", CASES)
def test_captured_and_replayed(cuda_device, t, n, k, gated, zeros):
    """Two graphs of one handle, replayed in turn, share its workspace."""
    h = tcg.Handle()
    sets = [data(t, n, k, gated, zeros, seed) for seed in (2, 3)]
    want = [call(h, s, gated).clone() for s in sets]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    h.set_stream(stream)
    graphs = []
    for s in sets:
        s["out"].zero_()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            call(h, s, gated)
    for _ in range(3):
        for g in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert same_bits(s["out"], w)
    # new weights and scales in the same places
    for a in ("x", "w", "scales"):
        sets[0][a].copy_(sets[1][a])
    if zeros:
        sets[0]["zeros"].copy_(sets[1]["zeros"])
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert same_bits(sets[0]["out"], want[1])
    tcg.check(tcg.tcg_get_device_error(h.h))
    del graphs
    h.close()


@pytest.mark.parametrize("gated", [False, True])
def test_capture_does_not_grow_the_workspace(cuda_device, gated):
    stream = torch.cuda.Stream()
    h = tcg.Handle(stream)
    s = data(500, 264, 520, gated, True)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):                        # a handle's first call binds it to the device
        call(h, {**s, "x": s["x"][:1]}, gated, s["out"][:1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s["out"].zero_()
        with pytest.raises(tcg.TcgError) as e:
            call(h, s, gated)
    assert e.value.status == tcg.TCG_STATUS_ALLOC_FAILED
    del graph
    h.close()


def test_two_streams_at_once(cuda_device):
    streams = [torch.cuda.Stream() for _ in range(2)]
    plain, handles = tcg.Handle(), [tcg.Handle(s) for s in streams]
    sets = [data(*c) for c in CASES[:2]]
    want = [call(plain, s, True).clone() for s in sets]
    for s in sets:
        s["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for h, s in zip(handles, sets):
            call(h, s, True)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert same_bits(s["out"], w)
    for h in (*handles, plain):
        tcg.check(tcg.tcg_get_device_error(h.h))
        h.close()


def test_other_stream_and_dropped_inputs(cuda_device):
    side = torch.cuda.Stream()
    h, plain = tcg.Handle(side), tcg.Handle()
    s = data(500, 264, 1032, True, True)
    want = call(plain, s, True).clone()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    mine = {k: v.clone() for k, v in s.items() if k not in ("out", "w")} | {"w": s["w"], "out": None}
    side.wait_stream(torch.cuda.current_stream())
    out = tcg.linear_4bit(h, mine["x"], mine["w"], mine["scales"], 32, zeros=mine["zeros"], act="silu", gated=True)
    shapes = [mine[k].shape for k in ("x", "scales", "zeros")]
    del mine
    junk = [torch.full(sh, 7.0, dtype=BF16, device="cuda") for sh in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert same_bits(out, want) and junk
    h.close()
    plain.close()


@pytest.mark.parametrize("t,n,k,gated,zeros", CASES)
def test_wait_that_runs_out(cuda_device, t, n, k, gated, zeros):
    """A load that never comes ends the product with an error, and the next call is right."""
    h = tcg.Handle()
    s = data(t, n, k, gated, zeros)
    want = call(h, s, gated).clone()
    tcg.check(tcg.tcg_get_device_error(h.h))
    tcg.tcg_set_debug(h.h, 2_000_000, 1)
    call(h, s, gated)
    assert tcg.tcg_get_device_error(h.h) == tcg.TCG_STATUS_TIMEOUT
    tcg.tcg_set_debug(h.h)
    assert same_bits(call(h, s, gated), want)
    tcg.check(tcg.tcg_get_device_error(h.h))
    h.close()


@pytest.mark.parametrize("gated", [False, True])
def test_many_tokens_without_features_of_x(cuda_device, gated):
    h = tcg.Handle()
    x = torch.empty(300, 8, dtype=BF16, device="cuda")[:, :0]
    w = torch.empty(24, 16, dtype=torch.uint8, device="cuda")[:, :0]
    scales = torch.ones(24, 0, dtype=BF16, device="cuda")
    out = tcg.linear_4bit(h, x, w, scales, 32, gated=gated)
    assert out.shape == (300, 12 if gated else 24) and not out.any()
    h.close()
