"""Prepared forward calls that split K, replayed on streams other than the one they were prepared on: the workspace that
belongs to the call is ready on each of them, and outlives the call as long as they need it."""
import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp

from gpu_helpers import announce, bits, require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def setup_module(_):
    require_gpu()


def case(M, K, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    X, W, W2 = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((M, K), (K, N), (K, N)))
    out = torch.empty((M, N), dtype=BF16, device="cuda")
    assert tp.tp_linear_ws(X, W).numel() > 0 and tp.tp_gated_linear_ws(X, W).numel() > 0     # K is split
    return X, W, W2, out


def busy(stream):
    """Work ahead of what follows on `stream`."""
    a = torch.ones((4096, 4096), dtype=BF16, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(20):
            b = a @ a
        a.record_stream(stream)
        del b


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("shape", [(3, 4096, 256), (64, 4096, 192)])
def test_replays_on_another_stream(shape, gated):
    announce(f"prepared on one stream, replayed on another: {shape} gated {gated}")
    X, W, W2, out = case(*shape)
    if gated:
        tp.tp_gated_linear(X, W, W2, out, ws=tp.tp_gated_linear_ws(X, W))
    else:
        tp.tp_linear(X, W, out, ws=tp.tp_linear_ws(X, W))
    want = bits(out)
    side = torch.cuda.Stream()
    # Ordered on the inputs alone; the memory that the workspace gets was written just before.
    torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    call = (tp.tp_gated_linear(X, W, W2, out, prepare=True) if gated else tp.tp_linear(X, W, out, prepare=True))
    for s in (side, torch.cuda.Stream(), side, None):
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        call(*([] if s is None else [s]))
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), want)


def test_a_call_dropped_while_its_stream_runs():
    announce("a prepared call dropped before its stream got to it")
    X, W, _, out = case(3, 4096, 256)
    ws = tp.tp_linear_ws(X, W)
    tp.tp_linear(X, W, out, ws=ws)
    want = bits(out)
    n = ws.numel()
    out.fill_(float("nan"))
    side = torch.cuda.Stream()
    busy(side)
    tp.tp_linear(X, W, out, prepare=True)(side)
    others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert np.array_equal(bits(out), want)
    assert all(bool((t == 255).all()) for t in others)


def test_prepared_inside_and_outside_a_capture():
    announce("prepared calls and captures")
    X, W, _, out = case(3, 4096, 256)
    tp.tp_linear(X, W, out, ws=tp.tp_linear_ws(X, W))
    split = bits(out)
    tp.tp_linear(X, W, out)
    whole = bits(out)
    before = tp.tp_linear(X, W, out, prepare=True)
    inside = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        before(torch.cuda.current_stream())
        call = tp.tp_linear(X, W, inside, prepare=True)     # without a workspace: K is not split
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        inside.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), split) and np.array_equal(bits(inside), whole)
        before()
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert np.array_equal(bits(out), split) and np.array_equal(bits(inside), whole)
