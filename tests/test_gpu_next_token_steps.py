"""The next-token example over several steps: one that is left out because its gradients are not finite leaves no trace."""
import os
import sys

import numpy as np
import pytest
import torch

from gpu_helpers import bits, require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def setup_module(_):
    require_gpu()


def everything(model):
    return [bits(x) for x in [*model.main.values(), *model.copies.values(), *model.m, *model.v, *sum(model.scales.values(), []), model.count]]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_that_is_left_out(bad, eight):
    """Before the first step and between others: nothing moves, the count neither, and the next step is the one that would have been."""
    import next_token_step as ex
    a, b = (ex.NextToken(64, 64, 96, 400, seed=6, eight=eight) for _ in range(2))
    ids, targets = ex.data(64, 400, 2)
    for step in range(1, 4):
        for m in (a, b):
            m.forward(ids, targets)
            m.backward(targets)
        kept, was = a.grads["head"].clone(), everything(a)
        a.grads["head"][7, 3] = bad
        norm = float(a.step(1e-2))
        assert not np.isfinite(norm)
        assert all(np.array_equal(x, y) for x, y in zip(everything(a), was))
        a.grads["head"].copy_(kept)
        a.step(1e-2)
        b.step(1e-2)
        torch.cuda.synchronize()
        assert int(a.count) == int(b.count) == step
        assert all(np.array_equal(x, y) for x, y in zip(everything(a), everything(b)))


def test_a_captured_step_that_is_left_out():
    import next_token_step as ex
    a, b = (ex.NextToken(64, 64, 96, 400, seed=6) for _ in range(2))
    ids, targets = ex.data(64, 400, 2)
    rate = torch.full((1,), 1e-2, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):      # (torch's own lazy set-up, outside the capture)
        ex.NextToken(64, 64, 96, 400, seed=6).step(rate)
    torch.cuda.synchronize()
    for m in (a, b):
        m.forward(ids, targets)
        m.backward(targets)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(rate)
    kept = a.grads["head"].clone()
    taken = 0
    for bad in (True, False, True, True, False, False):
        a.grads["head"].copy_(kept)
        if bad:
            a.grads["head"][0, 0] = float("nan")
        graph.replay()
        torch.cuda.synchronize()
        if not bad:
            b.step(rate)
            taken += 1
        torch.cuda.synchronize()
        assert int(a.count) == taken
        assert all(np.array_equal(x, y) for x, y in zip(everything(a), everything(b)))
