"""The next-token example over several steps: each one is AdamW's on the states that the one before left, and a step that is
left out because its gradients are not finite leaves no trace."""
import os
import sys

import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import loss as O

from gpu_helpers import bits, require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BF16 = torch.bfloat16
U = torch.finfo(torch.float32).eps / 2


def setup_module(_):
    require_gpu()


def f64(t):
    return t.detach().cpu().double().numpy()


def states(model):
    """m, v and (8 bits) their scales, as float64, by tensor."""
    if not model.scales:
        return [(f64(m), f64(v), None, None) for m, v in zip(model.m, model.v)]
    m, v = ([torch.empty(x.shape, device="cuda") for x in model.m] for _ in "mv")
    tp.tp_adamw_unpack(model.m, model.v, m, v, **model.scales)
    return [(f64(a), f64(b), f64(s), f64(r)) for a, b, s, r in zip(m, v, model.scales["m_scale"], model.scales["v_scale"])]


def everything(model):
    return [bits(x) for x in [*model.main.values(), *model.copies.values(), *model.m, *model.v, *sum(model.scales.values(), []), model.count]]


def spread(scale, shape):
    n = int(np.prod(shape))
    return np.repeat(scale, O.BLOCK)[:n].reshape(shape)


@pytest.mark.parametrize("kw", [dict(), dict(pieces=4), dict(eight=True)])
def test_each_step_goes_on_from_the_last(kw):
    """Weights and states after each of five steps, from those before it and its gradients, in float64.

    fp32: every operation is off by u, some ten of them to a term; m's two terms may cancel, so their sizes count.  8 bits:
    a code is the nearest of its square law (c + 1/4 of scale / top^2 away in the value at code c, and a root that is not
    zero at most one code)."""
    import next_token_step as ex
    model = ex.NextToken(200, 96, 160, 600, max_norm=0.5, seed=2, **kw)
    ids, targets = ex.data(200, 600, 1)
    b1, b2, rate = 0.9, 0.999, 1e-2
    for step in range(1, 6):
        model.forward(ids, targets)
        model.backward(targets)
        before, p0 = states(model), {k: f64(v) for k, v in model.main.items()}
        g = {k: f64(v) for k, v in model.grads.items()}
        norm = np.sqrt(sum((x ** 2).sum() for x in g.values()))
        factor = min(1.0, 0.5 / (norm + 1e-6))
        model.step(rate)
        torch.cuda.synchronize()
        assert int(model.count) == step
        for (k, w), (m0, v0, _, _), (m1, v1, ms, vs) in zip(model.main.items(), before, states(model)):
            decay = 0.0 if k == "bias" else 0.01
            p, m, v = O.adamw(p0[k], g[k], m0, v0, step=step, lr=rate, decay=decay, factor=factor)
            sizes = b1 * np.abs(m0) + (1 - b1) * factor * np.abs(g[k])
            move = rate * sizes / (1 - b1 ** step) / (np.sqrt(v / (1 - b2 ** step)) + 1e-8)
            assert (np.abs(f64(w) - p) <= 64 * U * move + 2.5 * U * np.abs(p) + 1e-30).all(), (step, k)
            if ms is None:
                assert (np.abs(m1 - m) <= 8 * U * sizes + 1e-37).all() and (np.abs(v1 - v) <= 16 * U * v + 1e-37).all(), (step, k)
            else:
                r, sm, sr = np.sqrt(v), spread(ms, m.shape), spread(vs, v.shape)
                cm, cr = 127 * np.sqrt(np.abs(m) / np.maximum(sm, 1e-30)), 255 * np.sqrt(r / np.maximum(sr, 1e-30))
                assert (np.abs(m1 - m) <= 1.01 * sm * (cm + 0.25) / 127 ** 2 + 8 * U * sizes + 1e-30).all(), (step, k)
                assert (np.abs(np.sqrt(v1) - r) <= 1.01 * sr * np.maximum(cr + 0.25, 1) / 255 ** 2 + 16 * U * r + 1e-18).all(), (step, k)
            if k in model.copies:
                assert torch.equal(model.copies[k], w.to(BF16)), k


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
