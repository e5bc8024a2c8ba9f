"""The next-token example: a step's gradients against the float64 forms chained by hand, its update against AdamW's
formula on the gradients it made, pieces of the vocabulary against the whole, tokens scored singly against the batch."""
import os
import sys

import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import linear as L
from oracle import loss as O

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BF16 = torch.bfloat16
U = torch.finfo(BF16).eps / 2
U32 = torch.finfo(torch.float32).eps / 2


def setup_module(_):
    require_gpu()


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, ref, steps):
    """2-norm: `steps` independent roundings to bf16 on the way, each at most U relative."""
    assert np.linalg.norm(f64(got) - ref) <= steps * U * np.linalg.norm(ref)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("tokens,width,inner,vocab,pieces", [(1, 64, 96, 200, 1), (77, 120, 200, 1000, 4), (256, 128, 192, 5000, 2)])
def test_one_step(tokens, width, inner, vocab, pieces, eight):
    import next_token_step as ex
    model = ex.NextToken(tokens, width, inner, vocab, pieces=pieces, eight=eight, max_norm=0.1)
    ids, targets = ex.data(tokens, vocab, 3)
    targets[0] = 5
    model.forward(ids, targets)
    model.backward(targets)
    t = targets.cpu().numpy()
    w = {k: f64(v) for k, v in model.copies.items()}
    x = f64(model.embedding[ids])
    y, gate, up = L.gated(x, w["gate"], w["up"], L.SILU)
    h, _ = L.linear(y, w["down"], f64(model.main["bias"]), x)
    ce = O.cross_entropy(h, w["head"].T, t)
    # A loss moves by at most its logits' range times h's and y's two roundings: near its 2-norm bound
    # |dh| |w| with |dh| <= 2 U |h|.
    reach = 2 * 3 * U * np.linalg.norm(h, axis=1) * np.linalg.norm(w["head"], axis=1).max()
    assert (np.abs(f64(model.loss) - ce["loss"]) <= reach + 1e-5 * (1 + np.abs(ce["loss"]))).all()
    # The rest from the block's own output on: its roundings are the block's test's.
    h = f64(model.block.out)
    lse = O.cross_entropy(h, w["head"].T, t)["lse"]
    back = O.cross_entropy_backward(h, w["head"].T, t, lse, g=1.0 / max(1, (t != -100).sum()))
    close(model.d_out, back["dX"], 3)                      # dz, the sum, d_out
    close(model.grads["head"], back["dW"].T, 2)            # dz (fp32 gradient)
    down = L.linear_backward(f64(model.block.y), w["down"], f64(model.d_out))
    close(model.grads["down"], down["dW"], 1)
    block = L.gated_backward(x, w["gate"], w["up"], f64(model.block.gate), f64(model.block.up), f64(model.block.d_y), L.SILU)
    close(model.grads["gate"], block["dWg"], 2)
    close(model.grads["up"], block["dWu"], 2)
    # The update, from these gradients.
    before = {k: f64(v) for k, v in model.main.items()}
    grads = {k: f64(v) for k, v in model.grads.items()}
    norm = float(model.step(1e-2))
    want = np.sqrt(sum((g ** 2).sum() for g in grads.values()))
    assert abs(norm - want) <= 1e-6 * want and int(model.count) == 1
    factor = min(1.0, 0.1 / (want + 1e-6))
    for k, v in model.main.items():
        decay = 0.0 if k == "bias" else 0.01
        p, _, _ = O.adamw(before[k], grads[k], 0 * grads[k], 0 * grads[k], step=1, lr=1e-2, decay=decay, factor=factor)
        # The first step moves by lr sign(g): a few u of it, more where g is near eps (g / (|g| + eps)).
        assert np.allclose(f64(v), p, rtol=2e-7, atol=1e-2 * 64 * U32), k
        if k in model.copies:
            assert torch.equal(model.copies[k], v.to(BF16)), k


@pytest.mark.parametrize("kw", [dict(), dict(pieces=4), dict(eight=True)])
def test_trains_and_scores(kw):
    import next_token_step as ex
    losses, norms, model = ex.train(steps=5, **kw)
    assert all(np.isfinite(losses)) and all(np.isfinite(norms)) and int(model.count) == 5
    ids, targets = ex.data(512, 1000)
    batch = model.forward(ids, targets)[:16].clone()
    single = ex.score(model, model.block.out[:16], targets[:16])
    torch.cuda.synchronize()
    # The same logits in another order of their sums.
    assert np.allclose(f64(single), f64(batch), rtol=0, atol=1e-4)


def test_a_step_in_a_graph():
    """Forward, backward, norm and update captured together: every replay is the eager step."""
    import next_token_step as ex
    ids, targets = ex.data(128, 600, 1)
    a, b = (ex.NextToken(128, 64, 96, 600, seed=4) for _ in range(2))
    rate = torch.full((1,), 1e-2, device="cuda")
    count = (targets != -100).sum().clamp(min=1).float().reciprocal()

    def step(m):
        m.forward(ids, targets)
        tp.tp_linear_ce_backward(m.block.out, m.copies["head"], targets, m.lse, dloss=count, dX=m.d_out, dW=m.grads["head"],
                                 weight_layout=ex.LINEAR, ws=m.bws)
        m.block.backward(m.x, m.d_out)
        m.step(rate)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):      # (torch's own lazy set-up, outside the capture)
        step(ex.NextToken(128, 64, 96, 600, seed=5))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for t in range(1, 4):
        rate.fill_(1e-2 / t)
        graph.replay()
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        assert int(a.count) == int(b.count) == t
        assert torch.equal(a.loss, b.loss)
        for k in a.main:
            assert torch.equal(a.main[k], b.main[k]) and torch.equal(a.grads[k], b.grads[k]), (t, k)
