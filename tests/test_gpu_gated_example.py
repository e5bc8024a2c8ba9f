"""The gated feed-forward example: its gradients against the float64 forms chained by hand, a falling loss, and
tokens served singly against the batch."""
import os
import sys

import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import linear as O

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BF16 = torch.bfloat16
U = torch.finfo(BF16).eps / 2


def setup_module(_):
    require_gpu()


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, ref, steps):
    """2-norm: `steps` independent roundings to bf16 on the way, each at most U relative."""
    assert np.linalg.norm(f64(got) - ref) <= steps * U * np.linalg.norm(ref)


@pytest.mark.parametrize("tokens,width,inner", [(1, 64, 96), (77, 120, 200), (256, 256, 384)])
def test_one_step(tokens, width, inner):
    import gated_ffn_step as ex
    block = ex.GatedFFN(tokens, width, inner, 5)
    g = torch.Generator().manual_seed(6)
    x, d = torch.randn((tokens, width), generator=g).to(BF16), torch.randn((tokens, width), generator=g).to(BF16)
    xd, dd = x.cuda(), d.cuda()
    block.forward(xd)
    block.backward(xd, dd)
    w = {k: f64(v) for k, v in block.w.items()}
    y, gate, up = O.gated(f64(x), w["gate"], w["up"], O.SILU)
    out, _ = O.linear(y, w["down"], f64(block.main["bias"]), f64(x))
    close(block.out, out, 2)                  # y, out
    down = O.linear_backward(y, w["down"], f64(d))
    close(block.grads["down"], down["dW"], 2)     # y (fp32 gradient)
    assert np.allclose(f64(block.grads["bias"]), down["dbias"], rtol=0, atol=1e-5 * tokens)
    back = O.gated_backward(f64(x), w["gate"], w["up"], gate, up, down["dX"], O.SILU)
    # gate, up, dY and dGate / dUp are each rounded once on the way, and the activation's derivative and the
    # product pass the rounding of gate and up on twice.
    close(block.d_x, back["dX"], 6)
    close(block.grads["gate"], back["dWg"], 6)
    close(block.grads["up"], back["dWu"], 6)
    before = [t.clone() for t in block.grads.values()]
    norm = float(block.clip(0.01))
    want = np.sqrt(sum((f64(t) ** 2).sum() for t in before))
    assert abs(norm - want) <= 1e-6 * want
    for t, b in zip(block.grads.values(), before):
        assert np.allclose(f64(t), f64(b) * min(1.0, 0.01 / (want + 1e-6)), rtol=1e-6, atol=0)


def test_trains_and_serves():
    import gated_ffn_step as ex
    losses, norms, block, x = ex.train()
    assert losses[-1] < 0.9 * losses[0] and all(np.isfinite(losses)) and all(np.isfinite(norms))
    batch, single = block.forward(x)[:16].clone(), ex.serve(block, x[:16])
    torch.cuda.synchronize()
    # The same sums in another order: y may land on the neighbouring bf16 value, and so may out.
    close(single, f64(batch), 2)
