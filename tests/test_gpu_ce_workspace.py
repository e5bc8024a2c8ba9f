"""One workspace of the vocabulary cross entropy for a batch and for every smaller one, each checked as a call of its own
(test_gpu_ce.py has the tolerances)."""
import pytest
import torch

import sharded_gemm_amd as tp

from gpu_helpers import announce, bits, require_gpu
from test_gpu_ce import BF16, F32, LINEAR, MATH, check_forward, forward, lay, make

pytestmark = pytest.mark.gpu


def setup_module(_):
    require_gpu()


# Sizes whose few tokens need more than the full batch: split K, twice the pairs, logits (fp32).
@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype,full,K,V,tokens", [(BF16, 1024, 1024, 4096, (300, 1, 1023)), (BF16, 100, 256, 40_000, (64, 65, 16)), (BF16, 2100, 512, 8192, (1, 64, 700)),
                                                   (BF16, 600, 519, 3001, (511, 512, 30)), (F32, 500, 256, 20_000, (16, 17, 1)), (F32, 300, 640, 1500, (64, 1, 129))])
def test_ragged_batches(dtype, full, K, V, tokens, layout):
    X, W, t = make(full, K, V, dtype, seed=full + K)
    Xd, Wd = X.cuda(), lay(W, layout)
    ws = tp.tp_linear_ce_ws(Xd, Wd, weight_layout=layout)
    for M in (full, *tokens, full):
        announce(f"ce {M} of {full} tokens, {K} -> {V} {dtype} layout {layout}")
        got = forward(X[:M], W, t[:M], layout, Xd=Xd[:M], Wd=Wd, ws=ws)
        check_forward(X[:M], W, t[:M], got, dtype)
        own = forward(X[:M], W, t[:M], layout, Xd=Xd[:M], Wd=Wd)
        assert all((bits(got[k]) == bits(own[k])).all() for k in got)


def test_smaller_batches_in_graphs():
    """A full batch, a ragged one and a token, captured on one workspace and replayed in turn."""
    full, K, V = 1024, 256, 4096
    X, W, t = make(full, K, V, BF16, seed=7)
    Xd, Wd, td = X.cuda(), lay(W, LINEAR), t.cuda()
    ws = tp.tp_linear_ce_ws(Xd, Wd, weight_layout=LINEAR)
    graphs = []
    for M in (full, 300, 1):
        loss = torch.empty(M, device="cuda")
        call = tp.tp_linear_ce(Xd[:M], Wd, td[:M], loss=loss, weight_layout=LINEAR, ws=ws, prepare=True)
        call()
        torch.cuda.synchronize()
        want = bits(loss)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(torch.cuda.current_stream())
        graphs.append((graph, loss, want))
    for _ in range(3):
        for _, loss, _ in graphs:
            loss.fill_(float("nan"))
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all((bits(loss) == want).all() for _, loss, want in graphs)
