"""The vocabulary cross entropy at the least widths and vocabularies, of few and of many tokens (tolerances as in
test_gpu_ce.py)."""
import pytest
import torch

from gpu_helpers import announce, require_gpu
from test_gpu_ce import BF16, F32, LINEAR, MATH, backward, check_backward, check_forward, f64, forward, lse_for, make

pytestmark = pytest.mark.gpu


def setup_module(_):
    require_gpu()


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("K,V", [(1, 1), (1, 2), (2, 1), (3, 700), (7, 65), (9, 1), (1, 3001), (31, 63), (40, 2)])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 127, 128, 600, 1100])
def test_tiny(M, K, V, dtype, layout):
    announce(f"ce tiny {M} x {K} -> {V} {dtype} layout {layout}")
    X, W, t = make(M, K, V, dtype, seed=M + 10 * K + V)
    check_forward(X, W, t, forward(X, W, t, layout), dtype)
    lse = lse_for(X, W)
    g = torch.rand(M, generator=torch.Generator().manual_seed(1)) / M
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=g), g=f64(g))
