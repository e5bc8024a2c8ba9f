"""The cross entropy's gradients where targets are drawn from the model's own probabilities.

dz is rounded to bf16 for both products, divided by the one dloss first: a target that the model thinks unlikely is then an
entry near -1, of which little is lost, but 1 - p of a likely one is any number.  A rounding is at most U = 2^-8 of its entry and
uniform within that, so U / sqrt(3) of it in the root mean square at most; entries' roundings do not know of each other, nor
of W's columns and X's rows, which are independent here, so the 2-norm of the error of dX and dW is at most U / sqrt(3) of
theirs.  A bf16 result adds as much again of its own (in squares).  A quarter is allowed for the draw.
"""
import numpy as np
import pytest
import torch

from oracle import loss as O

from gpu_helpers import announce, require_gpu
from test_gpu_ce import BF16, F32, LINEAR, MATH, backward, f64, half, lse_for

pytestmark = pytest.mark.gpu


def setup_module(_):
    require_gpu()


def likely(M, K, V, dtype, std, seed):
    """X, W, targets drawn from softmax(X W), and their mean probability."""
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((M, K), generator=g).to(dtype)
    W = (torch.randn((K, V), generator=g) * (std / K ** 0.5)).to(dtype)
    p = torch.softmax(X.double() @ W.double(), 1)
    t = torch.multinomial(p, 1, generator=g)[:, 0]
    return X, W, t, float(p.gather(1, t[:, None]).mean())


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("std", [1.0, 4.0, 6.0, 9.0])
@pytest.mark.parametrize("shape", [(400, 512, 2000), (700, 256, 4100)], ids=str)
def test_likely_targets(shape, std, layout):
    X, W, t, p = likely(*shape, BF16, std, seed=int(std))
    announce(f"ce likely targets {shape} layout {layout} std {std}: mean probability {p:.2f}")
    lse = lse_for(X, W)
    want = O.cross_entropy_backward(f64(X), f64(W), t.numpy(), f64(lse), g=1 / shape[0])
    for out, roundings in ((BF16, 2), (F32, 1)):
        got = backward(X, W, t, lse, layout, g=torch.full((1,), 1 / shape[0]), dx=out, dw=out)
        for k in ("dX", "dW"):
            off = np.linalg.norm(f64(got[k]) - want[k]) / np.linalg.norm(want[k])
            print(f"[off] {k} {out} p {p:.2f}: {off:.2e}")
            assert off <= 1.25 * half(BF16) * (roundings / 3) ** 0.5, (k, out, off)


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("std", [4.0, 9.0])
def test_likely_targets_in_fp32(std, layout):
    """Nothing is rounded to fewer bits there: (K / 32 + 64) u of the sizes that were added, a logit's error in dz among them."""
    X, W, t, p = likely(300, 256, 1500, F32, std, seed=3)
    lse = lse_for(X, W)
    want = O.cross_entropy_backward(f64(X), f64(W), t.numpy(), f64(lse), g=1 / 300)
    got = backward(X, W, t, lse, layout, g=torch.full((1,), 1 / 300))
    u = half(F32)
    dq = (256 / 32 + 33) * u * (np.abs(f64(X)) @ np.abs(f64(W))) + 4 * u * (1 + np.abs(f64(lse))[:, None] + np.abs(f64(X) @ f64(W)))
    each = 1.01 * dq * want["q"] / 300 + 8 * u * np.abs(want["dz"])
    for k, tol, size in (("dX", each @ np.abs(f64(W)).T, np.abs(want["dz"]) @ np.abs(f64(W)).T), ("dW", np.abs(f64(X)).T @ each, np.abs(f64(X)).T @ np.abs(want["dz"]))):
        assert (np.abs(f64(got[k]) - want[k]) <= tol + (1500 / 32 + 64) * u * size + 1e-37).all(), k
