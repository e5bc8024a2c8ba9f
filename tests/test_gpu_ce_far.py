"""The vocabulary cross entropy where logits or log-sum-exps are far from zero: entries masked by a weight's large negative
value, whole tiles of them, and rows that lie far away as a whole.

Rows of X hold ones and zeros, so that a logit is a sum of few weights, exact in fp32, and the tolerances count only what
comes after it: lse's own rounding and a few u of the sum; of a probability the exponent's rounding and exp2 (4 u (1 +
|z - lse|)), dz's half a step and the products' sums.
"""
import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import loss as O

from gpu_helpers import announce, require_gpu
from test_gpu_ce import BF16, F32, LINEAR, MATH, U, backward, f64, forward, half

pytestmark = pytest.mark.gpu

# Up to bf16's largest value; products with log2 e round up and down among them.
FAR = [1e8, 1.1e9, 2.0 ** 30, 2.5e9, 4.1e9, 1e10, 3.3e10, 7e10, 1e12, 1e20, 1e30, 3e30, 2e38, 3.3e38, torch.finfo(BF16).max]


def setup_module(_):
    require_gpu()


def lse_close(got, want):
    assert np.isfinite(f64(got)).all()
    assert (np.abs(f64(got) - want) <= 64 * U + 4 * U * np.abs(want)).all()


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 40, 600])
def test_masked_entries(M, dtype, layout):
    """Most of the vocabulary masked, in whole tiles and in parts of them: as if it were not there."""
    K, V = 64, 2100
    g = torch.Generator().manual_seed(M)
    for far in FAR:
        announce(f"ce masked {M} {dtype} layout {layout} by {far:g}")
        X = torch.zeros((M, K))
        X[:, 0] = 1
        X[torch.arange(M), 1 + torch.arange(M) % (K - 1)] = 1
        W = torch.randn((K, V), generator=g)
        W[0] = 0
        W[0, :1600] = -far * (1 + 0.3 * torch.rand(1600, generator=g))     # of different sizes ..
        W[0, 256:1024] = -far                                              # .. and alike
        W[0, 3:1600:500] = 0
        W = W.clamp(-torch.finfo(BF16).max, torch.finfo(BF16).max)
        X, W = X.to(dtype), W.to(dtype)
        t = 1600 + torch.arange(M) % 500
        want = O.cross_entropy(f64(X), f64(W), t.numpy())
        got = forward(X, W, t, layout)
        lse_close(got["lse"], want["lse"])
        assert (np.abs(f64(got["loss"]) - want["loss"]) <= 64 * U + 8 * U * (np.abs(want["lse"]) + np.abs(want["loss"]))).all()
        # A masked target has its own logit's loss, and a piece that is masked as a whole its own statistics.
        t = 300 + torch.arange(M) % 500
        part = forward(X, W[:, 256:1024].contiguous(), t, layout, begin=256)
        whole = O.cross_entropy(f64(X), f64(W[:, 256:1024]), t.numpy(), begin=256)
        lse_close(part["lse"], whole["lse"])
        assert (np.abs(f64(part["stats"][0]) - whole["stats"][0]) <= 2 * U * np.abs(whole["stats"][0])).all()
        assert ((f64(part["stats"][1]) >= 1 - 64 * U) & (f64(part["stats"][1]) <= 768 * (1 + 64 * U))).all()
        rest = forward(X, W[:, 1600:].contiguous(), t, layout, begin=1600)
        lse = torch.empty(M, device="cuda")
        tp.tp_ce_join(torch.stack([part["stats"], rest["stats"]]), t.cuda(), lse=lse)
        lse_close(lse, O.cross_entropy(f64(X), f64(torch.cat([W[:, 256:1024], W[:, 1600:]], 1)), np.zeros(M, np.int64))["lse"])


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 40, 600])
def test_rows_far_away(M, dtype, layout):
    """Every logit of a row large: one or a few of them carry the sum, and their loss is ln of how many."""
    K, V = 64, 1300
    for far in FAR:
        for sign in (1, -1):
            announce(f"ce far {M} {dtype} layout {layout} {sign * far:g}")
            # Steps of 2^-7 of the value, which bf16 holds: at 1e8 and more, e^-(a step) is nothing.
            step = 2.0 ** (np.floor(np.log2(far)) - 7)
            z = sign * far - step * (torch.arange(V) % 100)
            z[torch.arange(V) % 100 == 0] = z[0]
            z = z.clamp(-torch.finfo(BF16).max, torch.finfo(BF16).max)
            W = torch.zeros((K, V))
            W[0] = z
            X = torch.zeros((M, K))
            X[:, 0] = 1
            X, W = X.to(dtype), W.to(dtype)
            t = torch.arange(M) % 100
            want = O.cross_entropy(f64(X), f64(W), t.numpy())
            got = forward(X, W, t, layout)
            lse_close(got["lse"], want["lse"])
            loss = f64(got["loss"])
            ok = np.abs(want["loss"]) < 3e38
            assert (np.abs(loss - want["loss"])[ok] <= 64 * U + 8 * U * (np.abs(want["lse"]) + np.abs(want["loss"]))[ok]).all()
            assert (np.abs(f64(got["stats"][1]) - want["stats"][1]) <= 64 * U * want["stats"][1]).all()


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 600])
@pytest.mark.parametrize("base", [0.0, 1.25 * 2 ** 12, 1.25 * 2 ** 16, -1.25 * 2 ** 20, 1.25 * 2 ** 20, 2.0 ** 30, -1e20, 3e38])
def test_gradients_of_far_rows(base, M, dtype, layout):
    """e^(z - lse) of the lse that is given, however large both are."""
    announce(f"ce far backward {M} {dtype} layout {layout} {base:g}")
    K, V = 64, 700
    g = torch.Generator().manual_seed(M)
    unit = max(2.0 ** -7, 2.0 ** (np.floor(np.log2(abs(base))) - 23) * 8) if base else 2.0 ** -7
    X = torch.zeros((M, K))
    X[:, 0] = X[:, 1] = 1
    W = torch.randn((K, V), generator=g)
    W[0] = base
    # A few units of what fp32 resolves there (bf16 holds them); a spread of a few e-folds where that is possible.
    W[1] = -unit * torch.randint(0, 100 if unit < 1 else 2, (V,), generator=g) * (0.0625 / unit if unit < 0.0625 else 1)
    W[1, 7] = 0
    X, W = X.to(dtype), W.to(dtype)
    z = f64(X) @ f64(W)
    assert (z == z.astype(np.float32)).all()
    lse = torch.from_numpy(O.lse_of(z)).float()
    t = torch.arange(M) % V
    t[1] = -100
    want = O.cross_entropy_backward(f64(X), f64(W), t.numpy(), f64(lse))
    got = backward(X, W, t, lse, layout, dx=F32, dw=F32)
    near = np.abs(np.maximum(z - f64(lse)[:, None], -200))
    each = 4 * U * (1 + near) * want["q"] + (half(dtype) + 4 * U) * np.abs(want["dz"]) + torch.finfo(dtype).smallest_normal
    Xo = np.abs(f64(X)) * (t.numpy() != -100)[:, None]
    # dX without the two columns that only place the rows.
    for name, tol, cut in (("dX", each @ np.abs(f64(W)).T + (V / 32 + 64) * U * np.abs(want["dz"]) @ np.abs(f64(W)).T, np.s_[:, 2:]),
                           ("dW", Xo.T @ each + (M / 32 + 64) * U * Xo.T @ np.abs(want["dz"]), np.s_[:, :])):
        err = np.abs(f64(got[name]) - want[name])[cut]
        assert (err <= (tol + 2 * U * np.abs(want[name]) + 1e-37)[cut]).all(), (name, float(np.max(err / (tol[cut] + 1e-37))))
