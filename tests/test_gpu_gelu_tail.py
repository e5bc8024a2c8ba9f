"""GeLU (erf) and its derivative in fp32, element by element over the whole range, against 64 bits.

Each value is one product x * 1, so the pre-activation is x itself.  With u = 2^-24, the lower tail q = Phi(-|x|) is
relatively within (20 + 1.5 x^2) u: the fitted polynomial and its evaluation (reciprocal 1 ulp, eight fused steps of a sum
whose terms reach three times its value, coefficients rounded) 13 u, the products and exp2's own ulp 5 u, and exp2's argument,
rounded three times, x^2 log2(e) / 2 * ln 2 * 2.5 u.  x q or x (1 - q) adds two roundings; the derivative Phi + x phi adds
phi's (5 + 1.5 x^2) u and three roundings.  Results below the smallest normal number may be zero.
"""
import math

import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp

from gpu_helpers import announce, require_gpu

pytestmark = pytest.mark.gpu

F32 = torch.float32
U, TINY = 2.0 ** -24, 2.0 ** -126


def setup_module(_):
    require_gpu()


def values(n):
    x = np.concatenate([np.linspace(-15, 15, n - 2003), np.linspace(-1e-3, 1e-3, 2000), [0.0, 40.0, -40.0]])
    return torch.from_numpy(x).to(F32)


def forms(x):
    x = x.double().numpy()
    q = 0.5 * np.array([math.erfc(abs(v) / math.sqrt(2.0)) for v in x])
    cdf = np.where(x >= 0, 1.0 - q, q)
    pdf = np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    return x, q, cdf, pdf


def near(got, ref, tol, name):
    off = np.abs(got.cpu().double().numpy().reshape(-1) - ref) - tol
    assert (off <= 0).all(), f"{name}: worst {np.max(off):.3g} past the tolerance"


@pytest.mark.parametrize("few", [True, False])
def test_forward(few):
    announce(f"gelu, fp32, {'few rows' if few else 'tiles'}")
    x = values(20_000)
    one = torch.ones((1, 1), device="cuda")
    if few:      # one token, the values in the weight's columns
        out = torch.empty((1, x.numel()), device="cuda")
        tp.tp_linear(one, x.cuda().view(1, -1), out, act=tp.TP_ACT_GELU_ERF)
    else:
        out = torch.empty((x.numel(), 1), device="cuda")
        tp.tp_linear(x.cuda().view(-1, 1), one, out, act=tp.TP_ACT_GELU_ERF)
    torch.cuda.synchronize()
    v, q, cdf, _ = forms(x)
    near(out, v * cdf, U * (np.abs(v) * q * (20 + 1.5 * v * v) + 2 * np.abs(v * cdf)) + 2 * np.maximum(1, np.abs(v)) * TINY, "gelu")


def test_derivative():
    announce("gelu's derivative, fp32")
    x = values(20_000)
    one, d = torch.ones((1, 1), device="cuda"), torch.ones((x.numel(), 1), device="cuda")
    dX = torch.empty((x.numel(), 1), device="cuda")
    ws = tp.tp_linear_backward_ws(d, one, d, act=tp.TP_ACT_GELU_ERF)
    tp.tp_linear_backward(d, one, d, pre=x.cuda().view(-1, 1), dX=dX, act=tp.TP_ACT_GELU_ERF, ws=ws)
    torch.cuda.synchronize()
    v, q, cdf, pdf = forms(x)
    ref = cdf + v * pdf
    tol = U * (q * (20 + 1.5 * v * v) + cdf + np.abs(v) * pdf * (5 + 1.5 * v * v) + 3 * np.abs(ref))
    near(dX, ref, tol + 4 * np.maximum(1, np.abs(v)) * TINY, "derivative")
