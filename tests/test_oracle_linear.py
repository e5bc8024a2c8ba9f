"""The float64 forms of the linear layer, the gated block and clipping: gradients against central differences,
and values against hand-worked ones."""
import math

import numpy as np
import pytest

from oracle import linear as O

KINDS = [O.NONE, O.GELU_ERF, O.GELU_TANH, O.SILU, O.RELU]
STEP = 1e-5
# A central difference is off by STEP^2 f''' / 6 plus a rounding of f of about 2^-52 |f| / STEP; every f here is
# below 100 and its third derivative below 10.
TOL = 100 * (STEP ** 2 * 10 / 6 + 2.0 ** -52 * 100 / STEP)


def _difference(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += STEP
        lo[i] -= STEP
        g[i] = (f(hi) - f(lo)) / (2 * STEP)
    return g


@pytest.mark.parametrize("kind", KINDS)
def test_activation_gradient(kind):
    x = np.array([-6.0, -2.5, -1.0, -0.3, 0.4, 1.2, 3.0, 7.0])
    num = (O.act(kind, x + STEP) - O.act(kind, x - STEP)) / (2 * STEP)
    assert np.max(np.abs(num - O.act_grad(kind, x))) <= TOL


def test_activation_values():
    assert O.act(O.RELU, np.array([-1.0, 0.0, 2.0])).tolist() == [0.0, 0.0, 2.0]
    assert abs(O.act(O.SILU, np.array([1.0]))[0] - 1.0 / (1.0 + math.exp(-1.0))) < 1e-15
    assert abs(O.act(O.GELU_ERF, np.array([1.0]))[0] - 0.8413447460685429) < 1e-15
    assert abs(O.act(O.GELU_TANH, np.array([1.0]))[0] - 0.8411919906082768) < 1e-14


@pytest.mark.parametrize("kind", KINDS)
def test_linear_gradients(kind):
    r = np.random.default_rng(1)
    X, W, b, R, d = r.normal(size=(3, 4)), r.normal(size=(4, 5)), r.normal(size=5), r.normal(size=(3, 5)), r.normal(size=(3, 5))
    pre = O.linear(X, W, b, R, kind)[1]
    g = O.linear_backward(X, W, d, pre, kind)
    for name, x, f in (("dX", X, lambda v: (O.linear(v, W, b, R, kind)[0] * d).sum()),
                       ("dW", W, lambda v: (O.linear(X, v, b, R, kind)[0] * d).sum()),
                       ("dbias", b, lambda v: (O.linear(X, W, v, R, kind)[0] * d).sum())):
        assert np.max(np.abs(_difference(f, x) - g[name])) <= TOL, name
    assert np.max(np.abs(_difference(lambda v: (O.linear(X, W, b, v, kind)[0] * d).sum(), R) - d)) <= TOL


@pytest.mark.parametrize("kind", KINDS)
def test_gated_gradients(kind):
    r = np.random.default_rng(2)
    X, Wg, Wu, d = r.normal(size=(3, 4)), r.normal(size=(4, 5)), r.normal(size=(4, 5)), r.normal(size=(3, 5))
    _, gate, up = O.gated(X, Wg, Wu, kind)
    g = O.gated_backward(X, Wg, Wu, gate, up, d, kind)
    for name, x, f in (("dX", X, lambda v: (O.gated(v, Wg, Wu, kind)[0] * d).sum()),
                       ("dWg", Wg, lambda v: (O.gated(X, v, Wu, kind)[0] * d).sum()),
                       ("dWu", Wu, lambda v: (O.gated(X, Wg, v, kind)[0] * d).sum())):
        assert np.max(np.abs(_difference(f, x) - g[name])) <= TOL, name


def test_clip():
    norm, out = O.clip([np.array([3.0]), np.array([[4.0]])], 1.0, 0.0)
    assert norm == 5.0 and abs(out[0][0] - 0.6) < 1e-15 and abs(out[1][0, 0] - 0.8) < 1e-15
    norm, out = O.clip([np.array([0.3, 0.4])], 1.0)
    assert abs(norm - 0.5) < 1e-15 and out[0].tolist() == [0.3, 0.4]
    norm, out = O.clip([np.array([np.inf, 1.0])], 1.0)
    assert norm == np.inf and np.isnan(out[0][0]) and out[0][1] == 0.0
