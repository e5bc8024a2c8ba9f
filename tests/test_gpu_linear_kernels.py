"""Every kernel of the linear layer and the gated block (linear_kernel_cases.py; tests/test_linear_host.py holds that these
calls reach them all), all outputs against 64-bit products on the GPU.

Tolerances as in test_gpu_linear.py: an fp32 accumulation over n terms is within (n + 4) u(fp32) sum |x w|; an activation
moves an error by at most its slope (1.2) and adds 4e-7 (1 + |x|), its derivative 1e-6 (1 + |x|); each stored value adds
u(type), the backward's dPre, dGate and dUp being stored once before the products that read them.
"""
import pytest
import torch

import sharded_gemm_amd as tp

from gpu_helpers import Guarded, announce, require_gpu
from linear_kernel_cases import CASES

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SLOPE, ACT_ERR, DACT_ERR = 1.2, 4e-7, 1e-6
U32 = torch.finfo(F32).eps / 2


def setup_module(_):
    require_gpu()


def u(t):
    return torch.finfo(t).eps / 2


class Inputs:
    def __init__(self, dtype, odd, seed):
        self.dtype, self.odd = dtype, odd
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(self, rows, cols, std=1.0):
        """Normal values; odd: in a buffer of NaNs, rows one element apart, one element in."""
        v = (torch.randn((rows, cols), generator=self.g, device="cuda") * std).to(self.dtype)
        if not self.odd:
            return v
        base = torch.full((1 + rows * (cols + 1) + 8,), float("nan"), dtype=self.dtype, device="cuda")
        w = base[1:1 + rows * (cols + 1)].view(rows, cols + 1)[:, :cols]
        w.copy_(v)
        return w


def acc(a, b):
    return (a.shape[1] + 4) * U32 * (a.abs() @ b.abs())


def silu(x):
    s = torch.sigmoid(x)
    return x * s, s * (1 + x * (1 - s))


def near(got, ref, e, name):
    t = u(got.dtype) * (ref.abs() + e) + e
    bad = ~((got.double() - ref).abs() <= t)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off"


def forward(op, dtype, layout, M, K, N, odd):
    i = Inputs(dtype, odd, 1)
    X, std = i.mat(M, K), (2.0 / K) ** 0.5
    wl = (N, K) if layout == "linear" else (K, N)
    code = tp.TP_WEIGHTS_LINEAR if layout == "linear" else tp.TP_WEIGHTS_MATH

    def math(w):
        return w.double().t() if layout == "linear" else w.double()
    x = X.double()
    out, k1, k2 = (Guarded((M, N), dtype) for _ in range(3))
    if op == "linear":
        W, b, R = i.mat(*wl, std), torch.randn(N, generator=i.g, device="cuda"), i.mat(M, N)
        tp.tp_linear(X, W, out.t, bias=b, residual=R, pre_out=k1.t, act=tp.TP_ACT_SILU, weight_layout=code,
                     ws=tp.tp_linear_ws(X, W, weight_layout=code))
        torch.cuda.synchronize()
        pre = x @ math(W) + b.double()
        e = acc(x, math(W)) + U32 * pre.abs()
        near(k1.t, pre, e, "pre_out")
        y = silu(pre)[0] + R.double()
        near(out.t, y, SLOPE * e + ACT_ERR * (1 + pre.abs()) + 2 * U32 * y.abs(), "out")
    else:
        Wg, Wu = i.mat(*wl, std), i.mat(*wl, std)
        tp.tp_gated_linear(X, Wg, Wu, out.t, gate_out=k1.t, up_out=k2.t, weight_layout=code,
                           ws=tp.tp_gated_linear_ws(X, Wg, weight_layout=code))
        torch.cuda.synchronize()
        g, up, eg, eu = x @ math(Wg), x @ math(Wu), acc(x, math(Wg)), acc(x, math(Wu))
        near(k1.t, g, eg, "gate_out")
        near(k2.t, up, eu, "up_out")
        a = silu(g)[0]
        ea = SLOPE * eg + ACT_ERR * (1 + g.abs())
        near(out.t, a * up, ea * (up.abs() + eu) + a.abs() * eu + 2 * U32 * (a * up).abs(), "out")
    assert out.guards_intact() and k1.guards_intact() and k2.guards_intact()


def backward(op, dtype, layout, M, K, N, odd, f32_out):
    i = Inputs(dtype, odd, 2)
    X, d, pre = i.mat(M, K), i.mat(M, N), i.mat(M, N, 2.0)
    wl = (N, K) if layout == "linear" else (K, N)
    code = tp.TP_WEIGHTS_LINEAR if layout == "linear" else tp.TP_WEIGHTS_MATH
    odt = F32 if f32_out else dtype

    def math(w):
        return w.double().t() if layout == "linear" else w.double()
    x, dd, z = X.double(), d.double(), pre.double()
    a, da = silu(z)
    dX, dW, dW2, db = Guarded((M, K), odt), Guarded(wl, odt), Guarded(wl, odt), Guarded((N,), F32)
    old = [torch.zeros(wl, device="cuda") for _ in range(2)]
    if f32_out:      # added to what is there
        for o, t in zip(old, (dW.t, dW2.t)):
            o.copy_(torch.randn(wl, generator=i.g, device="cuda"))
            t.copy_(o)
        db.t.zero_()
    kw = dict(weight_layout=code, accumulate=f32_out, act=tp.TP_ACT_SILU)

    def weight_grad(got, o, dh, eh, name):
        want = x.t() @ dh + math(o)
        near(math(got).to(got.dtype), want, x.t().abs() @ eh + acc(x.t(), dh), name)
    if op == "linear_bwd":
        W = i.mat(*wl, 0.3)
        tp.tp_linear_backward(X, W, d, pre=pre, dX=dX.t, dW=dW.t, dbias=db.t,
                              ws=tp.tp_linear_backward_ws(X, W, d, act=tp.TP_ACT_SILU, weight_layout=code, dbias=db.t), **kw)
        torch.cuda.synchronize()
        dP, e_f = dd * da, dd.abs() * DACT_ERR * (1 + z.abs())
        e_dP = e_f + u(dtype) * ((dd * da).abs() + e_f)
        near(dX.t, dP @ math(W).t(), e_dP @ math(W).t().abs() + acc(dP, math(W).t()), "dX")
        weight_grad(dW.t, old[0], dP, e_dP, "dW")
        near(db.t, dP.sum(0), e_f.sum(0) + (M + 4) * U32 * dP.abs().sum(0), "dbias")
    else:
        Wg, Wu, up = i.mat(*wl, 0.3), i.mat(*wl, 0.3), i.mat(M, N)
        tp.tp_gated_linear_backward(X, Wg, Wu, pre, up, d, dX=dX.t, dW_gate=dW.t, dW_up=dW2.t,
                                    ws=tp.tp_gated_linear_backward_ws(X, d), **kw)
        torch.cuda.synchronize()
        v = up.double()
        dg, du = dd * v * da, dd * a
        e_g = (dd * v).abs() * DACT_ERR * (1 + z.abs()) + 2 * U32 * dg.abs()
        e_u = dd.abs() * DACT_ERR * (1 + z.abs()) + U32 * du.abs()
        e_g, e_u = e_g + u(dtype) * (dg.abs() + e_g), e_u + u(dtype) * (du.abs() + e_u)
        wg, wu = math(Wg).t(), math(Wu).t()
        e = e_g @ wg.abs() + e_u @ wu.abs() + (2 * N + 4) * U32 * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
        near(dX.t, dg @ wg + du @ wu, e, "dX")
        weight_grad(dW.t, old[0], dg, e_g, "dW_gate")
        weight_grad(dW2.t, old[1], du, e_u, "dW_up")
    assert all(t.guards_intact() for t in (dX, dW, dW2, db))


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_kernels(case):
    op, dtype, layout, M, K, N, odd = case
    announce(f"kernels {case}")
    dt = F32 if dtype == "f32" else BF16
    if op.endswith("bwd"):
        for f32_out in (False, True):
            backward(op, dt, layout, M, K, N, odd, f32_out)
    else:
        forward(op, dt, layout, M, K, N, odd)


@pytest.mark.parametrize("dtype,K,N", [(F32, 2047, 2049), (BF16, 4095, 4097)])
@pytest.mark.parametrize("layout", ["math", "linear"])
def test_weight_gradient_beside_the_last_element(dtype, K, N, layout):
    """Whole odd weights, whose gradient is one product over few tokens."""
    announce(f"weight gradient {dtype} {K} x {N} {layout}")
    backward("linear_bwd", dtype, layout, 40, K, N, 0, False)
