"""The linear layer and the gated block on the GPU, forward and backward, against their float64 forms.

Tolerances, per element, from the arithmetic (u(t) = eps(t) / 2, half a step of type t, relative):
 * a product's fp32 accumulation over n terms is within (n + 4) u(fp32) sum |x w| of exact, whatever its order;
 * an activation moves an error by at most its slope (below 1.2 for all of them) and adds at most
   4e-7 (1 + |x|) of its own (the error function's polynomial 1.5e-7 |x|, exp2 and reciprocal 1 ulp each);
 * a stored value adds u(type) relative; the backward's dPre, dGate and dUp are stored once in the operands' type
   before the products that read them.
"""
import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import linear as O

from gpu_helpers import Guarded, announce, bits, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
MATH, LINEAR = tp.TP_WEIGHTS_MATH, tp.TP_WEIGHTS_LINEAR
ACTS = [tp.TP_ACT_NONE, tp.TP_ACT_GELU_ERF, tp.TP_ACT_GELU_TANH, tp.TP_ACT_SILU, tp.TP_ACT_RELU]
SLOPE, ACT_ERR = 1.2, 4e-7
U32 = torch.finfo(F32).eps / 2

# (M, K, N): one token and one of everything, the edges of 16-row groups, tiles and K stages, odd sizes, whole tiles,
# and enough of them for the largest tiles.
SHAPES = [(1, 1, 1), (1, 512, 768), (2, 96, 40), (7, 33, 65), (16, 256, 128), (17, 130, 77), (64, 320, 200),
          (65, 63, 129), (130, 257, 200), (256, 512, 384), (333, 224, 520), (2048, 192, 2056)]


def setup_module(_):
    require_gpu()


def u(t):
    return torch.finfo(t).eps / 2


def rnd(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def place(t, stride_extra=0, offset=0):
    """`t` on the GPU inside a larger buffer of NaNs: rows `stride_extra` apart, starting `offset` elements in."""
    rows, cols = t.shape
    ld = cols + stride_extra
    base = torch.full((offset + rows * ld + 8,), float("nan"), dtype=t.dtype, device="cuda")
    v = base[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(t)
    return v


def check(got, ref, tol, name):
    g = f64(got)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} off, worst {np.max(np.abs(g - ref) / tol):.3g} x the tolerance"


def lay(W, layout):
    return W if layout == MATH else W.t().contiguous()


def unlay(dW, layout):
    return f64(dW) if layout == MATH else f64(dW).T


def product_err(A, B, n):
    """The accumulation's bound for A B over n terms."""
    return (n + 4) * U32 * (np.abs(A) @ np.abs(B))


def run_linear(M, K, N, dtype, layout, act, *, bias=True, residual=True, save=True, out_f32=False, strided=0, offset=0,
               in_place=False, seed=0, std_w=None):
    X, W = rnd((M, K), seed, dtype), rnd((K, N), seed + 1, dtype, std_w or (2.0 / K) ** 0.5)
    b = rnd((N,), seed + 2, F32) if bias else None
    R = rnd((M, N), seed + 3, dtype) if residual else None
    odt = F32 if out_f32 else dtype
    out, pre = Guarded((M, N), odt), Guarded((M, N), dtype) if save else None
    Rd = place(R, strided, offset) if residual else None
    if in_place:
        out.t.copy_(R)
        Rd = out.t
    tp.tp_linear(place(X, strided, offset), place(lay(W, layout), strided, offset), out.t, bias=b.cuda() if bias else None,
                 residual=Rd, pre_out=pre.t if save else None, act=act, weight_layout=layout)
    torch.cuda.synchronize()
    assert out.guards_intact() and (pre is None or pre.guards_intact())
    ref, rpre = O.linear(f64(X), f64(W), None if b is None else f64(b), None if R is None else f64(R), act)
    e_pre = product_err(f64(X), f64(W), K) + (U32 * np.abs(rpre) if bias else 0.0)
    e_out = SLOPE * e_pre + (0.0 if act == 0 else ACT_ERR * (1 + np.abs(rpre))) + 2 * U32 * np.abs(ref)
    check(out.t, ref, e_out + u(odt) * (np.abs(ref) + e_out), "out")
    if save:
        check(pre.t, rpre, e_pre + u(dtype) * (np.abs(rpre) + e_pre), "pre_out")
    return out.t, pre.t if save else None


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(shape, dtype, layout):
    announce(f"linear {shape} {dtype} layout {layout}")
    run_linear(*shape, dtype, layout, tp.TP_ACT_SILU, seed=10)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [2, 100])
def test_linear_activations(M, dtype, act):
    announce(f"linear act {act} {dtype} M {M}")
    run_linear(M, 96, 136, dtype, MATH, act, seed=20, std_w=0.4)   # pre-activations out to about 15
    run_linear(M, 64, 72, dtype, LINEAR, act, seed=21, residual=False, save=False)


@pytest.mark.parametrize("kw", [dict(bias=False, residual=False, save=False), dict(bias=True, residual=False, save=False),
                                dict(bias=False, residual=True, save=False), dict(bias=False, residual=False, save=True),
                                dict(out_f32=True), dict(in_place=True), dict(in_place=True, save=False)])
@pytest.mark.parametrize("M", [5, 192])
@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_linear_options(M, kw, layout):
    announce(f"linear options M {M} {kw} layout {layout}")
    run_linear(M, 192, 264, BF16, layout, tp.TP_ACT_GELU_ERF, seed=30, **kw)


@pytest.mark.parametrize("strided,offset", [(8, 0), (1, 0), (0, 1), (5, 3), (64, 8)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("M", [3, 150])
def test_linear_strides(M, layout, dtype, strided, offset):
    """Rows apart and off every vector alignment, with NaN between them: nothing outside the rows is used."""
    announce(f"linear strides M {M} {layout} {dtype} +{strided} @{offset}")
    run_linear(M, 160, 96, dtype, layout, tp.TP_ACT_GELU_TANH, strided=strided, offset=offset, seed=40)


@pytest.mark.parametrize("M", [4, 80, 300])
def test_linear_strided_outputs(M):
    K, N = 128, 64
    X, W, R = rnd((M, K), 1, BF16), rnd((K, N), 2, BF16, 0.1), rnd((M, N), 3, BF16)
    tight, pre_t = torch.empty((M, N), dtype=BF16, device="cuda"), torch.empty((M, N), dtype=BF16, device="cuda")
    kw = dict(residual=R.cuda(), act=tp.TP_ACT_SILU)
    tp.tp_linear(X.cuda(), W.cuda(), tight, pre_out=pre_t, **kw)
    for extra in (8, 3):
        wide = torch.full((M, N + extra), 7.0, dtype=BF16, device="cuda")
        pre = torch.full((M, N + extra), 7.0, dtype=BF16, device="cuda")
        tp.tp_linear(X.cuda(), W.cuda(), wide[:, :N], pre_out=pre[:, :N], **kw)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, :N], tight) and torch.equal(pre[:, :N], pre_t)
        assert bool((wide[:, N:] == 7.0).all()) and bool((pre[:, N:] == 7.0).all())


@pytest.mark.parametrize("M", [1, 6, 70, 200])
@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_a_bad_row_stays_one(M, layout):
    """NaN and infinities in one token's row, and in one weight's column, reach that row and column alone."""
    K, N = 101, 90
    X, W = rnd((M, K), 5, BF16), rnd((K, N), 6, BF16, 0.1)
    out = torch.empty((M, N), dtype=BF16, device="cuda")
    tp.tp_linear(X.cuda(), lay(W, layout).cuda(), out, weight_layout=layout)
    Xb, Wb = X.clone(), W.clone()
    r, c = M - 1, N - 1
    Xb[r, K - 1] = float("nan")
    Wb[K - 1, c] = float("inf")
    bad = torch.empty_like(out)
    tp.tp_linear(Xb.cuda(), lay(Wb, layout).cuda(), bad, weight_layout=layout)
    torch.cuda.synchronize()
    assert bool(torch.isnan(bad[r]).all())
    assert not bool(torch.isfinite(bad[:, c]).any())
    assert torch.equal(bad[:r, :c], out[:r, :c])


def run_linear_bwd(M, K, N, dtype, layout, act, *, dx_f32=False, dw_f32=False, accumulate=False, dbias=True, strided=0,
                   offset=0, seed=0):
    X, W = rnd((M, K), seed, dtype), rnd((K, N), seed + 1, dtype, 0.3)
    d, pre = rnd((M, N), seed + 2, dtype), rnd((M, N), seed + 3, dtype, 2.0)
    xdt, wdt = F32 if dx_f32 else dtype, F32 if dw_f32 else dtype
    wshape = (K, N) if layout == MATH else (N, K)
    dX, dW, db = Guarded((M, K), xdt), Guarded(wshape, wdt), Guarded((N,), F32)
    old_w, old_b = rnd(wshape, seed + 4, wdt), rnd((N,), seed + 5, F32)
    if accumulate:
        dW.t.copy_(old_w)
        db.t.copy_(old_b)
    Xd, Wd, dd = place(X, strided, offset), place(lay(W, layout), strided, offset), place(d, strided, offset)
    ws = tp.tp_linear_backward_ws(Xd, Wd, dd, act=act, weight_layout=layout, dbias=db.t if dbias else None)
    tp.tp_linear_backward(Xd, Wd, dd, pre=place(pre, strided, offset) if act else None, dX=dX.t, dW=dW.t,
                          dbias=db.t if dbias else None, act=act, weight_layout=layout, accumulate=accumulate, ws=ws)
    torch.cuda.synchronize()
    assert dX.guards_intact() and dW.guards_intact() and db.guards_intact()
    ref = O.linear_backward(f64(X), f64(W), f64(d), f64(pre), act)
    dP = ref["dPre"]
    # dPre: the derivative is within 1e-6 (1 + |pre|) of exact, then one rounding where there is an activation.
    e_f = 0.0 * dP if act == 0 else np.abs(f64(d)) * 1e-6 * (1 + np.abs(f64(pre)))
    e_dP = e_f if act == 0 else e_f + u(dtype) * (np.abs(dP) + e_f)
    aW, aX = np.abs(f64(W)), np.abs(f64(X))
    e = e_dP @ aW.T + product_err(dP, f64(W).T, N)
    check(dX.t, ref["dX"], e + u(xdt) * (np.abs(ref["dX"]) + e), "dX")
    want = ref["dW"] + (unlay(old_w, layout) if accumulate else 0.0)
    e = aX.T @ e_dP + product_err(f64(X).T, dP, M)
    check(torch.from_numpy(unlay(dW.t, layout)), want, e + u(wdt) * (np.abs(want) + e), "dW")
    if dbias:
        want = ref["dbias"] + (f64(old_b) if accumulate else 0.0)
        e = e_f.sum(0) + (M + 4) * U32 * np.abs(dP).sum(0)
        check(db.t, want, e + U32 * (np.abs(want) + e), "dbias")


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_backward(shape, dtype, layout):
    announce(f"linear backward {shape} {dtype} layout {layout}")
    run_linear_bwd(*shape, dtype, layout, tp.TP_ACT_SILU, seed=50)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_backward_activations(dtype, act):
    announce(f"linear backward act {act} {dtype}")
    run_linear_bwd(100, 96, 136, dtype, MATH, act, seed=60)


@pytest.mark.parametrize("kw", [dict(dx_f32=True), dict(dw_f32=True), dict(dw_f32=True, accumulate=True), dict(dbias=False),
                                dict(strided=8), dict(strided=3, offset=1), dict(dx_f32=True, dw_f32=True, strided=1)])
@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("act", [tp.TP_ACT_NONE, tp.TP_ACT_GELU_ERF])
def test_linear_backward_options(kw, layout, act):
    announce(f"linear backward options {kw} {layout} act {act}")
    run_linear_bwd(192, 128, 72, BF16, layout, act, seed=70, **kw)


def run_gated(M, K, F, dtype, layout, act, *, save=True, strided=0, offset=0, seed=0, merged=False):
    X = rnd((M, K), seed, dtype)
    Wg, Wu = rnd((K, F), seed + 1, dtype, (2.0 / K) ** 0.5), rnd((K, F), seed + 2, dtype, (2.0 / K) ** 0.5)
    if merged:    # one weight whose halves are the two projections
        both = torch.cat([lay(Wg, layout), lay(Wu, layout)], dim=1 if layout == MATH else 0).cuda()
        wg, wu = (both[:, :F], both[:, F:]) if layout == MATH else (both[:F], both[F:])
    else:
        wg, wu = place(lay(Wg, layout), strided, offset), place(lay(Wu, layout), strided, offset)
    out = Guarded((M, F), dtype)
    g, up = (Guarded((M, F), dtype), Guarded((M, F), dtype)) if save else (None, None)
    tp.tp_gated_linear(place(X, strided, offset), wg, wu, out.t, gate_out=g.t if save else None,
                       up_out=up.t if save else None, act=act, weight_layout=layout)
    torch.cuda.synchronize()
    assert out.guards_intact()
    ref, rg, ru = O.gated(f64(X), f64(Wg), f64(Wu), act)
    eg, eu = product_err(f64(X), f64(Wg), K), product_err(f64(X), f64(Wu), K)
    a = np.abs(O.act(act, rg))
    ea = SLOPE * eg + (0.0 if act == 0 else ACT_ERR * (1 + np.abs(rg)))
    e = ea * (np.abs(ru) + eu) + a * eu + 2 * U32 * np.abs(ref)
    check(out.t, ref, e + u(dtype) * (np.abs(ref) + e), "out")
    if save:
        assert g.guards_intact() and up.guards_intact()
        check(g.t, rg, eg + u(dtype) * (np.abs(rg) + eg), "gate_out")
        check(up.t, ru, eu + u(dtype) * (np.abs(ru) + eu), "up_out")


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated(shape, dtype, layout):
    announce(f"gated {shape} {dtype} layout {layout}")
    run_gated(*shape, dtype, layout, tp.TP_ACT_SILU, seed=80)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kw", [dict(), dict(save=False), dict(strided=8), dict(strided=3, offset=1), dict(merged=True)])
@pytest.mark.parametrize("M", [3, 96])
def test_gated_options(M, act, kw):
    announce(f"gated M {M} act {act} {kw}")
    run_gated(M, 160, 88, BF16, MATH, act, seed=90, **kw)
    run_gated(M, 72, 104, F32, LINEAR, act, seed=91, **kw)


def run_gated_bwd(M, K, F, dtype, layout, act, *, dx_f32=False, dw_f32=False, accumulate=False, strided=0, offset=0, seed=0,
                  merged=False):
    X = rnd((M, K), seed, dtype)
    Wg, Wu = rnd((K, F), seed + 1, dtype, 0.3), rnd((K, F), seed + 2, dtype, 0.3)
    g, up, d = rnd((M, F), seed + 3, dtype, 2.0), rnd((M, F), seed + 4, dtype), rnd((M, F), seed + 5, dtype)
    xdt, wdt = F32 if dx_f32 else dtype, F32 if dw_f32 else dtype
    wshape = (K, F) if layout == MATH else (F, K)
    dX = Guarded((M, K), xdt)
    old = [rnd(wshape, seed + 6 + i, wdt) for i in range(2)]
    if merged:
        dim = 1 if layout == MATH else 0
        both = torch.cat([lay(Wg, layout), lay(Wu, layout)], dim=dim).cuda()
        wg, wu = both.narrow(dim, 0, F), both.narrow(dim, F, F)
        grads = torch.empty(both.shape, dtype=wdt, device="cuda")
        dWs = [grads.narrow(dim, 0, F), grads.narrow(dim, F, F)]
        guards = [dX]
    else:
        wg, wu = place(lay(Wg, layout), strided, offset), place(lay(Wu, layout), strided, offset)
        guards = [dX, Guarded(wshape, wdt), Guarded(wshape, wdt)]
        dWs = [x.t for x in guards[1:]]
    if accumulate:
        for t, o in zip(dWs, old):
            t.copy_(o)
    Xd, dd = place(X, strided, offset), place(d, strided, offset)
    ws = tp.tp_gated_linear_backward_ws(Xd, dd)
    tp.tp_gated_linear_backward(Xd, wg, wu, place(g, strided, offset), place(up, strided, offset), dd, dX=dX.t, dW_gate=dWs[0],
                                dW_up=dWs[1], act=act, weight_layout=layout, accumulate=accumulate, ws=ws)
    torch.cuda.synchronize()
    assert all(x.guards_intact() for x in guards)
    ref = O.gated_backward(f64(X), f64(Wg), f64(Wu), f64(g), f64(up), f64(d), act)
    aerr = 0.0 if act == 0 else 1e-6 * (1 + np.abs(f64(g)))
    e_g = np.abs(f64(d) * f64(up)) * aerr + 2 * U32 * np.abs(ref["dGate"])
    e_u = np.abs(f64(d)) * aerr + U32 * np.abs(ref["dUp"])
    e_g, e_u = e_g + u(dtype) * (np.abs(ref["dGate"]) + e_g), e_u + u(dtype) * (np.abs(ref["dUp"]) + e_u)
    e = e_g @ np.abs(f64(Wg)).T + e_u @ np.abs(f64(Wu)).T + \
        (2 * F + 4) * U32 * (np.abs(ref["dGate"]) @ np.abs(f64(Wg)).T + np.abs(ref["dUp"]) @ np.abs(f64(Wu)).T)
    check(dX.t, ref["dX"], e + u(xdt) * (np.abs(ref["dX"]) + e), "dX")
    for t, o, name, dh, eh in ((dWs[0], old[0], "dWg", ref["dGate"], e_g), (dWs[1], old[1], "dWu", ref["dUp"], e_u)):
        want = ref[name] + (unlay(o, layout) if accumulate else 0.0)
        e = np.abs(f64(X)).T @ eh + product_err(f64(X).T, dh, M)
        check(torch.from_numpy(unlay(t, layout)), want, e + u(wdt) * (np.abs(want) + e), name)


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_backward(shape, dtype, layout):
    announce(f"gated backward {shape} {dtype} layout {layout}")
    run_gated_bwd(*shape, dtype, layout, tp.TP_ACT_SILU, seed=100)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("kw", [dict(), dict(dx_f32=True, dw_f32=True), dict(dw_f32=True, accumulate=True), dict(strided=8),
                                dict(strided=3, offset=1), dict(merged=True)])
def test_gated_backward_options(act, layout, kw):
    announce(f"gated backward act {act} layout {layout} {kw}")
    run_gated_bwd(128, 96, 72, BF16, layout, act, seed=110, **kw)


def test_empty_batch():
    """No rows: nothing is written by the forward; weight and bias gradients are zero, or stay."""
    X, W, d = (torch.empty((0, 24), dtype=BF16, device="cuda"), rnd((24, 16), 1, BF16).cuda(),
               torch.empty((0, 16), dtype=BF16, device="cuda"))
    tp.tp_linear(X, W, torch.empty_like(d))
    tp.tp_gated_linear(X, W, W.clone(), torch.empty_like(d))
    for acc in (False, True):
        dW, db = torch.ones((24, 16), device="cuda"), torch.ones(16, device="cuda")
        dW2, dW3 = torch.ones_like(dW), torch.ones_like(dW)
        ws = tp.tp_linear_backward_ws(X, W, d, act=tp.TP_ACT_SILU, dbias=db)
        tp.tp_linear_backward(X, W, d, pre=d, dX=torch.empty_like(X), dW=dW, dbias=db, act=tp.TP_ACT_SILU, accumulate=acc, ws=ws)
        tp.tp_gated_linear_backward(X, W, W.clone(), d, d, d, dX=torch.empty_like(X), dW_gate=dW2, dW_up=dW3, accumulate=acc,
                                    ws=tp.tp_gated_linear_backward_ws(X, d))
        torch.cuda.synchronize()
        for t in (dW, db, dW2, dW3):
            assert bool((t == (1.0 if acc else 0.0)).all())


def test_gradients_left_out():
    """Each gradient alone has the bits it has beside the others."""
    M, K, N = 96, 64, 80
    X, W, d, pre = rnd((M, K), 1, BF16).cuda(), rnd((K, N), 2, BF16).cuda(), rnd((M, N), 3, BF16).cuda(), rnd((M, N), 4, BF16).cuda()
    kw = dict(pre=pre, act=tp.TP_ACT_SILU)
    full = dict(dX=torch.empty_like(X), dW=torch.empty_like(W), dbias=torch.empty(N, device="cuda"))
    ws = tp.tp_linear_backward_ws(X, W, d, act=tp.TP_ACT_SILU, dbias=full["dbias"])
    tp.tp_linear_backward(X, W, d, ws=ws, **kw, **full)
    for name, t in full.items():
        one = torch.empty_like(t)
        tp.tp_linear_backward(X, W, d, ws=torch.empty_like(ws), **kw, **{name: one})
        torch.cuda.synchronize()
        assert torch.equal(one, t), name
    up = rnd((M, N), 5, BF16).cuda()
    W2 = rnd((K, N), 6, BF16).cuda()
    ws = tp.tp_gated_linear_backward_ws(X, d)
    a, b, c = torch.empty_like(X), torch.empty_like(W), torch.empty_like(W)
    tp.tp_gated_linear_backward(X, W, W2, pre, up, d, dX=a, dW_gate=b, dW_up=c, ws=ws)
    a1, b1, c1 = torch.empty_like(X), torch.empty_like(W), torch.empty_like(W)
    tp.tp_gated_linear_backward(X, W, W2, pre, up, d, dX=a1, ws=ws)
    tp.tp_gated_linear_backward(X, W, W2, pre, up, d, dW_gate=b1, dW_up=c1, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, a1) and torch.equal(b, b1) and torch.equal(c, c1)


@pytest.mark.parametrize("shape", [(1, 256, 192), (48, 128, 96), (300, 192, 256)])
def test_graph_replays_and_streams(shape):
    """A step captured once, replayed with eager work between, on a stream of its own: every replay has the eager bits."""
    M, K, F = shape
    X, R = rnd((M, K), 1, BF16).cuda(), rnd((M, K), 2, BF16).cuda()
    Wg, Wu, Wd = rnd((K, F), 3, BF16, 0.1).cuda(), rnd((K, F), 4, BF16, 0.1).cuda(), rnd((F, K), 5, BF16, 0.1).cuda()
    g, up, y = (torch.empty((M, F), dtype=BF16, device="cuda") for _ in range(3))
    out, dY, dX = torch.empty_like(X), torch.empty_like(y), torch.empty_like(X)
    grads = [torch.empty_like(Wg), torch.empty_like(Wu), torch.empty_like(Wd), torch.empty(K, device="cuda")]
    ws1, ws2 = tp.tp_linear_backward_ws(y, Wd, out, dbias=grads[3]), tp.tp_gated_linear_backward_ws(X, y)
    parts, norm = tp.tp_grad_parts(), torch.empty(1, device="cuda")
    clipped = [torch.empty_like(t) for t in grads]

    def step(stream):
        tp.tp_gated_linear(X, Wg, Wu, y, gate_out=g, up_out=up, stream=stream)
        tp.tp_linear(y, Wd, out, residual=R, stream=stream)
        tp.tp_linear_backward(y, Wd, out, dX=dY, dW=grads[2], dbias=grads[3], ws=ws1, stream=stream)
        tp.tp_gated_linear_backward(X, Wg, Wu, g, up, dY, dX=dX, dW_gate=grads[0], dW_up=grads[1], ws=ws2, stream=stream)
        tp.tp_grad_sumsq(grads, parts, stream=stream)
        tp.tp_grad_clip(grads, clipped, parts, max_norm=0.5, norm_out=norm, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    results = [out, dX, norm, *grads, *clipped]
    want = [t.clone() for t in results]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for _ in range(4):
        for t in results:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(results, want):
            assert np.array_equal(bits(t), bits(w))
        step(torch.cuda.current_stream())


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("M,K,N", [(4096, 64, 4096), (2048, 64, 6144), (2048, 96, 2048), (64, 2048, 6144), (96, 2048, 2048)])
def test_every_tile(M, K, N, layout):
    """Enough output for each of the bf16 tiles (256 x 256, 256 x 192, 256 x 128, 128 x 128), forward and backward, against
    64-bit products on the GPU."""
    announce(f"tiles {M} {K} {N} layout {layout}")
    X, d = rnd((M, K), 1, BF16).cuda(), rnd((M, N), 2, BF16).cuda()
    W, W2 = rnd((K, N), 3, BF16, 0.2).cuda(), rnd((K, N), 4, BF16, 0.2).cuda()
    Wl, W2l = lay(W, layout), lay(W2, layout)
    x, w, w2, dd = X.double(), W.double(), W2.double(), d.double()

    def acc(a, b):
        return (a.shape[1] + 4) * U32 * (a.abs() @ b.abs())

    def near(got, ref, e, name):
        assert bool(((got.double() - ref).abs() <= e + u(BF16) * (ref.abs() + e)).all()), name
    out = torch.empty((M, N), dtype=BF16, device="cuda")
    tp.tp_linear(X, Wl, out, weight_layout=layout)
    near(out, x @ w, acc(x, w), "linear")
    tp.tp_gated_linear(X, Wl, W2l, out, act=tp.TP_ACT_NONE, weight_layout=layout)
    g, up = x @ w, x @ w2
    eg, eu = acc(x, w), acc(x, w2)
    near(out, g * up, eg * (up.abs() + eu) + g.abs() * eu + 2 * U32 * (g * up).abs(), "gated")
    dX, dW, dW2 = torch.empty_like(X), torch.empty_like(Wl), torch.empty_like(Wl)
    tp.tp_linear_backward(X, Wl, d, dX=dX, dW=dW, weight_layout=layout)
    near(dX, dd @ w.t(), acc(dd, w.t()), "dX")
    near(dW if layout == MATH else dW.t(), x.t() @ dd, acc(x.t(), dd), "dW")
    gb, ub = g.to(BF16), up.to(BF16)
    tp.tp_gated_linear_backward(X, Wl, W2l, gb, ub, d, dX=dX, dW_gate=dW, dW_up=dW2, act=tp.TP_ACT_NONE, weight_layout=layout,
                                ws=tp.tp_gated_linear_backward_ws(X, d))
    torch.cuda.synchronize()
    dg, du = (dd * ub.double()), (dd * gb.double())
    rg, ru = u(BF16) * 1.01 * dg.abs(), u(BF16) * 1.01 * du.abs()      # each is stored once in bf16
    near(dX, dg @ w.t() + du @ w2.t(), rg @ w.t().abs() + ru @ w2.t().abs() + 2 * (acc(dg, w.t()) + acc(du, w2.t())), "gated dX")
    for got, h, r, name in ((dW, dg, rg, "dW_gate"), (dW2, du, ru, "dW_up")):
        near(got if layout == MATH else got.t(), x.t() @ h, x.t().abs() @ r + acc(x.t(), h), name)


# Few rows and few tiles with a long K: the products split K and join through the workspace.
SPLIT = [(1, 4096, 256, BF16, MATH), (3, 2056, 130, BF16, MATH), (16, 4100, 65, BF16, LINEAR), (1, 3000, 96, F32, MATH),
         (9, 1030, 50, F32, LINEAR), (40, 4096, 256, BF16, LINEAR), (64, 4096, 192, BF16, MATH), (100, 2080, 120, BF16, MATH),
         (100, 4097, 129, BF16, MATH), (70, 2051, 100, F32, LINEAR), (130, 1111, 77, F32, MATH)]


@pytest.mark.parametrize("case", SPLIT, ids=[str(c[:3]) for c in SPLIT])
def test_split_k(case):
    """With a workspace the result is within the same bounds, the same every time, and the workspace stays fit for the
    next call, also of another shape."""
    M, K, N, dtype, layout = case
    announce(f"split {case}")
    X, W, W2 = rnd((M, K), 1, dtype), rnd((K, N), 2, dtype, (2.0 / K) ** 0.5), rnd((K, N), 3, dtype, (2.0 / K) ** 0.5)
    Xd, Wd, W2d = X.cuda(), lay(W, layout).cuda(), lay(W2, layout).cuda()
    ws1, ws2 = tp.tp_linear_ws(Xd, Wd, weight_layout=layout), tp.tp_gated_linear_ws(Xd, Wd, weight_layout=layout)
    assert ws1.numel() > 0 and ws2.numel() > 0
    ws = torch.zeros(max(ws1.numel(), ws2.numel()), dtype=torch.uint8, device="cuda")
    out, both = Guarded((M, N), dtype), Guarded((M, N), dtype)
    ref, pre = O.linear(f64(X), f64(W), kind=tp.TP_ACT_SILU)
    e = SLOPE * product_err(f64(X), f64(W), K) + ACT_ERR * (1 + np.abs(pre)) + 2 * U32 * np.abs(ref)
    gref, rg, ru = O.gated(f64(X), f64(W), f64(W2), tp.TP_ACT_SILU)
    eu = product_err(f64(X), f64(W2), K)
    eg = e * (np.abs(ru) + eu) + np.abs(ref) * eu + 2 * U32 * np.abs(gref)
    first = None
    for _ in range(4):
        out.fill_sentinel()
        both.fill_sentinel()
        tp.tp_linear(Xd, Wd, out.t, act=tp.TP_ACT_SILU, weight_layout=layout, ws=ws)
        tp.tp_gated_linear(Xd, Wd, W2d, both.t, weight_layout=layout, ws=ws)
        torch.cuda.synchronize()
        assert out.guards_intact() and both.guards_intact()
        got = (bits(out.t), bits(both.t))
        first = first or got
        assert all(np.array_equal(a, b) for a, b in zip(first, got))
    check(out.t, ref, e + u(dtype) * (np.abs(ref) + e), "out")
    check(both.t, gref, eg + u(dtype) * (np.abs(gref) + eg), "gated out")


@pytest.mark.parametrize("shape", [(8, 128, 96), (2048, 64, 96), (4100, 40, 72), (3000, 33, 65), (16, 512, 2048)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_split_k_backward(shape, dtype, layout):
    """Many tokens against a small weight (and few against a wide one): the backward's products split K."""
    announce(f"split backward {shape} {dtype} layout {layout}")
    run_linear_bwd(*shape, dtype, layout, tp.TP_ACT_SILU, seed=120)
    run_linear_bwd(*shape, dtype, layout, tp.TP_ACT_NONE, seed=121, dbias=False)
    run_linear_bwd(*shape, dtype, layout, tp.TP_ACT_NONE, seed=122, dw_f32=True, accumulate=True)
    run_gated_bwd(*shape, dtype, layout, tp.TP_ACT_GELU_ERF, seed=123)


def test_prepared_calls():
    M, K, N = 33, 64, 48
    X, W = rnd((M, K), 1, BF16).cuda(), rnd((K, N), 2, BF16).cuda()
    a, b = torch.empty((M, N), dtype=BF16, device="cuda"), torch.empty((M, N), dtype=BF16, device="cuda")
    tp.tp_linear(X, W, a)
    call = tp.tp_linear(X, W, b, prepare=True)
    b.fill_(0)
    call()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    b.resize_(2 * M, 2 * N * 64)
    with pytest.raises(tp.TpError):
        call()


@pytest.mark.parametrize("dtype,K,N", [(F32, 2047, 2049), (BF16, 4095, 4097)])
@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_nothing_behind_the_last_element(dtype, K, N, layout):
    """A weight that ends within 8 bytes of its allocation, with columns past the edge in the last tile."""
    announce(f"last element {dtype} {K} x {N} layout {layout}")
    M = 40
    W = (torch.randn((K, N) if layout == MATH else (N, K), device="cuda") * 0.02).to(dtype)
    X = rnd((M, K), 1, dtype).cuda()
    out = torch.empty((M, N), dtype=dtype, device="cuda")
    tp.tp_linear(X, W, out, weight_layout=layout)
    dX, dW, d = torch.empty_like(X), torch.empty_like(W), rnd((M, N), 2, dtype).cuda()
    tp.tp_linear_backward(X, W, d, dX=dX, dW=dW, weight_layout=layout)
    torch.cuda.synchronize()
    w = W.double() if layout == MATH else W.double().t()
    for got, a, b in ((out, X.double(), w), (dX, d.double(), w.t())):
        ref = a @ b
        e = (a.shape[1] + 4) * U32 * (a.abs() @ b.abs())
        assert bool(((got.double() - ref).abs() <= e + u(dtype) * (ref.abs() + e)).all())


def test_far_offsets():
    """Operands whose last element lies past 2^32 bytes from their base."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    M, K, N = 40, 64, 96
    X, W = rnd((M, K), 1, BF16), rnd((K, N), 2, BF16)
    ref = torch.empty((M, N), dtype=BF16, device="cuda")
    far = (1 << 26) + 8                     # elements between rows: 40 rows reach 5.4e9 bytes
    for rows in (M, 5):
        tp.tp_linear(X[:rows].cuda(), W.cuda(), ref[:rows])
        base = torch.zeros(M * far, dtype=BF16, device="cuda").view(M, far)
        base[:rows, :K] = X[:rows].cuda()
        out = torch.empty((rows, N), dtype=BF16, device="cuda")
        tp.tp_linear(base[:rows, :K], W.cuda(), out)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[:rows])
        tp.tp_linear(X[:rows].cuda(), W.cuda(), base[:rows, K:K + N])
        torch.cuda.synchronize()
        assert torch.equal(base[:rows, K:K + N], ref[:rows])
        del base
        wide = torch.zeros(K * far, dtype=BF16, device="cuda").view(K, far)
        wide[:, :N] = W.cuda()
        out.zero_()
        tp.tp_linear(X[:rows].cuda(), wide[:, :N], out)
        torch.cuda.synchronize()
        assert torch.equal(out, ref[:rows])
        del wide
