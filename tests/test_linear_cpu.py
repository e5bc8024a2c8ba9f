"""Refusals of the linear layer, the gated block and gradient clipping: every bad argument is turned down before
anything is enqueued (no GPU here), by the C entry points and by the binding."""
import ctypes as C

import pytest
import torch

import sharded_gemm_amd as tp
from sharded_gemm_amd import _abi

BASE = 1 << 40          # a made-up address: no call below may get as far as using it
STEP = 1 << 24


def P(i):
    return BASE + i * STEP


def _linear(**kw):
    a = dict(dtype=tp.TP_BF16, act=tp.TP_ACT_SILU, weight_layout=0, out_dtype=tp.TP_BF16, M=64, N=48, K=32, X=P(0), W=P(1),
             bias=P(2), residual=P(3), out=P(4), pre_out=P(5))
    a.update(kw)
    return _abi.tp_linear_args(**a)


def _linear_bwd(**kw):
    a = dict(dtype=tp.TP_BF16, act=tp.TP_ACT_SILU, weight_layout=0, dx_dtype=tp.TP_BF16, dw_dtype=tp.TP_F32, M=64, N=48,
             K=32, X=P(0), W=P(1), dOut=P(2), pre=P(3), dX=P(4), dW=P(5), dbias=P(6), ws=P(7), ws_bytes=1 << 20)
    a.update(kw)
    return _abi.tp_linear_bwd_args(**a)


def _gated(**kw):
    a = dict(dtype=tp.TP_BF16, act=tp.TP_ACT_SILU, weight_layout=0, M=64, F=48, K=32, X=P(0), W_gate=P(1), W_up=P(2),
             out=P(3), gate_out=P(4), up_out=P(5))
    a.update(kw)
    return _abi.tp_gated_args(**a)


def _gated_bwd(**kw):
    a = dict(dtype=tp.TP_BF16, act=tp.TP_ACT_SILU, weight_layout=0, dx_dtype=tp.TP_BF16, dw_dtype=tp.TP_F32, M=64, F=48,
             K=32, X=P(0), W_gate=P(1), W_up=P(2), gate=P(3), up=P(4), dOut=P(5), dX=P(6), dW_gate=P(7), dW_up=P(8),
             ws=P(9), ws_bytes=1 << 20)
    a.update(kw)
    return _abi.tp_gated_bwd_args(**a)


ARG, UNS = _abi.TP_ERR_ARG, _abi.TP_ERR_UNSUPPORTED
COMMON = [(dict(dtype=7), ARG), (dict(act=5), ARG), (dict(act=-1), ARG), (dict(weight_layout=2), ARG), (dict(M=-1), ARG),
          (dict(K=0), ARG), (dict(K=1 << 31), UNS), (dict(M=1 << 31), UNS), (dict(M=1 << 30, K=1 << 16), UNS), (dict(K=1 << 26), UNS),
          (dict(X=None), ARG), (dict(X=P(0) + 1), ARG), (dict(X_ld=31), ARG), (dict(X_ld=1 << 31), UNS)]


def _refused(fn, args, want):
    lib = _abi.load()
    rc = getattr(lib, fn)(C.byref(args), None)
    assert rc == want, (rc, lib.tp_last_error())
    assert lib.tp_last_error()


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(N=0), ARG), (dict(out_dtype=9), ARG), (dict(W=None), ARG), (dict(out=None), ARG), (dict(W_ld=47), ARG),
    (dict(out_ld=47), ARG), (dict(residual_ld=1), ARG), (dict(pre_ld=2), ARG), (dict(bias=P(2) + 2), ARG),
    (dict(out=P(0)), ARG), (dict(out=P(1) + 64), ARG), (dict(out=P(2)), ARG), (dict(pre_out=P(4)), ARG),
    (dict(out=P(3), out_ld=64), ARG), (dict(out=P(3), out_dtype=tp.TP_F32), ARG), (dict(out=P(3) + 2), ARG),
    (dict(out=P(3), pre_out=P(3)), ARG), (dict(dtype=tp.TP_F32, out_dtype=tp.TP_BF16), ARG)])
def test_linear_refusals(kw, want):
    _refused("tp_linear", _linear(**kw), want)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(N=0), ARG), (dict(dx_dtype=9), ARG), (dict(dw_dtype=9), ARG), (dict(W=None), ARG), (dict(dOut=None), ARG),
    (dict(pre=None), ARG), (dict(pre_ld=3), ARG), (dict(accumulate=2), ARG),
    (dict(accumulate=1, dw_dtype=tp.TP_BF16), ARG), (dict(ws=None), ARG), (dict(ws_bytes=100), ARG),
    (dict(ws=P(7) + 8), ARG), (dict(dX=P(2)), ARG), (dict(dW=P(4)), ARG), (dict(dbias=P(7)), ARG), (dict(ws=P(3)), ARG),
    (dict(dX=P(1)), ARG), (dict(dtype=tp.TP_F32, dx_dtype=tp.TP_BF16), ARG)])
def test_linear_backward_refusals(kw, want):
    _refused("tp_linear_backward", _linear_bwd(**kw), want)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(F=0), ARG), (dict(W_up=None), ARG), (dict(W_gate=None), ARG), (dict(out=None), ARG), (dict(W_ld=5), ARG),
    (dict(gate_out=None), ARG), (dict(up_out=None), ARG), (dict(out=P(2)), ARG), (dict(gate_out=P(5)), ARG),
    (dict(keep_ld=47), ARG)])
def test_gated_refusals(kw, want):
    _refused("tp_gated_linear", _gated(**kw), want)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(F=0), ARG), (dict(W_up=None), ARG), (dict(gate=None), ARG), (dict(up=None), ARG), (dict(dOut=None), ARG),
    (dict(dW_up=None), ARG), (dict(dW_gate=None), ARG), (dict(ws=None), ARG), (dict(ws_bytes=12287), ARG),
    (dict(dX=P(5)), ARG), (dict(dW_up=P(7)), ARG), (dict(accumulate=1, dw_dtype=tp.TP_BF16), ARG), (dict(ws=P(4)), ARG)])
def test_gated_backward_refusals(kw, want):
    _refused("tp_gated_linear_backward", _gated_bwd(**kw), want)


def test_null_structures():
    lib = _abi.load()
    n = C.c_int64()
    for fn in ("tp_linear", "tp_linear_backward", "tp_gated_linear", "tp_gated_linear_backward"):
        assert getattr(lib, fn)(None, None) == ARG
    for fn in ("tp_linear_backward_ws", "tp_gated_linear_backward_ws"):
        assert getattr(lib, fn)(None, C.byref(n)) == ARG


def test_workspace_sizes():
    lib = _abi.load()
    n = C.c_int64()

    def size(fn, args):
        assert getattr(lib, fn)(C.byref(args), C.byref(n)) == 0, lib.tp_last_error()
        return n.value
    # No activation and no bias gradient: nothing to keep.
    assert size("tp_linear_backward_ws", _linear_bwd(act=0, dbias=None)) == 0
    assert size("tp_linear_backward_ws", _linear_bwd(dbias=None)) >= 64 * 48 * 2
    assert size("tp_linear_backward_ws", _linear_bwd(M=0)) == 0
    assert size("tp_linear_backward_ws", _linear_bwd()) >= 64 * 48 * 2 + 48 * 4
    assert size("tp_gated_linear_backward_ws", _gated_bwd()) >= 2 * 64 * 48 * 2
    # Whatever the rows, the bias gradient's partials stay within 1024 of them (past 64 rows each).
    assert size("tp_linear_backward_ws", _linear_bwd(act=0, dX=None, dW=None, M=1 << 20)) <= 1024 * 48 * 4


@pytest.mark.parametrize("gap,rc", [(47, ARG), (48, None), (52, None), (53, ARG)])
def test_interleaved_columns_share_nothing(gap, rc):
    """Column blocks of one [64, 100] matrix: apart when neither reaches into the other nor round the row's end."""
    lib = _abi.load()
    # (a bad later argument, so that nothing is enqueued where the outputs are fine)
    a = _gated(F=48, out_ld=100, keep_ld=100, gate_out=P(3) + 2 * gap, up_out=P(3) + 2 * gap)
    assert lib.tp_gated_linear(C.byref(a), None) == ARG
    msg = lib.tp_last_error().decode()
    assert msg == ("gate_out overlaps out" if rc else "up_out overlaps gate_out")


def test_empty_forward_is_a_no_op():
    lib = _abi.load()
    assert lib.tp_linear(C.byref(_linear(M=0, X=None, out=None, residual=None, pre_out=None)), None) == 0
    assert lib.tp_gated_linear(C.byref(_gated(M=0, X=None, out=None, gate_out=None, up_out=None)), None) == 0


def _grads(*rows):
    arr = (_abi.tp_grad_tensor * max(1, len(rows)))()
    for i, r in enumerate(rows):
        arr[i] = _abi.tp_grad_tensor(*r)
    return arr, len(rows)


G = (P(0), P(1), 1000, tp.TP_F32)


@pytest.mark.parametrize("rows", [
    [(P(0), P(1), 1000, 9)], [(P(0), P(1), -1, 0)], [(None, P(1), 5, 0)], [(P(0), None, 5, 0)],
    [(P(0) + 2, P(1), 5, 0)], [(P(0), P(1) + 1, 5, 1)],
    [(P(0), P(0) + 4, 1000, 0)],                                   # shifted onto itself
    [G, (P(2), P(1) + 3996, 10, 0)],                               # two outputs overlap
    [G, (P(1) + 400, P(3), 10, 0)],                                # an output over another gradient
    [(P(0), P(8), 10, 0)]])                                        # an output over the partial sums
def test_clip_refusals(rows):
    lib = _abi.load()
    arr, n = _grads(*rows)
    assert lib.tp_grad_clip(arr, n, P(8), 1, 1.0, 1e-6, P(9), None) == ARG
    assert lib.tp_last_error()


@pytest.mark.parametrize("kw", [dict(parts=None), dict(parts=P(8) + 4), dict(ranks=0), dict(ranks=65), dict(max_norm=-1.0),
                                dict(max_norm=float("nan")), dict(eps=-1e-9), dict(eps=float("nan")), dict(norm=P(9) + 2),
                                dict(norm=P(8) + 8), dict(norm=P(1)), dict(num=-1), dict(null=True)])
def test_clip_scalar_refusals(kw):
    lib = _abi.load()
    arr, n = _grads(G)
    if kw.get("null"):
        arr = None
    assert lib.tp_grad_clip(arr, kw.get("num", n), kw.get("parts", P(8)), kw.get("ranks", 1), kw.get("max_norm", 1.0),
                            kw.get("eps", 1e-6), kw.get("norm", P(9)), None) == ARG


@pytest.mark.parametrize("rows,parts", [([(P(0), None, 10, 9)], P(8)), ([(None, None, 10, 0)], P(8)), ([G], None),
                                        ([G], P(0) + 8), ([(P(0), None, -1, 0)], P(8))])
def test_sumsq_refusals(rows, parts):
    arr, n = _grads(*rows)
    assert _abi.load().tp_grad_sumsq(arr, n, parts, None) == ARG


def test_binding_refusals():
    """Shapes, dtypes, strides and devices are checked before a pointer is taken."""
    bf, f = torch.bfloat16, torch.float32

    def t(*shape, dtype=bf):
        return torch.zeros(shape, dtype=dtype)
    X, W, out = t(4, 8), t(8, 16), t(4, 16)
    for kw in (dict(W=t(16, 8)), dict(out=t(4, 8)), dict(bias=t(8, dtype=f)), dict(residual=t(4, 8)),
               dict(W=t(8, 32)[:, ::2]), dict(out=t(4, 1).expand(4, 16)), dict(pre_out=t(5, 16)),
               dict()):    # all well, but on the CPU
        a = dict(X=X, W=W, out=out)
        a.update(kw)
        with pytest.raises(ValueError):
            tp.tp_linear(**a)
    for kw in (dict(W=t(8, 16, dtype=f)), dict(bias=t(16)), dict(out=t(4, 16, dtype=torch.float16)),
               dict(residual=t(4, 16, dtype=f)), dict(X=t(4, 8, dtype=torch.float16))):
        a = dict(X=X, W=W, out=out)
        a.update(kw)
        with pytest.raises(TypeError):
            tp.tp_linear(**a)
    wide = t(8, 64)
    with pytest.raises(ValueError, match="one row stride"):
        tp.tp_gated_linear(X, wide[:, :16], t(8, 16), out)
    with pytest.raises(ValueError):
        tp.tp_gated_linear(X, t(8, 16), t(8, 15), out)
    with pytest.raises(ValueError):
        tp.tp_grad_sumsq([t(4)], torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        tp.tp_grad_clip([t(4)], [t(5)], torch.zeros(1024, dtype=torch.float64), max_norm=1.0)
    with pytest.raises(ValueError):
        tp.tp_grad_clip([t(4), t(4)], [t(4)], torch.zeros(1024, dtype=torch.float64), max_norm=1.0)
