"""Refusals of the vocabulary cross entropy and the AdamW step: every bad argument is turned down before anything is
enqueued (no GPU here), by the C entry points and by the binding."""
import ctypes as C

import pytest
import torch

import sharded_gemm_amd as tp
from sharded_gemm_amd import _abi

BASE = 1 << 40          # a made-up address: no call below may get as far as using it
STEP = 1 << 24
ARG, UNS = _abi.TP_ERR_ARG, _abi.TP_ERR_UNSUPPORTED


def P(i):
    return BASE + i * STEP


@pytest.fixture(autouse=True)
def _no_visible_gpu():
    if torch.cuda.is_available():
        pytest.skip("validation tests with made-up device addresses run on hosts without a GPU")


def _ce(**kw):
    a = dict(dtype=tp.TP_BF16, weight_layout=0, M=64, V=48, K=32, X=P(0), W=P(1), targets=P(2), stats=P(3), loss=P(4), lse=P(5),
             ws=P(6), ws_bytes=1 << 20)
    a.update(kw)
    return _abi.tp_linear_ce_args(**a)


def _bwd(**kw):
    a = dict(dtype=tp.TP_BF16, weight_layout=0, dx_dtype=tp.TP_BF16, dw_dtype=tp.TP_F32, M=64, V=48, K=32, X=P(0), W=P(1),
             targets=P(2), lse=P(3), dloss=P(4), dloss_stride=1, dlse=P(5), dlse_stride=0, dX=P(6), dW=P(7), ws=P(8),
             ws_bytes=1 << 20)
    a.update(kw)
    return _abi.tp_linear_ce_bwd_args(**a)


def _refused(rc, want):
    lib = _abi.load()
    assert rc == want, (rc, lib.tp_last_error())
    assert lib.tp_last_error()


COMMON = [(dict(dtype=7), ARG), (dict(weight_layout=2), ARG), (dict(M=-1), ARG), (dict(V=0), ARG), (dict(K=0), ARG),
          (dict(M=1 << 31), UNS), (dict(V=1 << 31), UNS), (dict(K=1 << 24), UNS), (dict(M=1 << 28, K=1 << 10), UNS), (dict(X=None), ARG), (dict(W=None), ARG),
          (dict(targets=None), ARG), (dict(X=P(0) + 1), ARG), (dict(targets=P(2) + 4), ARG), (dict(X_ld=31), ARG), (dict(X_ld=1 << 31), UNS),
          (dict(W_ld=47), ARG), (dict(vocab_begin=-1), ARG), (dict(vocab_begin=2 ** 63 - 40), ARG), (dict(ws=None), ARG), (dict(ws_bytes=100), ARG)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(stats=None, loss=None, lse=None), ARG), (dict(loss=P(4) + 2), ARG), (dict(loss=P(0)), ARG), (dict(lse=P(1) + 64), ARG),
    (dict(stats=P(4)), ARG), (dict(lse=P(2)), ARG), (dict(ws=P(6) + 8), ARG), (dict(ws=P(5)), ARG), (dict(ws=P(0)), ARG)])
def test_forward_refusals(kw, want):
    _refused(_abi.load().tp_linear_ce(C.byref(_ce(**kw)), None), want)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(dx_dtype=9), ARG), (dict(dw_dtype=9), ARG), (dict(dtype=tp.TP_F32, dx_dtype=tp.TP_BF16), ARG), (dict(lse=None), ARG), (dict(lse=P(3) + 2), ARG),
    (dict(dloss=P(4) + 1), ARG), (dict(dloss_stride=2), ARG), (dict(dlse_stride=-1), ARG), (dict(accumulate=2), ARG),
    (dict(accumulate=1, dw_dtype=tp.TP_BF16), ARG), (dict(piece=-1), ARG), (dict(dX=P(0)), ARG), (dict(dW=P(6)), ARG), (dict(dW=P(1)), ARG),
    (dict(dX=P(3)), ARG), (dict(dX_ld=31), ARG), (dict(dW_ld=47), ARG), (dict(ws=P(8) + 8), ARG), (dict(ws=P(7)), ARG), (dict(dW=P(5)), ARG)])
def test_backward_refusals(kw, want):
    _refused(_abi.load().tp_linear_ce_backward(C.byref(_bwd(**kw)), None), want)


@pytest.mark.parametrize("kw", [dict(pieces=0), dict(pieces=65), dict(M=-1), dict(stats=None), dict(targets=None), dict(loss=None, lse=None), dict(loss=P(0)),
                                dict(lse=P(2)), dict(stats=P(0) + 2), dict(targets=P(1) + 4)])
def test_join_refusals(kw):
    a = dict(stats=P(0), pieces=2, M=100, targets=P(1), loss=P(2), lse=P(3)) | kw
    rc = _abi.load().tp_ce_join(a["stats"], a["pieces"], a["M"], a["targets"], 0, a["loss"], a["lse"], None)
    _refused(rc, ARG)


def test_null_structures_and_workspaces():
    lib, n = _abi.load(), C.c_int64()
    for fn in ("tp_linear_ce", "tp_linear_ce_backward"):
        assert getattr(lib, fn)(None, None) == ARG
    for fn in ("tp_linear_ce_ws", "tp_linear_ce_backward_ws"):
        assert getattr(lib, fn)(None, C.byref(n)) == ARG

    def size(fn, args):
        assert getattr(lib, fn)(C.byref(args), C.byref(n)) == 0, lib.tp_last_error()
        return n.value
    assert size("tp_linear_ce_ws", _ce(M=0)) == 0
    # A pair for every 128 columns of a row, not the logits.
    assert size("tp_linear_ce_ws", _ce(M=8192, V=131072, K=4096, weight_layout=1)) < 8192 * (1024 + 16) * 8 + (1 << 20)
    # The gradient at one piece's logits, X^T and dX's sum: less with smaller pieces, not the whole vocabulary's.
    big = dict(M=8192, V=131072, K=4096, weight_layout=1, dw_dtype=tp.TP_BF16)
    keeps = 8192 * 4096 * (2 + 4)
    assert size("tp_linear_ce_backward_ws", _bwd(**big)) <= 2 * (1 << 28) + keeps + (1 << 20)
    assert size("tp_linear_ce_backward_ws", _bwd(piece=4096, **big)) <= 2 * 8192 * 4096 + keeps + (1 << 20)
    assert size("tp_linear_ce_backward_ws", _bwd(dX=None, dW=None)) == 0


def _tensor(**kw):
    a = dict(param=P(0), grad=P(1), m=P(2), v=P(3), m_scale=P(4), v_scale=P(5), copy=P(6), n=1000, param_dtype=tp.TP_F32,
             grad_dtype=tp.TP_F32, weight_decay=0.1)
    a.update(kw)
    return _abi.tp_adamw_tensor(**a)


def _args(**kw):
    a = dict(states=tp.TP_ADAMW_F32, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, ranks=1, max_norm=1.0)
    a.update(kw)
    return _abi.tp_adamw_args(**a)


@pytest.mark.parametrize("kw", [dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=P(0) + 2), dict(grad=P(1) + 1), dict(m=P(2) + 2),
                                dict(copy=P(6) + 1), dict(n=-1), dict(n=1 << 48), dict(param_dtype=5), dict(grad_dtype=5), dict(weight_decay=-0.1),
                                dict(weight_decay=float("nan")), dict(m=P(0)), dict(v=P(2) + 2000), dict(copy=P(1)), dict(grad=P(0))])
def test_step_refusals_of_a_tensor(kw):
    arr = (_abi.tp_adamw_tensor * 1)(_tensor(**kw))
    _refused(_abi.load().tp_adamw_step(arr, 1, C.byref(_args()), None), ARG)


@pytest.mark.parametrize("kw", [dict(m_scale=None), dict(v_scale=None), dict(m_scale=P(4) + 2), dict(v_scale=P(4) + 8), dict(m_scale=P(2) + 996)])
def test_step_refusals_of_8_bit_states(kw):
    arr = (_abi.tp_adamw_tensor * 1)(_tensor(**kw))
    _refused(_abi.load().tp_adamw_step(arr, 1, C.byref(_args(states=tp.TP_ADAMW_8BIT)), None), ARG)


@pytest.mark.parametrize("kw", [dict(states=2), dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")),
                                dict(eps=-1e-9), dict(step=0), dict(step_dev=P(9) + 4), dict(lr_dev=P(9) + 2), dict(norm_out=P(9)), dict(skip_nonfinite=1),
                                dict(skip_nonfinite=2), dict(parts=P(9) + 4), dict(parts=P(9), ranks=0), dict(parts=P(9), ranks=65),
                                dict(parts=P(9), max_norm=-1.0), dict(parts=P(9), clip_eps=float("nan")), dict(parts=P(0)), dict(parts=P(9), norm_out=P(9)),
                                dict(parts=P(9), norm_out=P(8) + 2), dict(step_dev=P(2)), dict(lr_dev=P(0) + 400)])
def test_step_refusals_of_the_rest(kw):
    arr = (_abi.tp_adamw_tensor * 1)(_tensor())
    _refused(_abi.load().tp_adamw_step(arr, 1, C.byref(_args(**kw)), None), ARG)


def test_step_refusals_of_the_list():
    lib = _abi.load()
    arr = (_abi.tp_adamw_tensor * 2)(_tensor(), _tensor(param=P(10), m=P(12), v=P(13), copy=P(6) + 1990))
    _refused(lib.tp_adamw_step(arr, 2, C.byref(_args()), None), ARG)          # two tensors' copies overlap
    _refused(lib.tp_adamw_step(arr, -1, C.byref(_args()), None), ARG)
    _refused(lib.tp_adamw_step(None, 1, C.byref(_args()), None), ARG)
    _refused(lib.tp_adamw_step(arr, 1, None, None), ARG)


@pytest.mark.parametrize("kw", [dict(m=None), dict(v_scale=None), dict(m_out=None), dict(n=-1), dict(out_dtype=4), dict(m_out=P(4) + 2), dict(v_out=P(4) + 8),
                                dict(m_out=P(0))])
def test_unpack_refusals(kw):
    a = dict(m=P(0), v=P(1), m_scale=P(2), v_scale=P(3), m_out=P(4), v_out=P(5), n=1000, out_dtype=tp.TP_F32) | kw
    arr = (_abi.tp_adamw_state * 1)(_abi.tp_adamw_state(**a))
    _refused(_abi.load().tp_adamw_unpack(arr, 1, None), ARG)


# ---- the binding -----------------------------------------------------------------

def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_wrong_tensors_of_the_cross_entropy():
    X, W, t = _t(4, 8), _t(8, 16), _t(4, dtype=torch.int64)
    ok = dict(loss=_t(4), ws=_t(8192, dtype=torch.uint8))
    with pytest.raises(ValueError, match="current GPU"):
        tp.tp_linear_ce(X, W, t, **ok)
    for args, kw, err in (((X, W, t.int()), ok, TypeError), ((X, W, t[:3]), ok, ValueError), ((X, W.bfloat16(), t), ok, TypeError),
                          ((X, W, None), ok, TypeError), ((X, W[:7], t), ok, ValueError), ((X, W, t), ok | dict(loss=_t(5)), ValueError),
                          ((X, W, t), ok | dict(lse=_t(4).double()), TypeError), ((X, W, t), ok | dict(stats=_t(4, 3)), ValueError),
                          ((X, W, t), ok | dict(loss=_t(4, 2)[:, 0]), ValueError), ((X.half(), W.half(), t), ok, TypeError)):
        with pytest.raises(err):
            tp.tp_linear_ce(*args, **kw)
    with pytest.raises(TypeError):
        tp.tp_ce_join(_t(3, 4), t, loss=_t(4))
    with pytest.raises(ValueError):
        tp.tp_ce_join(_t(2, 2, 4), t, loss=_t(4))
    lse, ws = _t(4), _t(1 << 20, dtype=torch.uint8)
    for kw, err in ((dict(dloss=_t(3)), ValueError), (dict(dloss=_t(4).double()), TypeError), (dict(dlse=0.5), TypeError), (dict(dX=_t(4, 9)), ValueError),
                    (dict(dW=_t(16, 8)), ValueError), (dict(dX=_t(4, 8).half()), TypeError), (dict(dX=_t(4, 8), ws=ws[::2]), ValueError)):
        with pytest.raises(err):
            tp.tp_linear_ce_backward(X, W, t, lse, **(dict(ws=ws) | kw))


def test_binding_refuses_wrong_tensors_of_the_step():
    p, i8, u8 = _t(300), _t(300, dtype=torch.int8), _t(300, dtype=torch.uint8)
    s = _t(2)
    ok = dict(params=[p], grads=[p], m=[p], v=[p], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="current GPU"):
        tp.tp_adamw_step(**ok)
    for kw, err in ((dict(grads=[]), ValueError), (dict(m=[]), ValueError), (dict(v=[_t(299)]), ValueError), (dict(m=[i8]), TypeError),
                    (dict(m=[i8], v=[u8]), ValueError), (dict(m=[i8], v=[u8], m_scale=[s], v_scale=[_t(3)]), ValueError),
                    (dict(m=[i8], v=[i8], m_scale=[s], v_scale=[s]), TypeError), (dict(m_scale=[s], v_scale=[s]), TypeError),
                    (dict(copies=[p]), ValueError), (dict(weight_decay=[0.1, 0.1]), ValueError), (dict(parts=_t(1024).double()), ValueError),
                    (dict(max_norm=1.0), ValueError), (dict(step=_t(1)), TypeError), (dict(lr=_t(1).double()), TypeError), (dict(norm_out=_t(2)), ValueError),
                    (dict(params=[_t(600)[::2]]), ValueError), (dict(params=[p.half()]), TypeError), (dict(grads=[_t(20)]), ValueError)):
        with pytest.raises(err):
            tp.tp_adamw_step(**(ok | kw))
    with pytest.raises(ValueError):
        tp.tp_adamw_unpack([i8], [u8], [p], [_t(300).bfloat16()], m_scale=[s], v_scale=[s])
