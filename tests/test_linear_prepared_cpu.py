"""A prepared forward call's own workspace and the streams that use it, with stand-ins for the GPU's tensors and streams:
it is zeroed before the call can be replayed anywhere, other streams are recorded with the allocator, and a capture, which
cannot wait, goes without."""
import ctypes as C

import pytest
import torch

from sharded_gemm_amd import _abi


class Stream:
    def __init__(self, ptr, log):
        self.cuda_stream, self._log = ptr, log

    def synchronize(self):
        self._log.append(("synchronize", self.cuda_stream))


class Workspace:
    device = torch.device("cuda", 0)

    def __init__(self, n, log):
        self._n, self._log = n, log

    def is_contiguous(self):
        return True

    def numel(self):
        return self._n

    def element_size(self):
        return 1

    def data_ptr(self):
        return 1 << 40

    def record_stream(self, stream):
        self._log.append(("record", stream))


@pytest.fixture
def gpu(monkeypatch):
    """The log of what happens on a stand-in GPU whose current stream is 7."""
    log = []
    state = dict(log=log, capturing=False)

    def zeros(n, **kw):
        log.append(("zeros", n))
        return Workspace(n, log)
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(7, log))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(_abi, "_torch_stream", lambda ptr, device: ptr, raising=False)
    monkeypatch.setattr(_abi, "_ws_bytes", lambda fn, args: 4096)
    return state


def forward_ws(stream=None, ws=None, prepare=True):
    args = _abi.tp_linear_args()
    r = _abi._forward_ws(None, args, ws, "cuda", stream, prepare)
    return args, r


def test_zeroed_before_any_stream_can_use_it(gpu):
    args, _ = forward_ws()
    assert gpu["log"] == [("zeros", 4096), ("synchronize", 7)]
    assert (args.ws, args.ws_bytes) == (1 << 40, 4096)


def test_none_during_a_capture(gpu):
    gpu["capturing"] = True
    args, (ws, own) = forward_ws()
    assert gpu["log"] == [] and ws is None and not own and not args.ws and args.ws_bytes == 0


def test_a_given_workspace_is_the_callers(gpu):
    mine = Workspace(100, gpu["log"])
    args, (ws, own) = forward_ws(ws=mine)
    assert ws is mine and not own and args.ws_bytes == 100 and gpu["log"] == []
    assert forward_ws(prepare=False)[1] == (None, False)


def test_replays_on_other_streams_are_recorded_once(gpu):
    ran = []
    call = _abi.Prepared(lambda s: ran.append(s.value) or 0, (), [], [C.c_void_p(7)], (), Workspace(64, gpu["log"]))
    for s in (7, 9, 9, None, 0, 9):
        call(*([] if s is None else [s]))
    assert ran == [7, 9, 9, 7, None, 9]
    assert gpu["log"] == [("record", 9), ("record", None)]


def test_a_stream_given_at_prepare_is_recorded(gpu):
    call = _abi.Prepared(lambda s: 0, (), [], [C.c_void_p(11)], (), Workspace(64, gpu["log"]))
    call()
    assert gpu["log"] == [("record", 11)]
