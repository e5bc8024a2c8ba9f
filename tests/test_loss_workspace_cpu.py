"""Workspaces of the vocabulary cross entropy (host only): one that was measured for a full batch serves any fewer tokens,
and the backward's stay within the bytes that the header states."""
import ctypes as C

import pytest
import torch

import sharded_gemm_amd as tp
from sharded_gemm_amd import _abi

BASE, STEP = 1 << 40, 1 << 38          # made-up addresses: no call below gets as far as using them


def P(i):
    return BASE + i * STEP


@pytest.fixture(autouse=True)
def _no_visible_gpu():
    if torch.cuda.is_available():
        pytest.skip("validation tests with made-up device addresses run on hosts without a GPU")


def forward_args(dtype, layout, M, K, V, **kw):
    a = dict(dtype=dtype, weight_layout=layout, M=M, V=V, K=K, X=P(0), W=P(1), targets=P(2), loss=P(3))
    return _abi.tp_linear_ce_args(**(a | kw))


def forward_bytes(dtype, layout, M, K, V):
    n = C.c_int64()
    assert _abi.load().tp_linear_ce_ws(C.byref(forward_args(dtype, layout, M, K, V)), C.byref(n)) == 0
    return n.value


# K, V: split K in few and many tiles, a rank's piece, odd sizes with padded copies, few columns, long and short K,
# several pieces of the weight.
SIZES = [(4096, 65536), (4096, 8192), (4096, 4096), (768, 32000), (1024, 1000), (4095, 32001), (1000, 8000), (4096, 33), (64, 128), (12288, 131072),
         (1021, 10007), (40, 600_000), (20_001, 3000)]
TOKENS = sorted(set([1, 2, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 448, 500, 511, 512, 513, 700, 1000, 1023,
                     1024, 1025, 2000, 4096, 8192, 10_000, 20_000, 32_640, 32_641, 100_000, 300_000] + list(range(64, 1200, 64)) + list(range(1, 70))))


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [tp.TP_BF16, tp.TP_F32])
@pytest.mark.parametrize("K,V", SIZES)
def test_a_full_batch_s_workspace_serves_fewer_tokens(K, V, dtype, layout):
    lib = _abi.load()
    bytes_of = [forward_bytes(dtype, layout, M, K, V) for M in TOKENS]
    assert bytes_of == sorted(bytes_of), [(m, b) for m, b, c in zip(TOKENS, bytes_of, bytes_of[1:]) if b > c]
    # The calls themselves: every check up to the workspace's is passed (the loss lies on X, which is looked at next).
    for full in (100, 500, 1024, 20_000):
        have = forward_bytes(dtype, layout, full, K, V)
        for M in TOKENS:
            if M <= full:
                args = forward_args(dtype, layout, M, K, V, loss=P(0), ws=P(4), ws_bytes=have)
                assert lib.tp_linear_ce(C.byref(args), None) == _abi.TP_ERR_ARG
                assert b"overlaps" in lib.tp_last_error(), (full, M, lib.tp_last_error())


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [tp.TP_BF16, tp.TP_F32])
def test_every_token_count(dtype, layout):
    for K, V in ((4096, 8192), (1000, 8000), (4095, 3000)):
        last = 0
        for M in range(1, 1400):
            n = forward_bytes(dtype, layout, M, K, V)
            assert n >= last, (K, V, M)
            last = n


def backward_bytes(dtype, layout, M, K, V, **kw):
    n, a = C.c_int64(), dict(dtype=dtype, weight_layout=layout, dx_dtype=dtype, M=M, V=V, K=K, dX=16, dW=16)
    assert _abi.load().tp_linear_ce_backward_ws(C.byref(_abi.tp_linear_ce_bwd_args(**(a | kw))), C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [tp.TP_BF16, tp.TP_F32])
@pytest.mark.parametrize("M", [1, 100, 1024, 5000, 32_768, 131_072, 1_048_576])
@pytest.mark.parametrize("K,V,odd", [(1024, 131072, False), (1024, 131001, False), (4095, 131001, True), (12288, 50000, False), (1000, 600_001, True), (300, 100, True)])
def test_the_backward_s_bytes(M, K, V, odd, dtype, layout):
    """What the header says it holds, part by part."""
    if (M + 63) // 64 * ((K + 63) // 64) >= 1 << 22:
        pytest.skip("past the grid")
    es, rows = (2 if dtype == tp.TP_BF16 else 4), (M + 63) // 64 * 64
    odd = dtype == tp.TP_BF16 and (odd or (layout == 0 and V % 8 != 0))
    sums = M * K * 4 * (16 if M < 8192 else 1)
    copies = (2 * M * (K + 63) + min(1 << 31, 2 * (K + 63) * (V + 63))) if odd else 128 * K
    rest = sums + copies + (257 << 20)
    p = min(rows * (V + 63), max(1 << 28, 8192 * rows)) * es
    assert backward_bytes(dtype, layout, M, K, V) <= p + K * rows * es + rest
    assert backward_bytes(dtype, layout, M, K, V, dW=None) <= p + rest
    assert backward_bytes(dtype, layout, M, K, V, piece=2048) <= rows * 2048 * es + K * rows * es + rest
    if dtype == tp.TP_BF16:
        assert backward_bytes(dtype, layout, M, K, V, dx_dtype=tp.TP_F32) <= p + K * rows * es + rest


def test_the_backward_s_bytes_at_sizes_that_are_stated():
    gib = 1 << 30
    assert abs(backward_bytes(tp.TP_BF16, 1, 131_072, 1024, 131_072) / gib - 2.75) < 0.01
    assert abs(backward_bytes(tp.TP_F32, 1, 131_072, 1024, 131_072) / gib - 4.5) < 0.01
    assert abs(backward_bytes(tp.TP_BF16, 1, 1024, 4095, 128_001) / gib - 1.3) < 0.05
