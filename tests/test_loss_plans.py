"""Which kernels the vocabulary cross entropy takes at sizes that no GPU test runs: the host code alone, built as in
test_loss_host.py."""
import ctypes as C

import pytest
import torch

import sharded_gemm_amd as tp
from sharded_gemm_amd import _abi

from test_loss_host import driver  # noqa: F401  (the fixture)

LARGE = ("tile256", "tile192", "tile128w")


def kernels(driver, *cases):  # noqa: F811
    out, _ = driver("choose", text="\n".join(" ".join(map(str, c)) for c in cases))
    return [line.split("; ") for line in out.strip().split("\n")]


# Weights [V, K] past 2^31 bytes, whose pieces have to stay below: M, K, V; then those of odd K, copied piece by piece.
PAST = [(800, 12288, 131072), (700, 10240, 128000), (512, 4096, 400000), (2048, 8192, 140000), (512, 16384, 70000), (1024, 12288, 131001), (8192, 12288, 262144)]
COPIED = [(700, 4095, 262144), (700, 4095, 262145), (1100, 2047, 600000)]


@pytest.mark.parametrize("M,K,V", PAST + COPIED)
def test_weights_past_the_kernels_offsets_run_on_large_tiles(driver, M, K, V):  # noqa: F811
    forward, backward = kernels(driver, ("ce", "bf16", "linear", M, K, V, 0, 0), ("ce_bwd", "bf16", "linear", M, K, V, 0, 0))
    assert all(k.split()[0] in LARGE for k in forward if "stats" in k)
    assert not [k for k in forward + backward if "general" in k]
    whole = 1 if V % 64 and (M, K, V) in PAST else 0        # the columns past the last 64 are a piece of their own, and small
    for kind in ("prob", "scaled a^T"):
        names = [k for k in backward if kind in k and "split" not in k]
        assert len(names) > whole and all(k.split()[0] in LARGE for k in names[whole:]), (kind, names)
    dx = [k for k in backward if ("slices" in k or "scaled a " in k) and "split" not in k]
    assert all(k.split()[0] in LARGE for k in dx[whole:]), dx


def test_as_with_an_even_piece(driver):  # noqa: F811
    """Pieces chosen below the limit are those that a caller would ask for."""
    for M, K, V, piece in ((800, 12288, 131072, 65536), (700, 10240, 128000, 64000)):
        a, b = kernels(driver, ("ce_bwd", "bf16", "linear", M, K, V, 0, 0), ("ce_bwd", "bf16", "linear", M, K, V, 0, piece))
        assert a == b


@pytest.mark.parametrize("layout", [0, 1])
def test_no_room_for_slices_that_cannot_run(layout):
    """A weight of [K, V] spans all its bytes in every piece: past 2^31 its dX is not cut, and nothing is kept for that."""
    def bytes_of(V):
        n = C.c_int64()
        a = _abi.tp_linear_ce_bwd_args(dtype=tp.TP_BF16, weight_layout=layout, dx_dtype=tp.TP_BF16, M=512, V=V, K=8192, dX=16, piece=8192)
        assert _abi.load().tp_linear_ce_backward_ws(C.byref(a), C.byref(n)) == 0
        return n.value
    part = 512 * 8192 * 4
    if torch.cuda.is_available():
        pytest.skip("on hosts without a GPU, like the driver's tests")
    near, past = bytes_of(8 * 8192), bytes_of(24 * 8192)   # pieces alike; 2^31 bytes are 131072 columns
    assert (near - past >= 2 * part) if layout == 0 else near == past
