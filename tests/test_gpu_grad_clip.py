"""The global gradient norm and clipping on the GPU, against their float64 form.

The squares are summed in 64 bits, so the norm is exact to far below fp32 and norm_out is off by its own rounding
(u(fp32), and 2^-40 for the sum); a clipped element by the factor's rounding and the product's (2 u(fp32)), and
half a step of its type.
"""
import math

import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import linear as O

from gpu_helpers import Guarded, announce, bits, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U32 = torch.finfo(F32).eps / 2


def setup_module(_):
    require_gpu()


def f64(t):
    return t.detach().cpu().double().numpy()


def rnd(n, seed, dtype, std=1.0):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def run(grads, max_norm, *, in_place=False, eps=1e-6, outs=None):
    parts, norm = tp.tp_grad_parts(), Guarded((1,), F32)
    outs = grads if in_place else outs or [torch.empty_like(g) for g in grads]
    tp.tp_grad_sumsq(grads, parts)
    tp.tp_grad_clip(grads, None if in_place else outs, parts, max_norm=max_norm, eps=eps, norm_out=norm.t)
    torch.cuda.synchronize()
    assert norm.guards_intact()
    return float(norm.t), outs


def check(host, got_norm, outs, max_norm, eps=1e-6):
    norm, want = O.clip([f64(g) for g in host], max_norm, eps)
    assert abs(got_norm - norm) <= (U32 + 2.0 ** -40) * norm
    for g, o, w in zip(host, outs, want):
        u = torch.finfo(g.dtype).eps / 2
        tol = 2 * U32 * np.abs(w) + u * np.abs(w) * (1 + 2 * U32) + (torch.finfo(g.dtype).smallest_normal * u * 2)
        assert (np.abs(f64(o) - w) <= tol).all()


SIZES = [[1], [0, 1, 0], [4096], [4095, 4097, 1, 15, 16, 17], [100, 1 << 20, 3, 12345], [7] * 63, [9] * 64, [5] * 65,
         [1000 + i for i in range(200)], [5_000_001]]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(sizes, kind, in_place):
    announce(f"clip {len(sizes)} tensors {kind} in_place {in_place}")
    dts = [F32 if kind == "f32" or (kind == "mixed" and i % 2) else BF16 for i in range(len(sizes))]
    host = [rnd(n, 100 + i, dt, 0.5) for i, (n, dt) in enumerate(zip(sizes, dts))]
    for limit in (0.25, 1e9):     # clipped, and below the limit
        norm, outs = run([h.cuda() for h in host], limit, in_place=in_place)
        check(host, norm, outs, limit)
        if limit == 1e9:
            assert all(torch.equal(o.cpu(), h) for o, h in zip(outs, host))


def test_no_tensors():
    assert run([], 1.0)[0] == 0.0
    assert run([torch.empty(0, device="cuda")], 1.0)[0] == 0.0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_alignment(dtype):
    """Tensors that start at any element, and outputs that do: nothing beside them is read or written."""
    for start in range(1, 9):
        n = 4096 * 3 + 5
        base = torch.full((n + 64,), float("nan"), dtype=dtype, device="cuda")
        base[start:start + n] = rnd(n, start, dtype).cuda()
        dst = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
        norm, _ = run([base[start:start + n]], 1.0, outs=[dst[9 - start:9 - start + n]])
        check([base[start:start + n].cpu()], norm, [dst[9 - start:9 - start + n]], 1.0)
        assert bool((dst[:9 - start] == 7.0).all()) and bool((dst[9 - start + n:] == 7.0).all())


def test_range_of_fp32():
    """Squares beyond fp32's range on both sides."""
    for scale in (1e30, 1e-30, 3e-39):
        h = [torch.tensor([3.0, 4.0]) * scale]
        norm, outs = run([h[0].cuda()], 1e-40 if scale < 1 else 1.0, eps=0.0)
        assert abs(norm - 5 * float(h[0][0]) / 3) <= 1e-6 * norm + 2e-45


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_not_finite(bad):
    h = rnd(10_000, 3, F32)
    h[9_999] = bad
    norm, outs = run([h.cuda(), rnd(5, 4, BF16).cuda()], 1.0)
    if math.isnan(bad):
        assert math.isnan(norm) and all(bool(torch.isnan(o).all()) for o in outs)
    else:
        assert norm == float("inf")
        assert bool((outs[0][:-1] == 0).all()) and math.isnan(float(outs[0][-1])) and bool((outs[1] == 0).all())


def test_zero_limit_and_zero_gradients():
    assert bool((run([rnd(100, 1, F32).cuda()], 0.0)[1][0] == 0).all())
    norm, outs = run([torch.zeros(5000, device="cuda")], 1.0)
    assert norm == 0.0 and bool((outs[0] == 0).all())
    # 0 / 0: the formula's NaN
    norm, outs = run([torch.zeros(5, device="cuda")], 0.0, eps=0.0)
    assert norm == 0.0 and bool(torch.isnan(outs[0]).all())


@pytest.mark.parametrize("ranks", [2, 8, 64])
def test_ranks(ranks):
    """Each rank's partials side by side, or added: the norm of all shards together."""
    shards = [rnd(3000 + r, 40 + r, F32) for r in range(ranks)]
    parts = tp.tp_grad_parts(ranks)
    for r, h in enumerate(shards):
        tp.tp_grad_sumsq([h.cuda()], parts[r * tp.TP_GRAD_PARTS:(r + 1) * tp.TP_GRAD_PARTS])
    norm, mine = torch.empty(1, device="cuda"), shards[1].cuda()
    tp.tp_grad_clip([mine], None, parts, max_norm=1.0, norm_out=norm, ranks=ranks)
    added = parts.view(ranks, -1).sum(0)
    norm2, mine2 = torch.empty(1, device="cuda"), shards[1].cuda()
    tp.tp_grad_clip([mine2], None, added, max_norm=1.0, norm_out=norm2)
    torch.cuda.synchronize()
    want = math.sqrt(sum(float((f64(h) ** 2).sum()) for h in shards))
    for n, m in ((norm, mine), (norm2, mine2)):
        assert abs(float(n) - want) <= (U32 + 2.0 ** -40) * want
        assert np.abs(f64(m) - f64(shards[1]) / (want + 1e-6)).max() <= 4 * U32 * np.abs(f64(shards[1])).max() / want


def test_same_bits_every_time():
    g = [rnd(1_000_003, 1, F32).cuda(), rnd(77_777, 2, BF16).cuda()]
    a = run(g, 0.1)
    for _ in range(3):
        b = run(g, 0.1)
        assert a[0] == b[0] and all(np.array_equal(bits(x), bits(y)) for x, y in zip(a[1], b[1]))
