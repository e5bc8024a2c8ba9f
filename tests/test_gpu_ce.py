"""The vocabulary cross entropy on the GPU, both directions, against its float64 form.

Tolerances.  A logit is a sum of K products in fp32 (exact products of bf16 values), 32 of them to a matrix
instruction: off by at most D = (K / 32 + 32) u sum |x w|, u = u(fp32); fp32 products add one u each.  The largest of a
row passes into lse whole; the sum of exponentials adds a few u a term and step (64 u), and lse's own rounding.  A
probability is off by D and the exponent's rounding relatively, dz by that and by half a step of the operands' type,
and the products' sums as the logits'.
"""
import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import loss as O

from gpu_helpers import Guarded, announce, bits, require_gpu
from loss_kernel_cases import CASES

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = torch.finfo(F32).eps / 2
MATH, LINEAR = 0, 1


def setup_module(_):
    require_gpu()


def f64(t):
    return t.detach().cpu().double().numpy()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def make(M, K, V, dtype, seed=0, std=2.0, ignored=0.1, whole=None):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((M, K), generator=g).to(dtype)
    W = (torch.randn((K, V), generator=g) * (std / K ** 0.5)).to(dtype)
    t = torch.randint(0, whole or V, (M,), generator=g)
    t[torch.rand(M, generator=g) < ignored] = -100
    return X, W, t


def lay(W, layout):
    return (W if layout == MATH else W.t().contiguous()).cuda()


def logit_error(X, W, dtype):
    K = X.shape[1]
    return (K / 32 + 32 + (dtype == F32)) * U * (np.abs(f64(X)) @ np.abs(f64(W)))


def forward(X, W, t, layout, *, begin=0, ignore=-100, what=("loss", "lse", "stats"), Wd=None, Xd=None, ws=None):
    Xd = X.cuda() if Xd is None else Xd
    Wd = lay(W, layout) if Wd is None else Wd
    M = Xd.shape[0]
    out = {k: Guarded((3, M) if k == "stats" else (M,), F32) for k in what}
    ws = tp.tp_linear_ce_ws(Xd, Wd, weight_layout=layout) if ws is None else ws
    tp.tp_linear_ce(Xd, Wd, t.cuda(), vocab_begin=begin, ignore_index=ignore, weight_layout=layout, ws=ws,
                    **{k: v.t for k, v in out.items()})
    torch.cuda.synchronize()
    assert all(v.guards_intact() for v in out.values())
    assert not ws.numel() or bool((ws[:4096] == 0).all())
    return {k: v.t for k, v in out.items()}


def check_forward(X, W, t, got, dtype, begin=0, ignore=-100):
    want = O.cross_entropy(f64(X), f64(W), t.numpy(), ignore, begin)
    dz = logit_error(X, W, dtype).max(axis=1)
    tol = dz + 64 * U + 4 * U * np.abs(want["lse"])
    if "lse" in got:
        assert (np.abs(f64(got["lse"]) - want["lse"]) <= tol).all()
    if "loss" in got:
        out = f64(got["loss"])
        lost = np.isinf(want["loss"])
        assert (out[lost] == want["loss"][lost]).all()
        ok = ~lost
        assert (np.abs(out[ok] - want["loss"][ok]) <= 2 * tol[ok] + U * np.abs(want["loss"][ok])).all()
        assert (out[t.numpy() == ignore] == 0).all()
    if "stats" in got:
        top, total, logit = f64(got["stats"])
        assert (np.abs(top - want["stats"][0]) <= dz).all()
        # against its own maximum
        rel = 2 * dz + 64 * U + 4 * U * np.abs(top)
        assert (np.abs(total * np.exp(top - want["stats"][0]) - want["stats"][1]) <= rel * want["stats"][1]).all()
        here = np.isfinite(want["stats"][2])
        assert (logit[~here] == -np.inf).all() and (np.abs(logit[here] - want["stats"][2][here]) <= dz[here]).all()


# M, K, V: the few-row kernel (1 to 16 rows, 64 of a linear weight), the small tiles with and without split K,
# the large ones, and nothing a multiple of anything.
SHAPES = [(1, 64, 1), (1, 64, 33), (3, 768, 1000), (7, 40, 5000), (16, 96, 2049), (17, 64, 4097), (33, 1024, 130), (64, 128, 65),
          (65, 100, 300), (257, 64, 1000), (515, 131, 777), (300, 2048, 200), (1030, 192, 9000), (2000, 64, 2056), (130, 32, 70000),
          (4096, 64, 4104)]


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, layout):
    announce(f"ce forward {shape} {dtype} layout {layout}")
    X, W, t = make(*shape, dtype, seed=sum(shape))
    check_forward(X, W, t, forward(X, W, t, layout), dtype)


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_alignment(dtype, layout):
    """Rows apart, and buffers that begin at any element."""
    for shape, skew, pad in (((70, 96, 500), 1, 3), ((2, 64, 300), 3, 5), ((600, 64, 1200), 0, 8), ((600, 64, 1200), 5, 0)):
        announce(f"ce strided {shape} skew {skew} pad {pad}")
        X, W, t = make(*shape, dtype, seed=5)

        def place(m):
            base = torch.full((m.shape[0] * (m.shape[1] + pad) + 16,), float("nan"), dtype=dtype, device="cuda")
            v = base[skew:skew + m.shape[0] * (m.shape[1] + pad)].view(m.shape[0], m.shape[1] + pad)[:, :m.shape[1]]
            v.copy_(m)
            return v
        Wl = W if layout == MATH else W.t().contiguous()
        check_forward(X, W, t, forward(X, W, t, layout, Xd=place(X), Wd=place(Wl)), dtype)


@pytest.mark.parametrize("what", [("loss",), ("lse",), ("stats",), ("loss", "stats")])
def test_outputs_apart(what):
    X, W, t = make(100, 64, 1000, BF16, seed=3)
    check_forward(X, W, t, forward(X, W, t, LINEAR, what=what), BF16)


@pytest.mark.parametrize("sizes", [[700], [300, 700], [64, 1, 500, 33], [96] * 8])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_pieces(sizes, M):
    """Every piece's statistics joined, in any order, are the whole vocabulary's loss."""
    X, W, t = make(M, 64, sum(sizes), BF16, seed=M)
    begins = np.cumsum([0] + sizes)
    stats = torch.empty((len(sizes), 3, M), device="cuda")
    order = np.random.RandomState(0).permutation(len(sizes))
    for i, k in enumerate(order):
        part = W[:, begins[k]:begins[k + 1]].contiguous()
        stats[i] = forward(X, part, t, MATH, begin=int(begins[k]), what=("stats",))["stats"]
    loss, lse = Guarded((M,), F32), Guarded((M,), F32)
    tp.tp_ce_join(stats, t.cuda(), loss=loss.t, lse=lse.t)
    torch.cuda.synchronize()
    assert loss.guards_intact() and lse.guards_intact()
    check_forward(X, W, t, dict(loss=loss.t, lse=lse.t), BF16)
    only = torch.empty(M, device="cuda")
    tp.tp_ce_join(stats, t.cuda(), lse=only)
    assert np.array_equal(bits(only), bits(lse.t))


def test_targets_at_the_edges():
    """Ids at both ends of a piece, beyond it, and beyond everything; an ignore_index that is an id."""
    X, W, _ = make(12, 64, 100, BF16, seed=1)
    big = 2 ** 63 - 1
    t = torch.tensor([50, 149, 49, 150, 0, big, -big - 1, -1, -100, 77, 100, 51])
    check_forward(X, W, t, forward(X, W, t, LINEAR, begin=50), BF16, begin=50)
    check_forward(X, W, t, forward(X, W, t, LINEAR, begin=50, ignore=77), BF16, begin=50, ignore=77)
    far = forward(X, W, t, LINEAR, begin=big - 100)
    assert float(far["loss"][5]) == float("inf") and bool((far["stats"][2] == -float("inf")).sum() == 12)
    all_off = torch.full((12,), -100)
    assert bool((forward(X, W, all_off, MATH)["loss"] == 0).all())


@pytest.mark.parametrize("M", [4, 130])
def test_far_and_infinite_logits(M):
    """Logits of +-80 and 3000, and infinities: the formula's value, and nobody else's row."""
    K, V = 64, 700
    for layout in (MATH, LINEAR):
        X = torch.zeros((M, K))
        W = torch.zeros((K, V))
        W[0] = torch.linspace(-1, 1, V)
        X[:, 0] = torch.tensor([80.0, -3000.0, 1e-3, float("inf")] * (M // 4) + [1.0] * (M % 4))
        X[1, 1], W[1, 5] = 1.0, -1e30
        t = torch.arange(M) * 5 % V
        X, W = X.to(BF16), W.to(BF16)
        got = forward(X, W, t, layout)
        want = O.cross_entropy(f64(X), f64(W), t.numpy())
        fine = np.isfinite(want["lse"])
        assert (np.isfinite(f64(got["lse"])) == fine).all() and fine.sum() >= M // 2
        # (bf16 products of one term: exact logits, so the maximum and the target's are too)
        tol = 64 * U + 4 * U * np.abs(want["lse"][fine])
        assert (np.abs(f64(got["lse"])[fine] - want["lse"][fine]) <= tol).all()
        # An infinite X against weights of either sign, none of them zero: logits +-inf, lse inf.
        assert np.array_equal(f64(got["lse"])[~fine], want["lse"][~fine]) and np.isposinf(want["lse"][~fine]).all()
    # plus infinity alone, minus infinity alone
    X = torch.ones((3, 32))
    W = torch.zeros((32, 130))
    W[0, 7] = float("inf")
    got = forward(X.to(BF16), W.to(BF16), torch.tensor([0, 7, 8]), MATH)
    assert bool((got["lse"] == float("inf")).all()) and bool(got["loss"][0] == float("inf")) and bool(torch.isnan(got["loss"][1]))
    got = forward(X.to(BF16), torch.full((32, 130), -float("inf")).to(BF16), torch.tensor([0, 7, 8]), MATH)
    assert bool((got["lse"] == -float("inf")).all()) and bool((got["stats"][1] == 0).all())
    # joined with a piece that holds something
    stats = torch.stack([got["stats"], forward(X.to(BF16), torch.zeros((32, 130)).to(BF16), torch.tensor([0, 7, 8]), MATH)["stats"]])
    lse = torch.empty(3, device="cuda")
    tp.tp_ce_join(stats, torch.tensor([0, 7, 8]).cuda(), lse=lse)
    assert np.allclose(f64(lse), np.log(130), rtol=1e-6)


def test_a_sure_row_has_no_negative_loss():
    """One logit far above the others: the loss is zero, not below."""
    X = torch.full((40, 32), 3.0)
    W = torch.zeros((32, 500))
    W[:, 9] = 1.37
    got = forward(X.to(BF16), W.to(BF16), torch.full((40,), 9), LINEAR)
    assert bool((got["loss"].abs() <= 0).all())


# ---- backward --------------------------------------------------------------------

def backward(X, W, t, lse, layout, *, g=None, h=None, begin=0, ignore=-100, dx=None, dw=None, piece=0, accumulate=False, start=None,
             Xd=None, Wd=None):
    dtype = X.dtype
    Xd = X.cuda() if Xd is None else Xd
    Wd = lay(W, layout) if Wd is None else Wd
    dX = Guarded(tuple(Xd.shape), dx or dtype) if dx is not False else None
    dW = Guarded(tuple(Wd.shape), dw or dtype) if dw is not False else None
    if start is not None:
        dW.t.copy_(start if layout == MATH else start.t())
    ws = tp.tp_linear_ce_backward_ws(Xd, Wd, weight_layout=layout, dX=dX.t if dX else None, dW=dW is not None, piece=piece)
    ws.fill_(255)       # need not be cleared
    tp.tp_linear_ce_backward(Xd, Wd, t.cuda(), lse.cuda(), dloss=None if g is None else g.cuda(), dlse=None if h is None else h.cuda(),
                             dX=dX.t if dX else None, dW=dW.t if dW else None, vocab_begin=begin, ignore_index=ignore,
                             weight_layout=layout, accumulate=accumulate, piece=piece, ws=ws)
    torch.cuda.synchronize()
    assert (dX is None or dX.guards_intact()) and (dW is None or dW.guards_intact())
    out = {}
    if dX:
        out["dX"] = dX.t
    if dW:
        out["dW"] = dW.t if layout == MATH else dW.t.t()
    return out


def check_backward(X, W, t, lse, got, g=1.0, h=0.0, begin=0, ignore=-100, start=None):
    dtype = X.dtype
    w = O.cross_entropy_backward(f64(X), f64(W), t.numpy(), f64(lse), g, h, ignore, begin)
    on = (t.numpy() != ignore)
    Xo = np.where(on[:, None], f64(X), 0.0)
    M, K, V = X.shape[0], X.shape[1], W.shape[1]
    far = np.where(on, np.abs(f64(lse)), 0.0)[:, None]
    gh = np.abs(np.broadcast_to(g, (M,)) + np.broadcast_to(h, (M,)))[:, None]
    Wf = f64(W)
    # of q relatively: the logit, 4 u for exp2 and its argument, and |lse| u for the common rounding.
    D = (K / 32 + 32 + 1) * U * (np.abs(Xo) @ np.abs(Wf))
    dq = D + 4 * U * (1 + far + np.abs(Xo @ Wf))
    each = 1.01 * dq * gh * w["q"] + (half(dtype) + 4 * U) * np.abs(w["dz"]) + torch.finfo(dtype).smallest_normal
    adz = np.abs(w["dz"])
    for name, got_t in got.items():
        want = w[name] + (0.0 if name == "dX" or start is None else f64(start))
        if name == "dX":
            tol = each @ np.abs(Wf).T + (V / 32 + 64) * U * (adz @ np.abs(Wf).T)
        else:
            tol = np.abs(Xo).T @ each + (M / 32 + 64) * U * (np.abs(Xo).T @ adz)
        tol = tol + (half(got_t.dtype) + U) * np.abs(want) + torch.finfo(got_t.dtype).smallest_normal
        assert (np.abs(f64(got_t) - want) <= tol).all(), (name, float(np.max(np.abs(f64(got_t) - want) / tol)))


BSHAPES = [(1, 64, 1), (1, 64, 33), (3, 96, 200), (17, 64, 130), (64, 128, 65), (65, 100, 300), (257, 64, 1000), (515, 131, 777),
           (1000, 192, 2049), (300, 320, 5000), (2048, 64, 1152), (130, 1024, 4096), (2300, 520, 2112)]


def lse_for(X, W):
    return torch.from_numpy(O.cross_entropy(f64(X), f64(W), np.zeros(X.shape[0], np.int64))["lse"]).float()


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", BSHAPES, ids=str)
def test_backward(shape, dtype, layout):
    announce(f"ce backward {shape} {dtype} layout {layout}")
    X, W, t = make(*shape, dtype, seed=sum(shape))
    lse = lse_for(X, W)
    M = shape[0]
    g = torch.rand(M, generator=torch.Generator().manual_seed(9)) / M
    got = backward(X, W, t, lse, layout, g=g)
    check_backward(X, W, t, lse, got, g=f64(g))


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("piece", [1, 64, 200, 640])
def test_backward_in_pieces(piece, dtype, layout):
    """Any pieces, dX in its own type or fp32; the vocabulary's end off every multiple."""
    X, W, t = make(150, 96, 1200 - 17, dtype, seed=piece)
    lse = lse_for(X, W)
    for out in (None, F32):
        announce(f"ce backward piece {piece} {dtype} {layout} out {out}")
        check_backward(X, W, t, lse, backward(X, W, t, lse, layout, piece=piece, dx=out, dw=out))


@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_backward_options(layout):
    X, W, t = make(200, 64, 500, BF16, seed=4)
    lse = lse_for(X, W)
    M = 200
    g, h = torch.rand(M), torch.rand(M) - 0.5
    one = torch.tensor([0.37])
    announce("ce backward: gradients at lse, one value for all")
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=g, h=h), g=f64(g), h=f64(h))
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=one, h=h), g=0.37 + 0 * f64(one), h=f64(h))
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=g, h=one), g=f64(g), h=f64(one))
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=one.expand(M)), g=f64(one))
    announce("ce backward: one output")
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, dx=False))
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, dw=False))
    announce("ce backward: accumulated")
    start = torch.randn(64, 500)
    check_backward(X, W, t, lse, backward(X, W, t, lse, layout, dw=F32, accumulate=True, start=start), start=start)


@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_backward_of_pieces_of_the_vocabulary(layout):
    """Two ranks' pieces: dX's partials add up, each has its dW; targets in either, or in neither."""
    X, W, t = make(90, 64, 700, BF16, seed=2)
    t[3] = 700          # no piece's
    lse = lse_for(X, W)
    parts = []
    for a, b in ((0, 300), (300, 700)):
        part = W[:, a:b].contiguous()
        got = backward(X, part, t, lse, layout, begin=a, dx=F32)
        check_backward(X, part, t, lse, got, begin=a)
        parts.append(f64(got["dX"]))
    want = O.cross_entropy_backward(f64(X), f64(W), t.numpy(), f64(lse))
    assert np.linalg.norm(sum(parts) - want["dX"]) <= half(BF16) * np.linalg.norm(np.abs(want["dz"]) @ np.abs(f64(W)).T)


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [5, 64, 200])
def test_ignored_rows_may_hold_anything(M, dtype, layout):
    """A padded batch's rest: NaN and infinities in X, lse and the gradients of ignored rows reach nothing."""
    X, W, t = make(M, 64, 300, dtype, seed=8, ignored=0.0)
    t[1::3] = -100
    lse = lse_for(X, W)
    g = torch.rand(M)
    bad = X.clone()
    bad[1::3] = float("nan")
    bad[1, 0] = float("inf")
    lse[1::3] = float("nan")
    gb = g.clone()
    gb[1::3] = float("nan")
    got = backward(bad, W, t, lse, layout, g=gb, h=gb)
    assert bool((got["dX"][1::3] == 0).all())
    check_backward(X, W, t, torch.nan_to_num(lse), got, g=f64(g), h=f64(g))
    f = forward(bad, W, t, layout)
    assert bool((f["loss"][1::3] == 0).all()) and bool(torch.isfinite(f["loss"]).all())
    everything = backward(bad, W, torch.full((M,), -100), lse, layout, g=gb)
    assert bool((everything["dX"] == 0).all()) and bool((everything["dW"] == 0).all())


@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_no_tokens(layout):
    X, W, t = make(0, 64, 300, BF16)
    assert forward(X, W, t, layout)["loss"].numel() == 0
    got = backward(X, W, t, torch.empty(0), layout)
    assert bool((got["dW"] == 0).all())
    start = torch.randn(64, 300)
    got = backward(X, W, t, torch.empty(0), layout, dw=F32, accumulate=True, start=start)
    assert torch.equal(got["dW"].cpu(), start)


@pytest.mark.parametrize("layout", [MATH, LINEAR])
def test_gradients_against_differences(layout):
    """The loss's own differences along random directions, in fp32."""
    M, K, V = 37, 48, 211
    X, W, t = make(M, K, V, F32, seed=11, std=1.0)
    lse = lse_for(X, W)
    got = backward(X, W, t, lse, layout)
    g = torch.Generator().manual_seed(12)
    for _ in range(4):
        a, b = torch.randn((M, K), generator=g).double().numpy(), torch.randn((K, V), generator=g).double().numpy()
        eps = 1e-5

        def total(s):
            return O.cross_entropy(f64(X) + s * a, f64(W) + s * b, t.numpy())["loss"].sum()
        want = (total(eps) - total(-eps)) / (2 * eps)
        have = (f64(got["dX"]) * a).sum() + (f64(got["dW"]) * b).sum()
        # fp32 results, and the difference's own error (eps^2, and 1e-16 / eps of a sum of some hundreds)
        assert abs(have - want) <= 1e-4 * (np.abs(f64(got["dX"]) * a).sum() + np.abs(f64(got["dW"]) * b).sum()) * 0.1 + 1e-6


# ---- as a program uses it ------------------------------------------------------------

@pytest.mark.parametrize("shape", [(2, 64, 3000), (48, 64, 3000), (700, 128, 3000)])
def test_same_bits_captured_and_eager(shape):
    announce(f"ce captured {shape}")
    X, W, t = make(*shape, BF16, seed=1)
    Xd, Wd, td = X.cuda(), lay(W, LINEAR), t.cuda()
    M = shape[0]
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dX, dW = torch.empty_like(Xd), torch.empty_like(Wd)
    ws = tp.tp_linear_ce_ws(Xd, Wd, weight_layout=LINEAR)
    bws = tp.tp_linear_ce_backward_ws(Xd, Wd, weight_layout=LINEAR, dX=dX, piece=1024)
    fwd = tp.tp_linear_ce(Xd, Wd, td, loss=loss, lse=lse, weight_layout=LINEAR, ws=ws, prepare=True)
    bwd = tp.tp_linear_ce_backward(Xd, Wd, td, lse, dX=dX, dW=dW, weight_layout=LINEAR, piece=1024, ws=bws, prepare=True)
    fwd()
    bwd()
    torch.cuda.synchronize()
    want = [bits(x) for x in (loss, lse, dX, dW)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        fwd(s)
        bwd(s)
    for _ in range(3):
        for x in (loss, lse, dX, dW):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(bits(x), w) for x, w in zip((loss, lse, dX, dW), want))
        fwd()
        bwd()
        torch.cuda.synchronize()
        assert all(np.array_equal(bits(x), w) for x, w in zip((loss, lse, dX, dW), want))


def test_on_another_stream_and_one_workspace_for_many_shapes():
    big = make(300, 64, 5000, BF16, seed=2)
    small = make(5, 64, 700, BF16, seed=3)
    ws = tp.tp_linear_ce_ws(big[0].cuda(), lay(big[1], LINEAR), weight_layout=LINEAR)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for X, W, t in (big, small, big, small):
            check_forward(X, W, t, forward(X, W, t, LINEAR, ws=ws), BF16)


@pytest.mark.parametrize("case", CASES, ids=lambda c: " ".join(map(str, c)))
def test_every_kernel(case):
    """The calls that between them launch every kernel there is."""
    op, dt, layout, M, K, V, odd, piece = case
    announce(f"ce kernels {case}")
    dtype, layout = (BF16 if dt == "bf16" else F32), (MATH if layout == "math" else LINEAR)
    X, W, t = make(M, K, V, dtype, seed=M + K + V)

    def place(m):
        if not odd:
            return m.cuda()
        base = torch.full((m.shape[0] * (m.shape[1] + odd) + 16,), float("nan"), dtype=dtype, device="cuda")
        v = base[odd:odd + m.shape[0] * (m.shape[1] + odd)].view(m.shape[0], m.shape[1] + odd)[:, :m.shape[1]]
        v.copy_(m)
        return v
    Xd, Wd = place(X), place(W if layout == MATH else W.t().contiguous())
    if op == "ce":
        check_forward(X, W, t, forward(X, W, t, layout, Xd=Xd, Wd=Wd), dtype)
    else:
        lse = lse_for(X, W)
        check_backward(X, W, t, lse, backward(X, W, t, lse, layout, piece=piece, Xd=Xd, Wd=Wd))


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1.0, 1e30])
def test_gradients_alike_are_not_rounded_alike(scale, layout):
    """One gradient for all tokens (a mean), whatever its bits: dX and dW are off by roundings that differ from element
    to element, u of their 2-norm for the result's and under half a u for dz's, not by the rounding of that gradient."""
    X, W, t = make(300, 128, 2000, BF16, seed=21, std=1.0)
    lse = lse_for(X, W)
    want = O.cross_entropy_backward(f64(X), f64(W), t.numpy(), f64(lse))
    for f in (1.0, 1.003, 1.0039, 1.5, 1.996):
        got = backward(X, W, t, lse, layout, g=torch.tensor([scale * f]))
        for k in ("dX", "dW"):
            w = want[k] * float(np.float32(scale * f))
            assert np.linalg.norm(f64(got[k]) - w) <= 1.5 * half(BF16) / 3 ** 0.5 * np.linalg.norm(w), (f, k)


def test_gradients_of_many_sizes():
    """Tokens whose gradients differ by 1e6, zeros among them, and penalties far above the losses' gradients."""
    X, W, t = make(200, 64, 500, BF16, seed=22)
    lse = lse_for(X, W)
    g = torch.logspace(-6, 0, 200) * (torch.arange(200) % 7 > 0)
    for layout in (MATH, LINEAR):
        check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=g), g=f64(g))
        check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=g * 1e-20, h=g.flip(0)), g=f64(g * 1e-20), h=f64(g.flip(0)))
        check_backward(X, W, t, lse, backward(X, W, t, lse, layout, g=0 * g, h=g), g=0.0, h=f64(g))
        none = backward(X, W, t, lse, layout, g=0 * g)
        assert bool((none["dX"] == 0).all()) and bool((none["dW"] == 0).all())
        # An infinite gradient is its own row's.
        bad = g.clone()
        bad[5] = float("inf")
        t2 = t.clone()
        t2[5] = 3
        got = backward(X, W, t2, lse, layout, g=bad)["dX"]
        rest = torch.arange(200) != 5
        check_backward(X[rest], W, t2[rest], lse[rest], dict(dX=got[rest.cuda()]), g=f64(g[rest]))
        assert not bool(torch.isfinite(got[5]).any())


def test_all_tokens_ignored():
    for dtype in (BF16, F32):
        X, W, _ = make(130, 64, 700, dtype, seed=23)
        t = torch.full((130,), 5)
        got = forward(X, W, t, MATH, ignore=5)
        assert bool((got["loss"] == 0).all())
        check_forward(X, W, t, dict(lse=got["lse"]), dtype, ignore=5)
        both = backward(X, W, t, torch.full((130,), float("nan")), MATH, g=torch.full((130,), float("inf")), ignore=5)
        assert bool((both["dX"] == 0).all()) and bool((both["dW"] == 0).all())


def test_two_calls_at_once():
    """Two streams, a workspace each, the same operands; against the calls one after another."""
    shapes = [(40, 256, 30000), (900, 192, 4100)]
    sets = []
    for i, shape in enumerate(shapes):
        X, W, t = make(*shape, BF16, seed=30 + i)
        Xd, Wd, td = X.cuda(), lay(W, LINEAR), t.cuda()
        for _ in range(2):
            out = [torch.empty(shape[0], device="cuda") for _ in range(2)] + [torch.empty_like(Xd), torch.empty_like(Wd)]
            calls = [tp.tp_linear_ce(Xd, Wd, td, loss=out[0], lse=out[1], weight_layout=LINEAR, prepare=True,
                                     ws=tp.tp_linear_ce_ws(Xd, Wd, weight_layout=LINEAR)),
                     tp.tp_linear_ce_backward(Xd, Wd, td, out[1], dX=out[2], dW=out[3], weight_layout=LINEAR, prepare=True,
                                              ws=tp.tp_linear_ce_backward_ws(Xd, Wd, weight_layout=LINEAR, dX=out[2]))]
            sets.append((out, calls))
    for _, calls in sets:
        for c in calls:
            c()
    torch.cuda.synchronize()
    want = [[bits(x) for x in out] for out, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for out, _ in sets:
        for x in out:
            x.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for (_, calls), s in zip(sets, streams):
            for c in calls:
                c(s)
    torch.cuda.synchronize()
    for (out, _), w in zip(sets, want):
        assert all(np.array_equal(bits(x), y) for x, y in zip(out, w))


def test_two_graphs_on_one_workspace():
    """Of different sizes, replayed in turn."""
    data = [make(*s, BF16, seed=40 + i) for i, s in enumerate([(3, 96, 5000), (600, 64, 2100)])]
    dev = [(X.cuda(), lay(W, MATH), t.cuda()) for X, W, t in data]
    ws = max((tp.tp_linear_ce_ws(X, W, weight_layout=MATH) for X, W, _ in dev), key=lambda w: w.numel())
    bws = max((tp.tp_linear_ce_backward_ws(X, W, weight_layout=MATH, dX=X, piece=512) for X, W, _ in dev), key=lambda w: w.numel())
    graphs = []
    for X, W, t in dev:
        out = [torch.empty(X.shape[0], device="cuda") for _ in range(2)] + [torch.empty_like(X), torch.empty_like(W)]
        fwd = tp.tp_linear_ce(X, W, t, loss=out[0], lse=out[1], ws=ws, prepare=True)
        bwd = tp.tp_linear_ce_backward(X, W, t, out[1], dX=out[2], dW=out[3], piece=512, ws=bws, prepare=True)
        fwd()
        bwd()
        torch.cuda.synchronize()
        want = [bits(x) for x in out]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s = torch.cuda.current_stream()
            fwd(s)
            bwd(s)
        graphs.append((graph, out, want))
    for _ in range(3):
        for _, out, _ in graphs:
            for x in out:
                x.fill_(float("nan"))
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want in graphs:
            assert all(np.array_equal(bits(x), w) for x, w in zip(out, want))


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("M", [3, 600])
def test_a_weight_past_32_bits(M, layout):
    """5 GB of it, 2.4e9 elements: lse, loss and dX against float64 on the GPU, a piece of the vocabulary at a time; dW
    at both ends and around element 2^31."""
    announce(f"ce long weight {M} layout {layout}")
    K, V = 4096, 600_000 - 8 * (M > 3)
    g = torch.Generator("cuda").manual_seed(M)
    X = torch.randn((M, K), generator=g, device="cuda").to(BF16)
    W = torch.empty((K, V) if layout == MATH else (V, K), dtype=BF16, device="cuda").normal_(0, K ** -0.5, generator=g)

    def part(n, m):
        return (W[:, n:n + m] if layout == MATH else W[n:n + m].t()).double()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[0], t[1], t[2] = V - 1, 0, 2 ** 31 // K
    got = forward(X, None, t, layout, Xd=X, Wd=W)
    step, x = 20_000, X.double()
    each, logit, most = [], torch.empty(M, dtype=torch.float64, device="cuda"), 0.0
    for n in range(0, V, step):
        z = x @ part(n, step)
        each.append(z.logsumexp(1))
        here = (t >= n) & (t < n + z.shape[1])
        logit[here] = z[here, t[here] - n]
        most = max(most, float((x.abs() @ part(n, step).abs()).max()))
    lse = torch.stack(each).logsumexp(0)
    D = (K / 32 + 32) * U * most
    tol = D + 64 * U + 4 * U * lse.abs()
    assert bool(((got["lse"] - lse).abs() <= tol).all())
    assert bool(((got["loss"] - (lse - logit)).abs() <= 2 * tol + U * (lse - logit).abs()).all())

    dX, dW = torch.empty_like(X), torch.empty_like(W)
    ws = tp.tp_linear_ce_backward_ws(X, W, weight_layout=layout, dX=dX)
    tp.tp_linear_ce_backward(X, W, t, got["lse"], dX=dX, dW=dW, weight_layout=layout, ws=ws)
    torch.cuda.synchronize()
    L = got["lse"].double()[:, None]
    h = half(BF16)
    # as check_backward: of q relatively D and the exponent's rounding, |z| <= `most`
    dq = D + 4 * U * (1 + float(L.abs().max()) + most)
    want, slack, ends = torch.zeros_like(x), torch.zeros_like(x), (0, 2 ** 31 // K // step * step, (V - 1) // step * step)
    for n in range(0, V, step):
        w = part(n, step)
        q = (x @ w - L).exp()
        dz = q.clone()
        here = ((t >= n) & (t < n + w.shape[1])).nonzero()[:, 0]
        dz[here, t[here] - n] -= 1
        each = 1.01 * dq * q + (h + 4 * U) * dz.abs() + torch.finfo(BF16).smallest_normal
        want += dz @ w.t().contiguous()
        slack += (each + (V / 32 + 64) * U * dz.abs()) @ w.abs().t().contiguous()
        if n in ends:
            dw = (dW[:, n:n + step] if layout == MATH else dW[n:n + step].t()).double()
            exact = x.t().contiguous() @ dz
            tol = x.abs().t().contiguous() @ (each + (M / 32 + 64) * U * dz.abs()) + (h + U) * exact.abs() + torch.finfo(BF16).smallest_normal
            assert bool(((dw - exact).abs() <= tol).all()), n
    assert bool(((dX.double() - want).abs() <= slack + (h + U) * want.abs() + torch.finfo(BF16).smallest_normal).all())


@pytest.mark.parametrize("layout", [MATH, LINEAR])
@pytest.mark.parametrize("M", [5, 300])
def test_strides_past_32_bits(M, layout):
    """Rows of X, of W and of their gradients far apart: the last begin past 2^32 bytes."""
    announce(f"ce far rows {M} layout {layout}")
    K, V = 64, 264
    X, W, t = make(M, K, V, BF16, seed=50 + M)
    lse = lse_for(X, W)
    Wl = W if layout == MATH else W.t().contiguous()

    def far(m):
        ld = 2 ** 31 // (m.shape[0] - 1) // 8 * 8 + 64
        v = torch.empty(2 ** 31 + 2 ** 20, dtype=BF16, device="cuda").as_strided(tuple(m.shape), (ld, 1), 64)
        v.copy_(m)
        return v
    for Xd, Wd in ((far(X), Wl.cuda()), (X.cuda(), far(Wl))):
        check_forward(X, W, t, forward(X, W, t, layout, Xd=Xd, Wd=Wd), BF16)
        check_backward(X, W, t, lse, backward(X, W, t, lse, layout, Xd=Xd, Wd=Wd))
    dX, dW = far(torch.zeros_like(X)), far(torch.zeros_like(Wl))
    Xd, Wd = X.cuda(), Wl.cuda()
    tp.tp_linear_ce_backward(Xd, Wd, t.cuda(), lse.cuda(), dX=dX, dW=dW, weight_layout=layout,
                             ws=tp.tp_linear_ce_backward_ws(Xd, Wd, weight_layout=layout, dX=dX))
    torch.cuda.synchronize()
    check_backward(X, W, t, lse, dict(dX=dX, dW=dW if layout == MATH else dW.t()))
