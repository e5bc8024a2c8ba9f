"""The AdamW step on the GPU, with fp32 and 8-bit states, against its float64 form.

Tolerances, in u = u(fp32).  m: three roundings of its two terms (4 u of them).  v: four (5 u).  The update: the square
root, the reciprocal and the hyperparameters are each off by a few u (16 u); its sum with the weight by u of both and
half a step of the weight's type.  8-bit states: the code is the nearest, so within 1/2 of where the float64 state
lies between codes, and as far as the state's own error moves that (1e-3 of a code).
"""
import math

import numpy as np
import pytest
import torch

import sharded_gemm_amd as tp
from oracle import linear as L
from oracle import loss as O

from gpu_helpers import GUARD, announce, bits, require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = torch.finfo(F32).eps / 2
TINY = torch.finfo(F32).smallest_normal
FILL = {BF16: 7.0, F32: 7.0, torch.int8: 77, torch.uint8: 77}


def setup_module(_):
    require_gpu()


def f64(t):
    return t.detach().cpu().double().numpy()


class Buf:
    """A GPU copy of a tensor at element `skew` of a larger one, whose rest has to stay."""

    def __init__(self, t, skew=0):
        self.base = torch.full((t.numel() + 2 * GUARD,), FILL[t.dtype], dtype=t.dtype, device="cuda")
        self.at, self.n = GUARD + skew, t.numel()
        self.t = self.base[self.at:self.at + self.n]
        self.t.copy_(t)

    def intact(self):
        v = FILL[self.base.dtype]
        return bool((self.base[:self.at] == v).all()) and bool((self.base[self.at + self.n:] == v).all())


def blocks(n):
    return -(-n // tp.TP_ADAMW_BLOCK)


class Group:
    """Tensors on the host, and guarded on the GPU."""

    def __init__(self, sizes, *, eight, param=F32, grad=F32, seed=0, copy=True, skew=0, zero=False, scale=0.01):
        g = torch.Generator().manual_seed(seed)
        self.eight = eight
        kinds = (lambda k, i: (F32, BF16)[i % 2]) if param == "mixed" else (lambda k, i: param if k == "p" else grad)
        self.host = dict(p=[], g=[], m=[], v=[], ms=[], vs=[])
        for i, n in enumerate(sizes):
            self.host["p"].append((torch.randn(n, generator=g) * 0.5).to(kinds("p", i)))
            self.host["g"].append((torch.randn(n, generator=g) * scale).to(kinds("g", i + 1)))
            if not eight:
                m, r = torch.randn(n, generator=g) * 0.3 * scale, torch.rand(n, generator=g) * scale
                self.host["m"].append(m * (not zero))
                self.host["v"].append(r * r * (not zero))
            else:
                self.host["m"].append(torch.randint(-127, 128, (n,), generator=g).to(torch.int8) * (not zero))
                self.host["v"].append(torch.randint(0, 256, (n,), generator=g).to(torch.uint8) * (not zero))
                self.host["ms"].append(torch.rand(blocks(n), generator=g) * scale * (not zero))
                self.host["vs"].append(torch.rand(blocks(n), generator=g) * scale * (not zero))
        self.dev = {k: [Buf(t, skew) for t in ts] for k, ts in self.host.items()}
        self.copies = [Buf(torch.zeros(n, dtype=BF16), skew) for n in sizes] if copy else None

    def views(self, k):
        return [b.t for b in self.dev[k]]

    def step(self, **kw):
        if self.eight:
            kw.update(m_scale=self.views("ms"), v_scale=self.views("vs"))
        return tp.tp_adamw_step(self.views("p"), self.views("g"), self.views("m"), self.views("v"),
                                copies=[b.t for b in self.copies] if self.copies else None, **kw)

    def intact(self):
        return all(b.intact() for bs in list(self.dev.values()) + [self.copies or []] for b in bs)

    def state(self, where, i):
        """(m, v) of tensor i in float64."""
        if not self.eight:
            return f64(where["m"][i]), f64(where["v"][i])
        m = O.values(f64(where["m"][i]), f64(where["ms"][i]), 127.0)
        return m, O.values(f64(where["v"][i]), f64(where["vs"][i]), 255.0) ** 2

    def check(self, factor=1.0, step=1, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, decays=None):
        torch.cuda.synchronize()
        assert self.intact()
        for i in range(len(self.host["p"])):
            decay = decays[i] if decays else 0.0
            m0, v0 = self.state(self.host, i)
            p0, g = f64(self.host["p"][i]), f64(self.host["g"][i]) * factor
            p, m, v = O.adamw(p0, g, m0, v0, step=step, lr=lr, beta1=beta1, beta2=beta2, eps=eps, decay=decay)
            tol_m = 6 * U * (np.abs(beta1 * m0) + np.abs((1 - beta1) * g)) + TINY
            tol_v = 12 * U * v + TINY
            got = {k: [b.t for b in bs] for k, bs in self.dev.items()}
            gp = got["p"][i]
            half = torch.finfo(gp.dtype).eps / 2
            r = np.sqrt(v / (1 - beta2 ** step))
            big = lr / (1 - beta1 ** step) * (np.abs(m) + np.abs(beta1 * m0) + np.abs((1 - beta1) * g)) / (r + eps)
            tol = (half + 2 * U) * np.abs(p) + 2 * U * np.abs(p0) + 32 * U * (big + lr * decay * np.abs(p0)) + TINY
            assert (np.abs(f64(gp) - p) <= tol).all()
            if self.copies:
                h = torch.finfo(BF16).eps / 2
                assert (np.abs(f64(self.copies[i].t) - p) <= tol + h * np.abs(p) * (1 + h)).all()
            if not self.eight:
                assert (np.abs(f64(got["m"][i]) - m) <= tol_m).all() and (np.abs(f64(got["v"][i]) - v) <= tol_v).all()
                continue
            for name, x, top in (("m", m, 127.0), ("v", np.sqrt(v), 255.0)):
                lies, scale = O.codes(x, top)
                q, s = f64(got[name][i]), f64(got[name + "s"][i])
                # v is an fp32 value: below the smallest normal number (TINY) it may be zero, so its root is off by
                # up to sqrt(TINY) = 1.1e-19, and where it is under that nothing is said of the code.  (m likewise,
                # from 2^-100 on.)
                least = math.sqrt(TINY) if name == "v" else 2.0 ** -99
                assert (np.abs(s - scale) <= 16 * U * scale + least).all()
                near = np.abs(q - lies) <= 0.5 + 1e-3
                near |= np.repeat(scale, O.BLOCK)[:len(q)] < least * 1e6
                if name == "v":      # a second moment that is there stays there
                    near |= (q == 1) & (lies > 0) & (lies < 0.5)
                    assert (q[x > least] > 0).all() and (q[x == 0] == 0).all()
                assert near.all(), np.abs(q - lies).max()


SIZES = [[1], [0, 1, 0], [255], [256], [257], [4096], [4095, 4097, 1, 15, 16, 17], [100, 1 << 18, 3, 12345], [7] * 39, [9] * 40,
         [300] * 41, [1000 + i for i in range(100)]]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_step(sizes, kind, eight):
    announce(f"adamw {len(sizes)} tensors {kind} eight {eight}")
    kw = dict(param=F32, grad=F32) if kind == "f32" else dict(param=BF16, grad=BF16) if kind == "bf16" else dict(param="mixed")
    g = Group(sizes, eight=eight, seed=len(sizes), **kw)
    decays = [0.1 * (i % 3) for i in range(len(sizes))]
    g.step(step=3, lr=1e-2, weight_decay=decays)
    g.check(step=3, lr=1e-2, decays=decays)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("skew", [1, 2, 3, 5])
def test_any_alignment(skew, eight):
    announce(f"adamw skew {skew} eight {eight}")
    for kind in (F32, BF16):
        g = Group([4096 * 2 + 5, 300], eight=eight, param=kind, grad=kind, skew=skew, seed=skew)
        g.step(step=1, lr=1e-3)
        g.check()


@pytest.mark.parametrize("eight", [False, True])
def test_first_steps_from_zero_states(eight):
    """Step by step from zeros, each against float64 from where the last one left the states."""
    g = Group([5000, 77], eight=eight, zero=True, seed=1)
    for t in range(1, 6):
        g.step(step=t, lr=1e-2, weight_decay=0.01)
        g.check(step=t, lr=1e-2, decays=[0.01, 0.01])
        g.host = {k: [b.t.cpu() for b in bs] for k, bs in g.dev.items()}


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("hyper", [dict(beta1=0.0, beta2=0.0), dict(beta1=0.99, beta2=0.9999), dict(eps=1e-3), dict(lr=0.0), dict(lr=1.0)])
def test_hyperparameters(hyper, eight):
    g = Group([3000], eight=eight, seed=2)
    kw = dict(lr=1e-3) | hyper
    g.step(step=1000, **kw)
    g.check(step=1000, **kw)


@pytest.mark.parametrize("eight", [False, True])
def test_clipping(eight):
    """The norm's factor in the same pass, as clipping and then stepping."""
    for limit, ranks in ((0.05, 1), (1e9, 1), (0.05, 4)):
        g = Group([3000, 5, 70_000], eight=eight, seed=3)
        parts = tp.tp_grad_parts(ranks)
        for r in range(ranks):
            tp.tp_grad_sumsq(g.views("g") if r == 0 else [torch.ones(10 * r, device="cuda")], parts[r * tp.TP_GRAD_PARTS:(r + 1) * tp.TP_GRAD_PARTS])
        norm = torch.empty(1, device="cuda")
        g.step(step=2, lr=1e-3, parts=parts, max_norm=limit, clip_eps=1e-6, norm_out=norm, ranks=ranks)
        want, _ = L.clip([f64(x) for x in g.host["g"]] + [np.ones(10 * r) for r in range(1, ranks)], limit, 1e-6)
        assert abs(float(norm) - want) <= 2 * U * want
        g.check(factor=float(np.float32(min(1.0, limit / (want + 1e-6)))), step=2)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_not_finite(bad, eight):
    g = Group([1000, 700], eight=eight, seed=4)
    g.dev["g"][0].t[300] = bad
    before = {k: [bits(b.t) if b.t.dtype in (F32, BF16) else b.t.cpu().numpy() for b in bs] for k, bs in g.dev.items()}
    parts, norm = tp.tp_grad_parts(), torch.zeros(1, device="cuda")
    tp.tp_grad_sumsq(g.views("g"), parts)
    g.step(step=1, lr=1e-3, parts=parts, max_norm=1.0, norm_out=norm, skip_nonfinite=True)
    torch.cuda.synchronize()
    assert not math.isfinite(float(norm)) and g.intact()
    for k, bs in g.dev.items():      # nothing else has changed
        for b, w in zip(bs, before[k]):
            assert np.array_equal(bits(b.t) if b.t.dtype in (F32, BF16) else b.t.cpu().numpy(), w)
    # Not skipped and not clipped: the element (with 8-bit states its block) is spoilt, nothing else.
    g.step(step=1, lr=1e-3)
    torch.cuda.synchronize()
    p = g.dev["p"][0].t
    assert bool(torch.isnan(p[300])) and int(torch.isfinite(p).sum()) == 999 and bool(torch.isfinite(g.dev["p"][1].t).all())
    if eight:
        m, v = torch.empty(1000, device="cuda"), torch.empty(1000, device="cuda")
        tp.tp_adamw_unpack([g.dev["m"][0].t], [g.dev["v"][0].t], [m], [v], m_scale=[g.dev["ms"][0].t], v_scale=[g.dev["vs"][0].t])
        lost = torch.zeros(1000, dtype=torch.bool)
        lost[256:512] = True
        assert torch.equal(~torch.isfinite(m).cpu(), lost) and torch.equal(~torch.isfinite(v).cpu(), lost)


def test_small_and_large_values():
    """Gradients from 1e-18 to 1e18 of a block's largest: fp32 states keep them, 8-bit ones keep every v above zero."""
    for eight in (False, True):
        g = Group([2048], eight=eight, zero=True)
        e = torch.linspace(-18, 0, 2048)
        for top in (1e-10, 1.0, 1e15):
            g.dev["g"][0].t.copy_(torch.pow(10.0, e) * top)
            g.host["g"][0] = g.dev["g"][0].t.cpu()
            for k in ("m", "v", "ms", "vs"):
                for b, h in zip(g.dev[k], g.host[k]):
                    b.t.zero_()
            g.dev["p"][0].t.copy_(g.host["p"][0])
            g.step(step=1, lr=1e-3)
            g.check(step=1)
    z = Group([600], eight=True, zero=True)
    z.dev["g"][0].t.zero_()
    z.step(step=1, lr=1e-3)
    torch.cuda.synchronize()
    assert all(bool((z.dev[k][0].t == 0).all()) for k in ("m", "v", "ms", "vs")) and torch.equal(z.dev["p"][0].t.cpu(), z.host["p"][0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[1], [255, 257, 0, 4096 * 3 + 7], [50] * 45])
def test_unpack(sizes, dtype):
    g = Group(sizes, eight=True, seed=6, skew=1)
    m, v = ([Buf(torch.zeros(n, dtype=dtype), 1) for n in sizes] for _ in "mv")
    tp.tp_adamw_unpack(g.views("m"), g.views("v"), [b.t for b in m], [b.t for b in v], m_scale=g.views("ms"), v_scale=g.views("vs"))
    torch.cuda.synchronize()
    half = torch.finfo(dtype).eps / 2
    # q / 127: two roundings (the constant's and the product's), its square twice those and one, the scale's product
    # one: 6 u for m and for sqrt(v), whose square is off by twice that and one more.
    for i in range(len(sizes)):
        for got, want, steps in zip((m[i], v[i]), g.state(g.host, i), (6, 13)):
            assert got.intact() and (np.abs(f64(got.t) - want) <= (half + (steps + 1) * U) * np.abs(want) + TINY).all()


def test_no_tensors():
    tp.tp_adamw_step([], [], [], [], step=1, lr=1e-3)
    parts, norm = tp.tp_grad_parts(), torch.empty(1, device="cuda")
    tp.tp_grad_sumsq([torch.full((4,), 3.0, device="cuda")], parts)
    tp.tp_adamw_step([], [], [], [], step=1, lr=1e-3, parts=parts, max_norm=1.0, norm_out=norm)
    assert float(norm) == 6.0


@pytest.mark.parametrize("eight", [False, True])
def test_device_step_and_rate_captured(eight):
    """A captured step follows the count and the rate on the device, and gives the eager bits."""
    announce(f"adamw captured, eight {eight}")
    a, b = Group([9000, 31], eight=eight, seed=7), Group([9000, 31], eight=eight, seed=7)
    count, rate = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    prepared = a.step(step=count, lr=rate, prepare=True)
    with torch.cuda.graph(graph):
        count.add_(1)
        prepared(torch.cuda.current_stream())
    for t in range(1, 4):
        rate.fill_(1e-2 / t)
        graph.replay()
        torch.cuda.synchronize()
        b.step(step=torch.tensor([t], device="cuda"), lr=torch.tensor([1e-2 / t], device="cuda"))
        torch.cuda.synchronize()
        assert int(count) == t
        for k in a.dev:
            for x, y in zip(a.dev[k], b.dev[k]):
                assert np.array_equal(x.t.cpu().view(torch.uint8).numpy(), y.t.cpu().view(torch.uint8).numpy())
    # The host's count gives the same step to the correction's rounding.
    c, d = Group([5000], eight=eight, seed=8), Group([5000], eight=eight, seed=8)
    c.step(step=torch.tensor([12], device="cuda"), lr=torch.tensor([0.01], device="cuda"))
    d.step(step=12, lr=0.01)
    c.check(step=12, lr=0.01)
    d.check(step=12, lr=0.01)


def test_on_another_stream():
    g = Group([100_000], eight=True, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g.step(step=1, lr=1e-3, stream=side)
    torch.cuda.synchronize()
    g.check()


def test_two_steps_at_once():
    """Two streams, tensors of their own, one norm and one gradient for both."""
    a, b = Group([300_000, 17], eight=True, seed=10), Group([300_000, 17], eight=True, seed=10)
    parts = tp.tp_grad_parts()
    tp.tp_grad_sumsq(a.views("g"), parts)
    torch.cuda.synchronize()
    sides = torch.cuda.Stream(), torch.cuda.Stream()
    for g, s in zip((a, b), sides):
        g.dev["g"] = a.dev["g"]
        g.step(step=1, lr=1e-3, parts=parts, max_norm=0.5, clip_eps=1e-6, stream=s)
    torch.cuda.synchronize()
    for k in a.dev:
        assert all(torch.equal(x.t, y.t) for x, y in zip(a.dev[k], b.dev[k]))
    norm = math.sqrt(sum(float((f64(x) ** 2).sum()) for x in a.host["g"]))
    a.check(factor=float(np.float32(0.5 / (norm + 1e-6))))


def test_a_tensor_past_32_bits():
    """2^32 elements and some: parts of it against the same parts as tensors of their own, to the bit."""
    n = 2 ** 32 + 777
    announce("adamw 2^32 elements")
    g = torch.Generator("cuda").manual_seed(3)
    p = torch.empty(n, dtype=BF16, device="cuda").normal_(0, 0.5, generator=g)
    d = torch.empty(n, dtype=BF16, device="cuda").normal_(0, 0.01, generator=g)
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(blocks(n), device="cuda"), torch.zeros(blocks(n), device="cuda")
    B = tp.TP_ADAMW_BLOCK
    spans = [(0, 70_000), (2 ** 31 // B * B - 40 * B, 80 * B), (2 ** 32 - 40 * B, 40 * B + 777)]
    s = dict(p=[], g=[], m=[], v=[], ms=[], vs=[])
    for at, k in spans:
        for name, x in (("p", p), ("g", d), ("m", m), ("v", v)):
            s[name].append(x[at:at + k].clone())
        for name, x in (("ms", ms), ("vs", vs)):
            s[name].append(x[at // B:at // B + blocks(k)].clone())
    for t in (1, 2):
        tp.tp_adamw_step([p], [d], [m], [v], m_scale=[ms], v_scale=[vs], step=t, lr=1e-2, weight_decay=0.1)
        tp.tp_adamw_step(s["p"], s["g"], s["m"], s["v"], m_scale=s["ms"], v_scale=s["vs"], step=t, lr=1e-2, weight_decay=0.1)
    del d
    torch.cuda.synchronize()
    mo, vo = torch.empty(n, dtype=BF16, device="cuda"), torch.empty(n, dtype=BF16, device="cuda")
    tp.tp_adamw_unpack([m], [v], [mo], [vo], m_scale=[ms], v_scale=[vs])
    smo, svo = [torch.empty_like(x) for x in s["p"]], [torch.empty_like(x) for x in s["p"]]
    tp.tp_adamw_unpack(s["m"], s["v"], smo, svo, m_scale=s["ms"], v_scale=s["vs"])
    torch.cuda.synchronize()
    for i, (at, k) in enumerate(spans):
        for big, little in ((p, s["p"]), (m, s["m"]), (v, s["v"]), (mo, smo), (vo, svo)):
            assert torch.equal(big[at:at + k], little[i])
        for big, little in ((ms, s["ms"]), (vs, s["vs"])):
            assert torch.equal(big[at // B:at // B + blocks(k)], little[i])
    assert bool((ms > 0).all()) and bool((vs > 0).all())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
def test_many_elements_at_once(kind, eight):
    """Above 2^25 elements in a call chunks are longer; the same bits as from a call for each tensor."""
    announce(f"adamw many elements {kind} eight {eight}")
    types = dict(f32=[(F32, F32)], bf16=[(BF16, BF16)], mixed=[(F32, BF16), (BF16, F32)])[kind]
    sizes = [2 ** 25 + 3, 5, 4096, 4097, 1024, 1023, 3000 + 257, 9_000_001, 0, 4095] + [2000 + i for i in range(60)]
    g = torch.Generator("cuda").manual_seed(5)
    calls = []
    for _ in range(2):
        g.manual_seed(5)
        s = dict(p=[], g=[], m=[], v=[], ms=[], vs=[], c=[])
        for i, n in enumerate(sizes):
            pt, gt = types[i % len(types)]
            s["p"].append(torch.randn(n, generator=g, device="cuda").to(pt))
            s["g"].append((torch.randn(n, generator=g, device="cuda") * 0.01).to(gt))
            s["m"].append(torch.zeros(n, dtype=torch.int8 if eight else F32, device="cuda"))
            s["v"].append(torch.zeros(n, dtype=torch.uint8 if eight else F32, device="cuda"))
            s["ms"].append(torch.zeros(blocks(n), device="cuda"))
            s["vs"].append(torch.zeros(blocks(n), device="cuda"))
            s["c"].append(torch.zeros(n, dtype=BF16, device="cuda"))
        calls.append(s)
    one, each = calls
    parts = tp.tp_grad_parts()
    tp.tp_grad_sumsq(one["g"], parts)
    kw = dict(lr=1e-2, weight_decay=0.1, parts=parts, max_norm=3.0)

    def scales(s, a, b):
        return dict(m_scale=s["ms"][a:b], v_scale=s["vs"][a:b]) if eight else {}
    for t in (1, 2):
        tp.tp_adamw_step(one["p"], one["g"], one["m"], one["v"], copies=one["c"], step=t, **scales(one, 0, len(sizes)), **kw)
        for i in range(1, len(sizes)):
            tp.tp_adamw_step(*(each[k][i:i + 1] for k in ("p", "g", "m", "v")), copies=each["c"][i:i + 1], step=t, **scales(each, i, i + 1), **kw)
        first = dict((k, each[k][0]) for k in each)      # in four parts, each of whole blocks
        cuts = [0, 4096 * 2000, 4096 * 4001 + 256, 2 ** 25 - 4096, sizes[0]]
        for a, b in zip(cuts, cuts[1:]):
            tp.tp_adamw_step(*([first[k][a:b]] for k in ("p", "g", "m", "v")), copies=[first["c"][a:b]], step=t,
                             **(dict(m_scale=[first["ms"][a // 256:a // 256 + blocks(b - a)]], v_scale=[first["vs"][a // 256:a // 256 + blocks(b - a)]]) if eight else {}), **kw)
    torch.cuda.synchronize()
    for k in one:
        assert all(torch.equal(x, y) for x, y in zip(one[k], each[k])), k
    assert all(bool((x != 0).any()) for x in one["m"] if x.numel())


@pytest.mark.parametrize("scale, n", [(s, 1 << 20) for s in (1e-30, 1e-18, 1e-14, 1e-8, 1.0, 1e15)] + [(s, (1 << 25) + 300) for s in (1e-14, 1.0)])
def test_codes_to_the_bit(scale, n):
    """States after a first step against the same operations in fp32 on the CPU, each rounded by itself: nothing may
    differ, near the middle between two codes and at magnitudes where the hardware's root is not taken included."""
    announce(f"adamw codes {scale} {n}")
    g = Group([n], eight=True, zero=True, seed=12, copy=False, scale=scale)
    if scale == 1.0:      # and blocks whose elements differ by up to 1e9
        d = g.host["g"][0]
        d[:n // 2] *= torch.pow(10.0, -9 * torch.rand(n // 2, generator=torch.Generator().manual_seed(1)))
        g.dev["g"][0].t.copy_(d)
    g.step(step=1, lr=1e-3)
    torch.cuda.synchronize()
    # numpy: its roots are rounded to the nearest (torch's, on the CPU, are off by a step now and then).
    f = np.float32
    d = g.host["g"][0].numpy()
    m = d * f(1.0 - 0.9)
    v = (d * f(1.0 - 0.999)) * d
    for name, x, top in (("m", m, f(127)), ("v", np.sqrt(v), f(255))):
        a = np.pad(np.abs(x), (0, -n % 256)).reshape(-1, 256)
        s = a.max(axis=1, keepdims=True)
        assert np.array_equal(g.dev[name + "s"][0].t.cpu().numpy(), s[:, 0])
        with np.errstate(invalid="ignore"):
            q = np.where(s > 0, np.rint(top * np.sqrt(a / s)), f(0)).reshape(-1)[:n]
        q = np.maximum(q, (x > 0).astype(f)) if name == "v" else np.copysign(q, x)
        assert q.dtype == f and np.array_equal(g.dev[name][0].t.cpu().numpy().astype(f), q)


@pytest.mark.parametrize("eight", [False, True])
def test_no_eps(eight):
    g = Group([5000], eight=eight, seed=13)
    g.step(step=100, lr=1e-3, eps=0.0)
    g.check(step=100, eps=0.0)
