"""What is measured of the feed-forward operators: the linear layer with bias, activation and residual in its
product, the gated linear block, their backward passes, and the global gradient norm with clipping.

``run`` computes one pass, in plain torch operations (``own`` false) or through the library (``own`` true).
Shapes: X[M, K]; W[K, N] ("math") or [N, K] ("linear"); the gated block's N is its width F.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_TORCH = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}
ACTS = ("none", "gelu_erf", "gelu_tanh", "silu", "relu")
MOST_FLOPS = 1.2e12         # of a drawn bf16 case (the largest listed one has 1.24e12)
MOST_FLOPS_F32 = 1.0e11
MOST_GRADS = 190_000_000    # elements of a drawn clipping case (the largest listed one has 201e6)


def listed():
    return [
        # The down projection of one token: GPT-3 175B's share at TP = 8, weights as a linear layer stores them.
        dict(name="linear-decode-1", op="linear", dtype=BF16, M=1, K=6144, N=12288, layout="linear", act="none",
             bias=True, residual=True, save=False, sliced=False),
        # The smallest call: three tokens through GPT-2 small's per-rank projection.
        dict(name="linear-decode-3-small", op="linear", dtype=BF16, M=3, K=768, N=768, layout="math", act="gelu_erf",
             bias=True, residual=False, save=False, sliced=False),
        # GPT-2 small's column-parallel layer in training: bias and GeLU in the product, the pre-activation kept.
        dict(name="linear-gelu-save", op="linear", dtype=BF16, M=4096, K=768, N=768, layout="math", act="gelu_erf",
             bias=True, residual=False, save=True, sliced=True),
        # Nothing a multiple of anything, in fp32: a ragged batch through an odd layer.
        dict(name="linear-odd-f32", op="linear", dtype=F32, M=515, K=1021, N=1531, layout="linear", act="silu",
             bias=True, residual=True, save=False, sliced=False),
        # Training backward at GPT-3 6.7B's widths (TP = 8): dX, dW and the bias gradient.
        dict(name="linear-backward", op="linear_bwd", dtype=BF16, M=8192, K=2048, N=4096, layout="math",
             act="gelu_erf", bias=True, sliced=False),
        # One token through a gated block at GPT-3 175B's per-rank widths.
        dict(name="gated-decode-1", op="gated", dtype=BF16, M=1, K=12288, N=6144, layout="linear", act="silu",
             save=False, sliced=False),
        # A small decode batch, weights in the math layout, cut in place from the full weight.
        dict(name="gated-decode-12", op="gated", dtype=BF16, M=12, K=4096, N=2048, layout="math", act="gelu_erf",
             save=False, sliced=True),
        # The training forward at GPT-3 175B's per-rank widths, both pre-activations kept.
        dict(name="gated-forward-large", op="gated", dtype=BF16, M=4096, K=12288, N=6144, layout="math", act="silu",
             save=True, sliced=False),
        # The training backward at GPT-3 6.7B's per-rank widths.
        dict(name="gated-backward", op="gated_bwd", dtype=BF16, M=8192, K=4096, N=2048, layout="math", act="silu",
             sliced=False),
        # A ragged batch through odd widths, backward.
        dict(name="gated-backward-odd", op="gated_bwd", dtype=BF16, M=1021, K=1337, N=999, layout="linear",
             act="gelu_tanh", sliced=False),
        # The gradients of one small layer: a few matrices and their vectors.
        dict(name="clip-small", op="clip", grads="layer", dtype=F32, width=768, inner=768, layers=1, scale=0.01),
        # Eight layers of a gated block at GPT-3 6.7B's per-rank widths, fp32 main gradients (805 MB).
        dict(name="clip-large", op="clip", grads="layer", dtype=F32, width=4096, inner=2048, layers=8, scale=0.001),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], about half of them odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.35 and v >= 64:
        v = v // 64 * 64
    elif kind < 0.5 and v >= 8:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd", "clip"))
    if op == "clip":
        if rng.random() < 0.5:
            return dict(op=op, grads="any", dtype=rng.choice((F32, BF16, "mixed")), count=rng.randint(1, 60),
                        most=_spread(rng, 16, MOST_GRADS // 60), sizes=rng.randrange(1 << 30),
                        scale=rng.choice((1e-6, 0.001, 0.1)))
        while True:
            c = dict(op=op, grads="layer", dtype=rng.choice((F32, BF16)), width=_spread(rng, 8, 6144),
                     inner=_spread(rng, 8, 6144), layers=rng.randint(1, 8), scale=rng.choice((1e-6, 0.001, 0.1)))
            if sum(_grad_sizes(c)) <= MOST_GRADS:
                return c
    dtype = BF16 if rng.random() < 0.75 else F32
    while True:
        decode = not op.endswith("_bwd") and rng.random() < 0.45
        c = dict(op=op, dtype=dtype, M=_spread(rng, 1, 64) if decode else _spread(rng, 1, 8192),
                 K=_spread(rng, 16, 12288), N=_spread(rng, 16, 12288), layout=rng.choice(("math", "linear")),
                 act=rng.choice(ACTS), sliced=rng.random() < 0.3)
        if op == "linear":
            c.update(bias=rng.random() < 0.6, residual=rng.random() < 0.5, save=rng.random() < 0.4)
        elif op == "linear_bwd":
            c.update(bias=rng.random() < 0.6)
        elif op == "gated":
            c.update(save=rng.random() < 0.5)
        if work(c)["flops"] <= (MOST_FLOPS if dtype == BF16 else MOST_FLOPS_F32):
            return c


# ---- inputs ------------------------------------------------------------------

def _grad_sizes(case):
    if case["grads"] == "layer":   # a gated block: gate, up and down weights, two vectors
        w, f = case["width"], case["inner"]
        return [w * f, w * f, f * w, w, f] * case["layers"]
    r = random.Random(case["sizes"])
    return [int(round(math.exp(r.uniform(0.0, math.log(case["most"]))))) for _ in range(case["count"])]


def _grad_dtypes(case):
    n = len(_grad_sizes(case))
    if case["dtype"] != "mixed":
        return [case["dtype"]] * n
    r = random.Random(case["sizes"] + 1)
    return [r.choice((F32, BF16)) for _ in range(n)]


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(_TORCH[dtype])

    if case["op"] == "clip":
        return dict(grads=[normal((n,), case["scale"], d) for n, d in zip(_grad_sizes(case), _grad_dtypes(case))])
    M, K, N, dt = case["M"], case["K"], case["N"], case["dtype"]

    def weight():
        shape = (K, N) if case["layout"] == "math" else (N, K)
        if not case["sliced"]:
            return normal(shape, 0.02, dt)
        # one rank's columns of a full weight, read in place (the column-parallel shard's row stride)
        return normal((shape[0], 2 * shape[1]), 0.02, dt)[:, shape[1]:]

    s = dict(X=normal((M, K), 1.0, dt))
    if case["op"].startswith("linear"):
        s["W"] = weight()
    else:
        s["Wg"], s["Wu"] = weight(), weight()
    std = 0.02 * math.sqrt(K)
    if case["op"] == "linear":
        s["bias"] = normal((N,), 0.1, F32) if case["bias"] else None
        s["residual"] = normal((M, N), 1.0, dt) if case["residual"] else None
    elif case["op"] == "linear_bwd":
        s["dOut"] = normal((M, N), 0.01, dt)
        s["pre"] = normal((M, N), std, dt) if case["act"] != "none" else None
    elif case["op"] == "gated_bwd":
        s["dOut"] = normal((M, N), 0.01, dt)
        s["gate"], s["up"] = normal((M, N), std, dt), normal((M, N), std, dt)
    return s


def prepare(case, seed):
    s = dict(case=case, **_inputs(case, seed))
    # What a program keeps: the buffers that the calls write, and a workspace.
    if case["op"] == "clip":
        s["outs"] = [torch.empty_like(t) for t in s["grads"]]
        s["norm"] = torch.empty(1, device="cuda")
    else:
        M, N = case["M"], case["N"]
        dt = _TORCH[case["dtype"]]
        if case["op"] in ("linear", "gated"):
            s["out"] = torch.empty((M, N), dtype=dt, device="cuda")
            for name in ("pre_out",) if case["op"] == "linear" else ("gate_out", "up_out"):
                s[name] = torch.empty((M, N), dtype=dt, device="cuda") if case["save"] else None
        else:
            s["dX"] = torch.empty_like(s["X"])
            for name in ("W", "Wg", "Wu"):
                if name in s:
                    s["d" + name] = torch.empty(s[name].shape, dtype=dt, device="cuda")
            if case["op"] == "linear_bwd":
                s["dbias"] = torch.empty(N, device="cuda") if case["bias"] else None
    if own:
        s["call"] = _own_call(s)   # the library's prepared call: arguments marshalled once, run many times
    return s


# ---- the library's calls -------------------------------------------------------

def _own_call(s):
    import sharded_gemm_amd as tp
    c = s["case"]
    if c["op"] == "clip":
        parts = tp.tp_grad_parts()
        sumsq = tp.tp_grad_sumsq(s["grads"], parts, prepare=True)
        clip = tp.tp_grad_clip(s["grads"], s["outs"], parts, max_norm=1.0, eps=1e-6, norm_out=s["norm"], prepare=True)

        def both():
            sumsq()
            clip()
        return both
    act = dict(none=tp.TP_ACT_NONE, gelu_erf=tp.TP_ACT_GELU_ERF, gelu_tanh=tp.TP_ACT_GELU_TANH, silu=tp.TP_ACT_SILU,
               relu=tp.TP_ACT_RELU)[c["act"]]
    kw = dict(act=act, weight_layout=tp.TP_WEIGHTS_MATH if c["layout"] == "math" else tp.TP_WEIGHTS_LINEAR,
              prepare=True)
    if c["op"] == "linear":
        return tp.tp_linear(s["X"], s["W"], s["out"], bias=s["bias"], residual=s["residual"], pre_out=s["pre_out"],
                            **kw)
    if c["op"] == "gated":
        return tp.tp_gated_linear(s["X"], s["Wg"], s["Wu"], s["out"], gate_out=s["gate_out"], up_out=s["up_out"],
                                  **kw)
    if c["op"] == "linear_bwd":
        ws = tp.tp_linear_backward_ws(s["X"], s["W"], s["dOut"], act=act, weight_layout=kw["weight_layout"],
                                      dbias=s["dbias"])
        return tp.tp_linear_backward(s["X"], s["W"], s["dOut"], pre=s["pre"], dX=s["dX"], dW=s["dW"],
                                     dbias=s["dbias"], ws=ws, **kw)
    ws = tp.tp_gated_linear_backward_ws(s["X"], s["dOut"])
    return tp.tp_gated_linear_backward(s["X"], s["Wg"], s["Wu"], s["gate"], s["up"], s["dOut"], dX=s["dX"],
                                       dW_gate=s["dWg"], dW_up=s["dWu"], ws=ws, **kw)


def _outputs(s):
    c = s["case"]
    names = dict(linear=("out", "pre_out"), gated=("out", "gate_out", "up_out"), linear_bwd=("dX", "dW", "dbias"),
                 gated_bwd=("dX", "dWg", "dWu"), clip=("norm", "outs"))[c["op"]]
    return {n: s[n] for n in names if s[n] is not None}


# ---- the plain form ------------------------------------------------------------

def _act(name, x):
    if name == "none":
        return x
    if name == "gelu_erf":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    return torch.where(x > 0, x, torch.zeros_like(x))


def _act_grad(name, x):
    if name == "none":
        return torch.ones_like(x)
    if name == "gelu_erf":
        return (0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
                + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi)))
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * x * x)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return p * (1.0 + x * (1.0 - p))
    return torch.where(x > 0, torch.ones_like(x), torch.zeros_like(x))


def _plain(s):
    c = s["case"]
    if c["op"] == "clip":
        # The sum runs over hundreds of millions of squares: in 64 bits.
        norm = torch.sqrt(torch.stack([t.double().square().sum() for t in s["grads"]]).sum())
        scale = torch.clamp(1.0 / (norm + 1e-6), max=1.0).float()
        return dict(norm=norm.float().reshape(1), outs=[(t.float() * scale).to(t.dtype) for t in s["grads"]])
    dt = s["X"].dtype
    x = s["X"].float()

    def mat(w):   # as [K, N]
        w = w.float()
        return w if c["layout"] == "math" else w.t()

    def lay(dw):
        return (dw if c["layout"] == "math" else dw.t().contiguous()).to(dt)

    if c["op"] == "linear":
        pre = x @ mat(s["W"])
        if s["bias"] is not None:
            pre = pre + s["bias"]
        out = _act(c["act"], pre)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        r = dict(out=out.to(dt))
        if c["save"]:
            r["pre_out"] = pre.to(dt)
        return r
    if c["op"] == "gated":
        gate, up = x @ mat(s["Wg"]), x @ mat(s["Wu"])
        r = dict(out=(_act(c["act"], gate) * up).to(dt))
        if c["save"]:
            r.update(gate_out=gate.to(dt), up_out=up.to(dt))
        return r
    d = s["dOut"].float()
    if c["op"] == "linear_bwd":
        if s["pre"] is not None:
            d = d * _act_grad(c["act"], s["pre"].float())
        r = dict(dX=(d @ mat(s["W"]).t()).to(dt), dW=lay(x.t() @ d))
        if c["bias"]:
            r["dbias"] = d.sum(0)
        return r
    gate, up = s["gate"].float(), s["up"].float()
    dg, du = d * up * _act_grad(c["act"], gate), d * _act(c["act"], gate)
    return dict(dX=(dg @ mat(s["Wg"]).t() + du @ mat(s["Wu"]).t()).to(dt), dWg=lay(x.t() @ dg), dWu=lay(x.t() @ du))


def run(state):
    if own:
        state["call"]()
        return _outputs(state)
    return _plain(state)


# ---- sizes and the 64-bit definition -------------------------------------------

def work(case):
    if case["op"] == "clip":
        sizes = _grad_sizes(case)
        total = sum(n * _SIZE[d] for n, d in zip(sizes, _grad_dtypes(case)))
        return dict(bytes=2.0 * total + 4, flops=3.0 * sum(sizes))
    M, K, N, es = case["M"], case["K"], case["N"], _SIZE[case["dtype"]]
    if case["op"] == "linear":
        cells = M * K + K * N + M * N * (1 + case["residual"] + case["save"])
        return dict(bytes=float(es * cells + 4 * N * case["bias"]), flops=2.0 * M * K * N)
    if case["op"] == "gated":
        return dict(bytes=float(es * (M * K + 2 * K * N + M * N * (1 + 2 * case["save"]))), flops=4.0 * M * K * N)
    if case["op"] == "linear_bwd":
        cells = 2 * M * K + 2 * K * N + M * N * (1 + (case["act"] != "none"))
        return dict(bytes=float(es * cells + 4 * N * case["bias"]), flops=4.0 * M * K * N)
    return dict(bytes=float(es * (2 * M * K + 4 * K * N + 3 * M * N)), flops=8.0 * M * K * N)


def _phi(z):
    """The standard normal distribution function in 64 bits."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_act(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "gelu_erf":
        density = torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
        return z * _phi(z), _phi(z) + z * density
    if name == "gelu_tanh":   # z / (1 + e^{-2 v}), v = sqrt(2 / pi) (z + 0.044715 z^3)
        root = math.sqrt(2 / math.pi)
        p = torch.special.expit(2 * root * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * 2 * root * (1 + 0.134145 * z.square())
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * (1 - p)
    on = (z > 0).double()
    return z * on, on


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "clip":
        total = sum(float((t.double() ** 2).sum()) for t in s["grads"])
        norm = math.sqrt(total)
        factor = min(1.0, 1.0 / (norm + 1e-6))
        return dict(norm=torch.tensor([norm], dtype=torch.float64, device="cuda"),
                    outs=[t.double() * factor for t in s["grads"]])
    linear_layout = case["layout"] == "linear"
    w = {k: s[k].double().t() if linear_layout else s[k].double() for k in ("W", "Wg", "Wu") if k in s}
    x = s["X"].double()

    def of_weight(a, b):   # a^T b as the weight lies
        return torch.mm(b.t(), a) if linear_layout else torch.mm(a.t(), b)

    if case["op"] == "linear":
        z = torch.mm(x, w["W"])
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(case["act"], z)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return dict(out=y, pre_out=z) if case["save"] else dict(out=y)
    if case["op"] == "gated":
        g, u = torch.mm(x, w["Wg"]), torch.mm(x, w["Wu"])
        y = _exact_act(case["act"], g)[0] * u
        return dict(out=y, gate_out=g, up_out=u) if case["save"] else dict(out=y)
    d = s["dOut"].double()
    if case["op"] == "linear_bwd":
        if s["pre"] is not None:
            d = d * _exact_act(case["act"], s["pre"].double())[1]
        r = dict(dX=torch.mm(d, w["W"].t()), dW=of_weight(x, d))
        if case["bias"]:
            r["dbias"] = d.sum(dim=0)
        return r
    a, da = _exact_act(case["act"], s["gate"].double())
    dg, du = d * s["up"].double() * da, d * a
    return dict(dX=torch.mm(dg, w["Wg"].t()) + torch.mm(du, w["Wu"].t()), dWg=of_weight(x, dg), dWu=of_weight(x, du))
