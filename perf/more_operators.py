"""What is measured of the end of a training step: the softmax cross entropy of a vocabulary projection (loss and
gradients, the logits never kept, the vocabulary whole or one rank's piece) and the AdamW step over many tensors
(states in 32 or in 8 bits).

``run`` computes one pass, in plain torch operations (``own`` false) or through the library (``own`` true).
Shapes: X[M, K]; W[K, V] ("math") or [V, K] ("linear"); targets[M], some of them ignored.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_TORCH = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}
IGNORE = -100
BLOCK = 256                 # elements that share a scale in 8-bit states
BETA1, BETA2, EPS = 0.9, 0.95, 1e-8
MAX_NORM, CLIP_EPS = 1.0, 1e-6
MOST_FLOPS = 9.0e12         # of a drawn bf16 case (the largest listed one has 9.9e12)
MOST_FLOPS_F32 = 1.0e11
MOST_ELEMENTS = 190_000_000  # of a drawn optimizer case (the largest listed one has 201e6)


def listed():
    return [
        # One token scored against a small model's vocabulary: the smallest call, bound by latency.
        dict(name="ce-score-1", op="ce", dtype=BF16, M=1, K=768, V=32000, layout="linear", pieces=1, piece=0),
        # A few dozen tokens of answers scored at GPT-3 6.7B's width.
        dict(name="ce-score-24", op="ce", dtype=BF16, M=24, K=4096, V=65536, layout="linear", pieces=1, piece=0),
        # The training forward at GPT-2 small's width.
        dict(name="ce-forward", op="ce", dtype=BF16, M=4096, K=768, V=50000, layout="linear", pieces=1, piece=0),
        # One rank of eight at GPT-3 6.7B's width: its piece's statistics, joined with the other ranks'.
        dict(name="ce-forward-shard", op="ce", dtype=BF16, M=8192, K=4096, V=16384, layout="math", pieces=8, piece=3),
        # Nothing a multiple of anything, in fp32.
        dict(name="ce-forward-odd-f32", op="ce", dtype=F32, M=515, K=1021, V=10007, layout="linear", pieces=1, piece=0),
        # The training backward at GPT-3 6.7B's width: both gradients, with a gradient at the log-sum-exp (z-loss).
        dict(name="ce-backward", op="ce_bwd", dtype=BF16, M=8192, K=4096, V=32768, layout="linear", pieces=1, piece=0,
             dlse=True),
        # One rank of two at GPT-3 175B's width.
        dict(name="ce-backward-large", op="ce_bwd", dtype=BF16, M=4096, K=12288, V=32768, layout="linear", pieces=2,
             piece=1, dlse=False),
        # A ragged batch through odd widths, weights in the math layout.
        dict(name="ce-backward-odd", op="ce_bwd", dtype=BF16, M=1021, K=1336, V=5003, layout="math", pieces=1, piece=0,
             dlse=False),
        # One small layer's tensors, clipped and stepped.
        dict(name="adamw-small", op="adamw", bits=32, tensors="layer", param=F32, grad=F32, copy=True, clip=True,
             width=768, inner=768, layers=1),
        # Eight layers of a gated block at GPT-3 6.7B's per-rank widths: fp32 main weights and their bf16 copies.
        dict(name="adamw-large", op="adamw", bits=32, tensors="layer", param=F32, grad=F32, copy=True, clip=True,
             width=4096, inner=2048, layers=8),
        # The same with states in 8 bits.
        dict(name="adamw8-large", op="adamw", bits=8, tensors="layer", param=F32, grad=F32, copy=True, clip=True,
             width=4096, inner=2048, layers=8),
        # Tensors of any size one behind another, bf16 weights and gradients, no clipping.
        dict(name="adamw8-odd", op="adamw", bits=8, tensors="any", param=BF16, grad=BF16, copy=False, clip=False,
             count=37, most=3_000_000, sizes=20240607),
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
    op = rng.choice(("ce", "ce", "ce_bwd", "ce_bwd", "adamw", "adamw"))
    if op == "adamw":
        bits = rng.choice((32, 8))
        param = rng.choice((F32, F32, BF16))
        c = dict(op=op, bits=bits, param=param, grad=rng.choice((F32, BF16)), copy=param == F32 and rng.random() < 0.7,
                 clip=rng.random() < 0.6)
        while True:
            if rng.random() < 0.5:
                c.update(tensors="any", count=rng.randint(1, 60), most=_spread(rng, 16, MOST_ELEMENTS // 60),
                         sizes=rng.randrange(1 << 30))
            else:
                c.update(tensors="layer", width=_spread(rng, 8, 6144), inner=_spread(rng, 8, 6144),
                         layers=rng.randint(1, 8))
            if sum(_tensor_sizes(c)) <= MOST_ELEMENTS:
                return c
            for k in ("count", "most", "sizes", "width", "inner", "layers"):
                c.pop(k, None)
    dtype = BF16 if rng.random() < 0.8 else F32
    while True:
        few = op == "ce" and rng.random() < 0.4
        pieces = rng.choice((1, 1, 2, 8))
        c = dict(op=op, dtype=dtype, M=_spread(rng, 1, 64) if few else _spread(rng, 16, 16384),
                 K=_spread(rng, 64, 12288), V=_spread(rng, 500, 140_000), layout=rng.choice(("math", "linear")),
                 pieces=pieces, piece=rng.randrange(pieces))
        if op == "ce_bwd":
            c.update(dlse=rng.random() < 0.4)
        if work(c)["flops"] <= (MOST_FLOPS if dtype == BF16 else MOST_FLOPS_F32) and c["M"] * c["V"] <= 400_000_000:
            return c


# ---- inputs ------------------------------------------------------------------

def _tensor_sizes(case):
    if case["tensors"] == "layer":   # a gated block: gate, up and down weights, two vectors
        w, f = case["width"], case["inner"]
        return [w * f, w * f, f * w, w, f] * case["layers"]
    r = random.Random(case["sizes"])
    return [int(round(math.exp(r.uniform(0.0, math.log(case["most"]))))) for _ in range(case["count"])]


def _places(case):
    """Where each tensor begins in its kind's buffer: on 64 elements in a layer, else one right behind another."""
    at, places = 0, []
    for n in _tensor_sizes(case):
        places.append((at, n))
        at += n
        if case["tensors"] == "layer":
            at = -(-at // 64) * 64
    return places, at


def _blocks(n):
    return -(-n // BLOCK)


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(_TORCH[dtype])


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ce_inputs(case, seed):
    g = _generator(seed)
    M, K, V, dt = case["M"], case["K"], case["V"], case["dtype"]
    # Logits of standard deviation 2; targets favour small ids, a tenth is ignored.
    s = dict(X=_normal(g, (M, K), 1.0, dt),
             W=_normal(g, (K, V) if case["layout"] == "math" else (V, K), 2.0 / math.sqrt(K), dt))
    u = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
    whole = V * case["pieces"]
    s["targets"] = (u.square() * whole).long().clamp_(max=whole - 1)
    s["targets"][torch.rand(M, generator=g, device="cuda") < 0.1] = IGNORE
    if case["op"] == "ce":
        if case["pieces"] > 1:   # the other ranks' statistics: maximum, sum of exponentials, the target's logit
            P = case["pieces"]
            top = 8.0 + torch.rand((P, M), generator=g, device="cuda")
            total = V * math.exp(-7.0) * (0.5 + torch.rand((P, M), generator=g, device="cuda"))
            holder = torch.div(s["targets"], V, rounding_mode="floor")
            logit = torch.where(holder == torch.arange(P, device="cuda")[:, None],
                                torch.randn((P, M), generator=g, device="cuda") * 2.0,
                                torch.full((P, M), -math.inf, device="cuda"))
            s["stats"] = torch.stack([top, total, logit], 1).contiguous()   # [P, 3, M]
        return s
    # What the forward left, and the gradients that arrive: of the mean loss, and of a penalty on lse.
    w = s["W"].float() if case["layout"] == "math" else s["W"].float().t()
    z = s["X"].float() @ w
    top = z.max(1, keepdim=True).values
    s["lse"] = (z.sub_(top).exp_().sum(1).log() + top[:, 0]) + math.log(case["pieces"])
    count = (s["targets"] != IGNORE).sum().clamp(min=1).float()
    s["dloss"] = torch.full((M,), 1.0, device="cuda") / count
    s["dlse"] = 2e-4 * s["lse"] / count if case["dlse"] else None
    return s


def _adamw_inputs(case, seed):
    g = _generator(seed)
    places, total = _places(case)
    s = dict(param=_normal(g, (total,), 0.02, case["param"]), grad=_normal(g, (total,), 0.01, case["grad"]))
    m = torch.randn(total, generator=g, device="cuda") * 0.003
    r = 0.001 + 0.01 * torch.rand(total, generator=g, device="cuda")    # square roots of second moments
    if case["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:
        for name, x, top, kind in (("m", m, 127.0, torch.int8), ("v", r, 255.0, torch.uint8)):
            s[name], scales = torch.zeros(total, dtype=kind, device="cuda"), []
            for at, n in places:
                code, scale = _codes(x[at:at + n], top)
                s[name][at:at + n] = code.to(kind)
                scales.append(scale)
            s[name + "_scale"] = torch.cat(scales)
    s["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
    # The sum of squares as the gradient norm's pass leaves it: partial sums in 64 bits.
    s["parts"] = torch.zeros(1024, dtype=torch.float64, device="cuda")
    s["parts"][0] = s["grad"].double().square().sum()
    return s


# The step is far enough into training for both corrections to differ from one.
STEP, RATE, DECAY = 20, 3e-4, 0.1


def _decay_of(n_of, i):
    """Weight decay of tensor i: none for a layer's vectors."""
    return 0.0 if n_of == "layer" and i % 5 >= 3 else DECAY


def prepare(case, seed):
    # What a program keeps: inputs, the buffers that the calls write, a workspace.
    if case["op"] == "adamw":
        s = dict(case=case, **_adamw_inputs(case, seed))
        if case["bits"] == 8:
            s["m_value"], s["v_value"] = (torch.zeros(s["m"].numel(), dtype=torch.bfloat16, device="cuda") for _ in "mv")
        if own:
            s["call"] = _own_adamw(s)
        return s
    s = dict(case=case, **_ce_inputs(case, seed))
    M = case["M"]
    if case["op"] == "ce":
        s["loss"], s["new_lse"] = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    else:
        s["dX"], s["dW"] = torch.empty_like(s["X"]), torch.empty_like(s["W"])
    if own:
        s["call"] = _own_ce(s)
    return s


# ---- the library's calls -------------------------------------------------------

def _own_ce(s):
    import sharded_gemm_amd as tp
    c = s["case"]
    layout = tp.TP_WEIGHTS_MATH if c["layout"] == "math" else tp.TP_WEIGHTS_LINEAR
    kw = dict(vocab_begin=c["piece"] * c["V"], ignore_index=IGNORE, weight_layout=layout)
    if c["op"] == "ce_bwd":
        ws = tp.tp_linear_ce_backward_ws(s["X"], s["W"], weight_layout=layout, dX=s["dX"])
        return tp.tp_linear_ce_backward(s["X"], s["W"], s["targets"], s["lse"], dloss=s["dloss"], dlse=s["dlse"],
                                        dX=s["dX"], dW=s["dW"], ws=ws, prepare=True, **kw)
    ws = tp.tp_linear_ce_ws(s["X"], s["W"], weight_layout=layout)
    if c["pieces"] == 1:
        return tp.tp_linear_ce(s["X"], s["W"], s["targets"], loss=s["loss"], lse=s["new_lse"], ws=ws, prepare=True,
                               **kw)
    piece = tp.tp_linear_ce(s["X"], s["W"], s["targets"], stats=s["stats"][c["piece"]], ws=ws, prepare=True, **kw)
    join = tp.tp_ce_join(s["stats"], s["targets"], loss=s["loss"], lse=s["new_lse"], ignore_index=IGNORE, prepare=True)

    def both():
        piece()
        join()
    return both


def _views(s, name):
    return [s[name][at:at + n] for at, n in _places(s["case"])[0]]


def _scale_views(s, name):
    at, views = 0, []
    for n in _tensor_sizes(s["case"]):
        views.append(s[name][at:at + _blocks(n)])
        at += _blocks(n)
    return views


def _own_adamw(s):
    import sharded_gemm_amd as tp
    c = s["case"]
    count = len(_tensor_sizes(c))
    kw = dict(lr=RATE, beta1=BETA1, beta2=BETA2, eps=EPS, step=STEP,
              weight_decay=[_decay_of(c["tensors"], i) for i in range(count)],
              copies=_views(s, "copy") if c["copy"] else None)
    if c["clip"]:
        kw.update(parts=s["parts"], max_norm=MAX_NORM, clip_eps=CLIP_EPS)
    m, v = _views(s, "m"), _views(s, "v")
    if c["bits"] == 32:
        return tp.tp_adamw_step(_views(s, "param"), _views(s, "grad"), m, v, prepare=True, **kw)
    scales = dict(m_scale=_scale_views(s, "m_scale"), v_scale=_scale_views(s, "v_scale"))
    step = tp.tp_adamw_step(_views(s, "param"), _views(s, "grad"), m, v, prepare=True, **scales, **kw)
    values = tp.tp_adamw_unpack(m, v, _views(s, "m_value"), _views(s, "v_value"), prepare=True, **scales)

    def both():
        step()
        values()
    return both


def _outputs(s):
    c = s["case"]
    if c["op"] == "ce":
        r = dict(loss=s["loss"], lse=s["new_lse"])
        if c["pieces"] > 1:
            r["stats"] = s["stats"][c["piece"]]
        return r
    if c["op"] == "ce_bwd":
        return dict(dX=s["dX"], dW=s["dW"])
    r = dict(param=s["param"])
    if c["copy"]:
        r["copy"] = s["copy"]
    if c["bits"] == 32:
        r.update(m=s["m"], v=s["v"])
    else:   # what the codes stand for, and their scales
        r.update(m=s["m_value"], v=s["v_value"], m_scale=s["m_scale"], v_scale=s["v_scale"])
    return r


# ---- the plain form ------------------------------------------------------------

def _as_kv(s, W):
    """The weight as [K, V]."""
    return W if s["case"]["layout"] == "math" else W.t()


def _plain_ce(s):
    c = s["case"]
    M, V, begin = c["M"], c["V"], c["piece"] * c["V"]
    z = s["X"].float() @ _as_kv(s, s["W"].float())
    top = z.max(1).values
    local = s["targets"] - begin
    here = (local >= 0) & (local < V)
    logit = z.gather(1, local.clamp(0, V - 1)[:, None])[:, 0]
    logit = torch.where(here, logit, torch.full_like(logit, -math.inf))
    total = z.sub_(top[:, None]).exp_().sum(1)
    if c["pieces"] > 1:
        s["stats"][c["piece"]] = torch.stack([top, total, logit])
        most = s["stats"][:, 0].max(0).values
        total = (s["stats"][:, 1] * torch.exp(s["stats"][:, 0] - most)).sum(0)
        logit = s["stats"][:, 2].max(0).values
        top = most
    s["new_lse"] = top + torch.log(total)
    s["loss"] = torch.where(s["targets"] == IGNORE, torch.zeros_like(top), s["new_lse"] - logit)
    return _outputs(s)


def _plain_ce_backward(s):
    c = s["case"]
    M, V, begin, dt = c["M"], c["V"], c["piece"] * c["V"], s["X"].dtype
    x, w = s["X"].float(), _as_kv(s, s["W"].float())
    on = (s["targets"] != IGNORE).float()
    g = s["dloss"] * on
    both = g if s["dlse"] is None else g + s["dlse"] * on
    d = (x @ w).sub_(s["lse"][:, None]).exp_().mul_(both[:, None])
    local = s["targets"] - begin
    here = (local >= 0) & (local < V)
    d.scatter_add_(1, local.clamp(0, V - 1)[:, None], -(g * here)[:, None])
    s["dX"] = (d @ w.t()).to(dt)
    s["dW"] = (x.t() @ d if c["layout"] == "math" else d.t() @ x).to(dt)
    return _outputs(s)


def _per_block(x, scale):
    """scale[b] at every element of block b of x."""
    return scale.repeat_interleave(BLOCK)[:x.numel()]


def _codes(x, top):
    """Square-law codes of x, BLOCK elements to a scale: x = scale * sign(q) (q / top)^2, to the nearest q."""
    n = x.numel()
    a = x.new_zeros(_blocks(n) * BLOCK)
    a[:n] = x.abs()
    scale = a.view(-1, BLOCK).max(1).values
    part = x.abs() / _per_block(x, scale.clamp(min=1e-37))
    q = torch.round(top * torch.sqrt(part)).clamp(max=top)
    if top == 255.0:   # a second moment that is there stays there
        q = torch.where((x > 0) & (q < 1), torch.ones_like(q), q)
    return q * torch.sign(x), scale


def _values(q, scale, top):
    q = q.to(scale.dtype)
    return torch.sign(q) * (q / top).square() * _per_block(q, scale)


def _step(param, grad, m, v, factor, decay, real):
    """One tensor's step in `real`: (param, m, v)."""
    g = grad.to(real) * factor
    m = BETA1 * m.to(real) + (1.0 - BETA1) * g
    v = BETA2 * v.to(real) + (1.0 - BETA2) * g * g
    p = param.to(real)
    move = (m / (1.0 - BETA1 ** STEP)) / (torch.sqrt(v / (1.0 - BETA2 ** STEP)) + EPS)
    return p - RATE * (decay * p + move), m, v


def _plain_adamw(s):
    c = s["case"]
    factor = 1.0
    if c["clip"]:
        factor = torch.clamp(MAX_NORM / (torch.sqrt(s["parts"].sum()) + CLIP_EPS), max=1.0).float()
    blocks = 0
    for i, (at, n) in enumerate(_places(c)[0]):
        here = slice(at, at + n)
        decay = _decay_of(c["tensors"], i)
        if c["bits"] == 32:
            p, s["m"][here], s["v"][here] = _step(s["param"][here], s["grad"][here], s["m"][here], s["v"][here],
                                                  factor, decay, torch.float32)
        else:
            span = slice(blocks, blocks + _blocks(n))
            blocks = span.stop
            m = _values(s["m"][here], s["m_scale"][span], 127.0)
            v = _values(s["v"][here], s["v_scale"][span], 255.0).square()
            p, m, v = _step(s["param"][here], s["grad"][here], m, v, factor, decay, torch.float32)
            for name, x, top in (("m", m, 127.0), ("v", torch.sqrt(v), 255.0)):
                code, s[name + "_scale"][span] = _codes(x, top)
                s[name][here] = code.to(s[name].dtype)
                x = _values(code, s[name + "_scale"][span], top)
                s[name + "_value"][here] = (x if name == "m" else x.square()).to(torch.bfloat16)
        s["param"][here] = p.to(s["param"].dtype)
        if c["copy"]:
            s["copy"][here] = p.to(torch.bfloat16)
    return _outputs(s)


def run(state):
    if own:
        state["call"]()
        return _outputs(state)
    op = state["case"]["op"]
    return _plain_ce(state) if op == "ce" else _plain_ce_backward(state) if op == "ce_bwd" else _plain_adamw(state)


# ---- sizes and the 64-bit definition -------------------------------------------

def work(case):
    if case["op"] == "adamw":
        n = sum(_tensor_sizes(case))
        each = 2 * _SIZE[case["param"]] + _SIZE[case["grad"]] + 2 * case["copy"]
        if case["bits"] == 32:
            each += 16
        else:   # codes read and written, and the values that are handed out
            each += 4 + 4
        scales = 16.0 * sum(_blocks(k) for k in _tensor_sizes(case)) if case["bits"] == 8 else 0.0
        return dict(bytes=float(each) * n + scales + 8192 * case["clip"], flops=(16.0 if case["bits"] == 32 else 30.0) * n)
    M, K, V, es = case["M"], case["K"], case["V"], _SIZE[case["dtype"]]
    if case["op"] == "ce":
        rows = 8 + 8 + (12 * case["pieces"] if case["pieces"] > 1 else 0)
        return dict(bytes=float(es * (M * K + V * K) + rows * M), flops=2.0 * M * V * K + 3.0 * M * V)
    # Without the logits kept, the backward cannot do without the product that gave them.
    return dict(bytes=float(2 * es * (M * K + V * K) + (16 + 4 * case["dlse"]) * M), flops=6.0 * M * V * K + 3.0 * M * V)


def _exact_codes(x, top):
    """(what the codes of x stand for, scales), in 64 bits."""
    n = x.numel()
    rows = torch.nn.functional.pad(x, (0, _blocks(n) * BLOCK - n)).view(-1, BLOCK)
    scale = rows.abs().amax(1, keepdim=True)
    ratio = torch.where(scale > 0, rows.abs() / scale, torch.zeros_like(rows))
    q = torch.floor(top * ratio.sqrt() + 0.5)
    if top == 255.0:
        q = torch.maximum(q, (rows > 0).double())
    return (torch.sgn(rows) * scale * (q / top) ** 2).reshape(-1)[:n], scale[:, 0]


def _exact_adamw(case, seed):
    s = _adamw_inputs(case, seed)
    norm = math.sqrt(float(s["parts"].sum()))
    factor = min(1.0, MAX_NORM / (norm + CLIP_EPS)) if case["clip"] else 1.0
    out = {k: s[k].double() for k in ("param", "m", "v")}
    if case["bits"] == 8:   # between tensors: nothing
        out["m"].zero_()
        out["v"].zero_()
    scales, blocks = dict(m=[], v=[]), 0
    for i, (at, n) in enumerate(_places(case)[0]):
        part = slice(at, at + n)
        g = s["grad"][part].double() * factor
        m, v = s["m"][part].double(), s["v"][part].double()
        if case["bits"] == 8:
            of = torch.arange(n, device="cuda") // BLOCK + blocks
            blocks += _blocks(n)
            m = m * m.abs() / 127.0 ** 2 * s["m_scale"].double()[of]
            v = ((v / 255.0) ** 2 * s["v_scale"].double()[of]) ** 2
        m, v = m + (1.0 - BETA1) * (g - m), v + (1.0 - BETA2) * (g ** 2 - v)
        rise = m / (1.0 - BETA1 ** STEP) / ((v / (1.0 - BETA2 ** STEP)) ** 0.5 + EPS)
        old = out["param"][part]
        out["param"][part] = old * (1.0 - RATE * _decay_of(case["tensors"], i)) - RATE * rise
        if case["bits"] == 8:
            m, sm = _exact_codes(m, 127.0)
            r, sr = _exact_codes(v.sqrt(), 255.0)
            v = r ** 2
            scales["m"].append(sm)
            scales["v"].append(sr)
        out["m"][part], out["v"][part] = m, v
    if case["copy"]:   # the gaps between tensors hold zeros there
        out["copy"] = torch.zeros_like(out["param"])
        for at, n in _places(case)[0]:
            out["copy"][at:at + n] = out["param"][at:at + n]
    if case["bits"] == 8:
        out["m_scale"], out["v_scale"] = torch.cat(scales["m"]), torch.cat(scales["v"])
    return out


def exact(case, seed):
    if case["op"] == "adamw":
        return _exact_adamw(case, seed)
    s = _ce_inputs(case, seed)
    M, V, begin = case["M"], case["V"], case["piece"] * case["V"]
    w = s["W"].double() if case["layout"] == "math" else s["W"].double().t()
    z = torch.mm(s["X"].double(), w)
    rows = torch.arange(M, device="cuda")
    keep = s["targets"] != IGNORE
    held = (s["targets"] >= begin) & (s["targets"] < begin + V)
    column = torch.where(held, s["targets"] - begin, torch.zeros_like(s["targets"]))
    if case["op"] == "ce":
        own_lse = torch.logsumexp(z, 1)
        at = torch.where(held, z[rows, column], z.new_tensor(-math.inf))
        r = {}
        lse, logit = own_lse, at
        if case["pieces"] > 1:
            top = z.amax(1)
            r["stats"] = torch.stack([top, torch.exp(own_lse - top), at])
            st = s["stats"].double()
            of = [own_lse if p == case["piece"] else st[p, 0] + torch.log(st[p, 1]) for p in range(case["pieces"])]
            lse = torch.logsumexp(torch.stack(of), 0)
            logit = torch.stack([at if p == case["piece"] else st[p, 2] for p in range(case["pieces"])]).amax(0)
        return dict(loss=torch.where(keep, lse - logit, torch.zeros_like(lse)), lse=lse, **r)
    g = torch.where(keep, s["dloss"].double(), z.new_zeros(()))
    h = torch.where(keep, s["dlse"].double(), z.new_zeros(())) if s["dlse"] is not None else torch.zeros_like(g)
    d = torch.exp(z - s["lse"].double()[:, None]) * (g + h)[:, None]
    d[rows, column] -= torch.where(held, g, torch.zeros_like(g))
    dX = torch.mm(d, w.t())
    dW = torch.mm(s["X"].double().t(), d) if case["layout"] == "math" else torch.mm(d.t(), s["X"].double())
    return dict(dX=dX, dW=dW)
