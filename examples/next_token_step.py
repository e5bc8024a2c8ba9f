"""A language model's training step around the gated feed-forward block: loss, gradients, norm and update.

    python examples/next_token_step.py           # needs an MI355X and the built library

    x = E[tokens];  h = block(x)                 GatedFFN of gated_ffn_step.py
    loss = mean of -ln softmax(h W_head^T)[next] tp_linear_ce (the logits are never kept)
    dh, dW_head                                  tp_linear_ce_backward
    block's gradients                            tp_linear_backward, tp_gated_linear_backward
    norm, clipping and AdamW                     tp_grad_sumsq, tp_adamw_step (one pass, fp32 main weights)

The head may be cut into ``pieces`` of the vocabulary, as tensor-parallel ranks hold it: each piece leaves its
statistics, ``tp_ce_join`` makes the loss of them, and the pieces' input gradients are partial sums
(``tp_partial_reduce``).  The optimizer's states are fp32 or, with ``eight``, 8-bit codes.
"""
from __future__ import annotations

import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for path in (HERE, os.path.dirname(HERE)):
    if path not in sys.path:
        sys.path.insert(0, path)

import sharded_gemm_amd as tp  # noqa: E402
from gated_ffn_step import GatedFFN  # noqa: E402

BF16 = torch.bfloat16
LINEAR = tp.TP_WEIGHTS_LINEAR


class NextToken:
    """Embedding, block, head, their gradients and the optimizer's state, for one number of tokens."""

    def __init__(self, tokens, width, inner, vocab, *, pieces=1, eight=False, max_norm=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7)
        if vocab % pieces:
            raise ValueError("the pieces divide the vocabulary")
        self.tokens, self.pieces, self.part, self.max_norm = tokens, pieces, vocab // pieces, max_norm
        self.embedding = torch.randn((vocab, width), generator=g, device="cuda").to(BF16)     # (kept as it is)
        self.block = GatedFFN(tokens, width, inner, seed)
        self.main = dict(self.block.main, head=torch.randn((vocab, width), generator=g, device="cuda") * width ** -0.5)
        self.grads = dict(self.block.grads, head=torch.zeros((vocab, width), device="cuda"))
        self.copies = dict(self.block.w, head=self.main["head"].to(BF16))    # what the products read
        self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.stats = torch.empty((pieces, 3, tokens), device="cuda")
        self.d_out = torch.empty((tokens, width), dtype=BF16, device="cuda")
        self.d_parts = [torch.empty((tokens, width), device="cuda") for _ in range(pieces)] if pieces > 1 else None
        head, dx = self.head(0), self.d_parts[0] if pieces > 1 else self.d_out
        self.ws = tp.tp_linear_ce_ws(self.block.out, head, weight_layout=LINEAR)
        self.bws = tp.tp_linear_ce_backward_ws(self.block.out, head, weight_layout=LINEAR, dX=dx)
        self.parts, self.norm = tp.tp_grad_parts(), torch.empty(1, device="cuda")
        self.count = torch.zeros(1, dtype=torch.int64, device="cuda")        # steps taken, on the device
        blocks = [-(-v.numel() // tp.TP_ADAMW_BLOCK) for v in self.main.values()]
        if eight:
            self.m, self.v = ([torch.zeros(v.shape, dtype=t, device="cuda") for v in self.main.values()]
                              for t in (torch.int8, torch.uint8))
            self.scales = dict(m_scale=[torch.zeros(b, device="cuda") for b in blocks],
                               v_scale=[torch.zeros(b, device="cuda") for b in blocks])
        else:
            self.m, self.v = ([torch.zeros_like(v) for v in self.main.values()] for _ in "mv")
            self.scales = {}

    def head(self, i, of=None):
        """Piece i of the head's weights (or of their gradient)."""
        return (self.copies if of is None else of)["head"][i * self.part:(i + 1) * self.part]

    def forward(self, ids, targets):
        """Per-token losses; targets of -100 count for nothing."""
        self.x = self.embedding[ids]
        h = self.block.forward(self.x)
        for i in range(self.pieces):
            out = dict(loss=self.loss, lse=self.lse) if self.pieces == 1 else dict(stats=self.stats[i])
            tp.tp_linear_ce(h, self.head(i), targets, vocab_begin=i * self.part, weight_layout=LINEAR, ws=self.ws, **out)
        if self.pieces > 1:
            tp.tp_ce_join(self.stats, targets, loss=self.loss, lse=self.lse)
        return self.loss

    def backward(self, targets):
        """Gradients of the mean loss over the tokens that count."""
        scale = 1.0 / (targets != -100).sum().clamp(min=1).float()
        for i in range(self.pieces):
            dx = self.d_parts[i] if self.pieces > 1 else self.d_out
            tp.tp_linear_ce_backward(self.block.out, self.head(i), targets, self.lse, dloss=scale, dX=dx,
                                     dW=self.head(i, self.grads), vocab_begin=i * self.part, weight_layout=LINEAR, ws=self.bws)
        if self.pieces > 1:
            tp.tp_partial_reduce(self.d_parts, [self.d_parts[0]])
            self.d_out.copy_(self.d_parts[0])
        self.block.backward(self.x, self.d_out)

    def step(self, rate, decay=0.01):
        """One clipped AdamW step of every weight, and the products' copies of them; with gradients that are not finite, none."""
        self.count.add_(1)
        grads = [self.grads[k] for k in self.main]
        tp.tp_grad_sumsq(grads, self.parts)
        tp.tp_adamw_step(list(self.main.values()), grads, self.m, self.v, step=self.count, lr=rate,
                         weight_decay=[0.0 if k == "bias" else decay for k in self.main],
                         copies=[self.copies.get(k) for k in self.main], parts=self.parts, max_norm=self.max_norm,
                         norm_out=self.norm, skip_nonfinite=True, **self.scales)
        self.count.sub_(torch.isfinite(self.norm).logical_not().long())      # the states did not take that one
        return self.norm


def data(tokens, vocab, seed=0):
    """Tokens whose next one is a fixed function of them, an eighth of them ignored."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    targets = (ids * 5 + 1) % vocab
    targets[torch.rand(tokens, generator=g, device="cuda") < 0.125] = -100
    return ids, targets


def train(tokens=512, width=128, inner=192, vocab=1000, steps=40, rate=1e-2, **kw):
    """The mean losses and norms of the steps, and the model."""
    model = NextToken(tokens, width, inner, vocab, **kw)
    ids, targets = data(tokens, vocab)
    losses, norms = [], []
    for _ in range(steps):
        loss = model.forward(ids, targets)
        losses.append(loss.sum() / (targets != -100).sum())
        model.backward(targets)
        norms.append(model.step(rate).clone())
    return [float(v) for v in losses], [float(v) for v in norms], model


def score(model, h, targets):
    """The losses of rows of h one token at a time, through a prepared call."""
    row, target, loss = h[:1].clone(), targets[:1].clone(), torch.empty(1, device="cuda")
    ws = tp.tp_linear_ce_ws(row, model.copies["head"], weight_layout=LINEAR)
    call = tp.tp_linear_ce(row, model.copies["head"], target, loss=loss, weight_layout=LINEAR, ws=ws, prepare=True)
    out = []
    for t in range(h.shape[0]):
        row.copy_(h[t:t + 1])
        target.copy_(targets[t:t + 1])
        call()
        out.append(loss.clone())
    return torch.cat(out)


def main():
    for kw in (dict(), dict(pieces=4), dict(eight=True)):
        losses, norms, model = train(**kw)
        ids, targets = data(512, 1000)
        batch = model.forward(ids, targets)[:32]
        single = score(model, model.block.out[:32], targets[:32])
        torch.cuda.synchronize()
        print("%-16s loss %.4f -> %.4f, norm %.3f -> %.3f; one token at a time: largest difference %.2g" %
              (kw or "fp32 states", losses[0], losses[-1], norms[0], norms[-1], float((single - batch).abs().max())))


if __name__ == "__main__":
    main()
